"""The quantised latent cache at the ends of its ranges: scales far apart, rows of nothing, queries and rows of any size,
codes that are no numbers, many short items, and the merge over a list of any contents."""
import math
import random

import pytest

from test_gpu_5_operators import BOUNDS, D, SCALE, attend, gen, m, randn  # noqa: F401
from test_gpu_6_operator_edges import capped  # noqa: F401
from test_gpu_7_operator_draws import check_formula
from test_gpu_8_quant import ALL, Cache, attention, check_tokens, keys, page_bytes, power, quantised, values

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def places(c, b, n):
    js = torch.arange(n, device="cuda")
    return c.table[b].long()[js // c.rpp], js % c.rpp


def set_scales(c, b, codes):
    """Scale codes of a sequence's rows: [n] (all four blocks) or [n, 4]."""
    page, slot = places(c, b, len(codes))
    c.scales()[page, slot] = (codes if codes.dim() == 2 else codes.view(-1, 1).expand(-1, 4)).to(torch.uint8)


def set_codes(c, b, codes):
    page, slot = places(c, b, len(codes))
    c.codes()[page, slot] = codes.to(torch.uint8)


FORMS = [(16, 1, 256), (128, 3, 3000), (128, 310, 1000)]  # heads, new tokens, rows: one item, cut row tiles, whole row tiles


@pytest.mark.parametrize("H,q_len,n", FORMS)
@pytest.mark.parametrize("first,second", [(147, 12), (12, 147), (146, 12), (200, 60), (60, 200), (127, 11), (246, 11),
                                          (11, 246), (140, 70)])
def test_tiles_whose_scales_lie_far_apart(m, H, q_len, n, first, second):  # noqa: F811
    """Tiles of 128 rows with one scale each, by turns of two: every row counts in the sum of the weights."""
    g = gen(first)
    c = Cache(g, [n], 64)
    js = torch.arange(n, device="cuda")
    set_scales(c, 0, torch.where(js // 128 % 2 == 0, first, second))
    # logits of a few units: a row's values are some 2^7 times its scale
    q = (randn(g, q_len, H, D).double() * power(torch.tensor(127 - 7 - max(first, second), device="cuda"))).to(torch.bfloat16)
    q[:, ::3] = 0
    out, lse = attention(m, c, q, [q_len], [n])
    assert m.csa_read_device_status() == 0
    check_tokens(c, q, out, lse, [q_len], [n], ALL, 0, [(0, i) for i in {0, q_len // 2, q_len - 1}])


def check_tiny(c, q, out, lse, n, tokens):
    """As check_tokens, with what results below 2^-126 lose as bf16: half of their step of 2^-133 at most."""
    for i in tokens:
        kv = c.rows(0, range(n - q.shape[0] + i + 1))
        o, l, to, tl = attend(q[i].double(), kv)
        assert float(((out[i].double() - o).abs() - to - 2.0**-133).max()) <= 0, i
        assert float(((lse[i].double() - l).abs() - tl).max()) <= 0, i


@pytest.mark.parametrize("H,q_len,n", FORMS)
@pytest.mark.parametrize("scale", [0, 1, 5, 6, 9, 10, 11, 20])
def test_rows_of_next_to_nothing(m, H, q_len, n, scale):  # noqa: F811
    """The least scales there are, with codes of 0 (a pool of zero bytes has scales of 0) and with others."""
    g = gen(scale)
    c = Cache(g, [n], 64)
    q = randn(g, q_len, H, D)
    c.scales()[:] = scale
    kept = c.codes().clone()
    c.codes()[:] = 0
    out, lse = attention(m, c, q, [q_len], [n])
    assert m.csa_read_device_status() == 0
    assert bool((out == 0).all())
    want = torch.log(torch.arange(n - q_len + 1, n + 1, device="cuda").double()).view(-1, 1)
    assert float(((lse.double() - want).abs() - 2.0**-20 * (1 + want)).max()) <= 0
    c.codes()[:] = kept
    out, lse = attention(m, c, q, [q_len], [n])
    check_tiny(c, q, out, lse, n, sorted({0, q_len // 2, q_len - 1}))
    # some rows of ordinary size among them
    set_scales(c, 0, torch.where(torch.arange(n, device="cuda") % 97 == 5, 118, scale))
    out, lse = attention(m, c, q, [q_len], [n])
    check_tokens(c, q, out, lse, [q_len], [n], ALL, 0, [(0, i) for i in {0, q_len // 2, q_len - 1}])


@pytest.mark.parametrize("H,q_len,n", FORMS)
@pytest.mark.parametrize("size,scale", [(100, 190), (126, 240), (30, 246), (60, 220), (126, 127)])
def test_large_queries_that_large_rows_do_not_meet(m, H, q_len, n, size, scale):  # noqa: F811
    """Queries in the first 128 dims, rows in the others: every logit is 0, whatever the sizes."""
    g = gen(size)
    c = Cache(g, [n], 64)
    q = (randn(g, q_len, H, D).double().clamp(-1.5, 1.5) * power(torch.tensor(size, device="cuda"))).to(torch.bfloat16)
    q[..., 128:] = 0
    c.codes()[..., :128] = 0
    c.scales()[:] = scale
    set_scales(c, 0, torch.where(torch.arange(n, device="cuda") // 128 % 2 == 0, scale, scale - 20))
    out, lse = attention(m, c, q, [q_len], [n])
    assert m.csa_read_device_status() == 0
    check_tokens(c, q, out, lse, [q_len], [n], ALL, 0, [(0, i) for i in {0, q_len // 2, q_len - 1}])


@pytest.mark.parametrize("H,q_len,n", FORMS)
@pytest.mark.parametrize("size,scale", [(-118, 248), (-110, 244), (-124, 252), (80, 30), (94, 12)])
def test_small_queries_of_large_rows_and_the_other_way_round(m, H, q_len, n, size, scale):  # noqa: F811
    """Logits of ordinary size from factors that are near the ends of the range.  A weight times its row's scale is kept in
    fp16 over the largest such product so far, which counts between 2^7 and 2^15: it is off by up to half of fp16's least
    step, 2^-25, beside what attend() counts, so by 2^-32 of the largest product at most, times the row's value over
    its scale.  (Rows of one scale in a tile, or 2^20 apart: each is kept over its own.)"""
    g = gen(scale)
    c = Cache(g, [n], 64)
    c.codes()[:] = torch.randint(0, 0x38, c.codes().shape, generator=g, device="cuda").to(torch.uint8)  # values below 1
    c.codes()[:] += (128 * torch.randint(0, 2, c.codes().shape, generator=g, device="cuda")).to(torch.uint8)
    c.scales()[:] = scale
    # rows of next to nothing in every other tile: tiles in which each row keeps a scale of its own
    js = torch.arange(n, device="cuda")
    set_scales(c, 0, torch.where((js // 128 % 2 == 0) & (js % 3 == 0), scale - 20 if scale > 40 else scale + 20, scale))
    q = (randn(g, q_len, H, D).double() * power(torch.tensor(size, device="cuda"))).to(torch.bfloat16)
    out, lse = attention(m, c, q, [q_len], [n])
    assert m.csa_read_device_status() == 0
    for i in {0, q_len // 2, q_len - 1}:
        kv = c.rows(0, range(n - q_len + i + 1))
        x = SCALE * (q[i].double() @ kv.t())
        d = float(2.0**-14 * SCALE * (q[i].double().abs() @ kv.abs().t()).amax())
        assert 2.0**-6 < float(x.abs().max()) and d < 2.0**8  # (2^22 of scale * sum |q_i k_i| at most)
        o, l, to, tl = attend(q[i].double(), kv)
        page, slot = places(c, 0, kv.shape[0])
        s = power(c.scales()[page, slot, 0].long() - 127)
        y = (torch.exp(x - l[:, None]) * s).amax(-1)
        to = to + 2.0**-32 * y[:, None] * (kv.abs() / s[:, None]).sum(0)
        assert float(((out[i].double() - o).abs() - to).max()) <= 0, i
        assert float(((lse[i].double() - l).abs() - tl).max()) <= 0, i


def test_codes_that_are_no_numbers(m):  # noqa: F811
    """The codes 0x7F and 0xFF are NaN in attention: those who see one get NaN, nobody else does."""
    g = gen(31)
    lens, n, W = [390, 2], [400, 300], 100
    c = Cache(g, n, 64)
    for b, j, d, code in ((0, 40, 5, 0x7F), (0, 250, 500, 0xFF), (1, 100, 300, 0x7F)):
        c.codes()[c.table[b, j // 64], j % 64, d] = code
    bad = {0: {40, 250}, 1: {100}}
    q = randn(g, sum(lens), 16, D)
    out, lse = attention(m, c, q, lens, n, W, 3)
    assert m.csa_read_device_status() == 0
    nan = 0
    for b, i in [(0, i) for i in range(0, 390, 13)] + [(0, 30), (0, 29), (0, 129), (0, 130), (1, 0), (1, 1)]:
        p, t = n[b] - lens[b] + i, (0, 390)[b] + i
        js = keys(p, W, 3)
        kv = c.rows(b, js)
        for k, j in enumerate(js):
            if j in bad[b]:
                kv[k, 0] = math.nan
        nan += not bool(torch.isfinite(kv).all())
        check_formula(out[t], lse[t], q[t].double(), kv, (b, i))
    assert nan >= 8
    out, lse = attention(m, c, q, [0, 2], n)             # without a window
    assert bool(torch.isnan(out[:2]).all()) and bool(torch.isnan(lse[:2]).all())


def test_nan_before_logits_of_minus_infinity(m):  # noqa: F811
    """A NaN in the first of the pieces that many rows are worked off in, and logits of -infinity in all of the last one."""
    g = gen(32)
    n, q_len, H, piece = 530000, 305, 128, 4096 * 128
    c = Cache(g, [n], 64, fill=False)
    c.codes()[:] = torch.randint(0, 0x38, c.codes().shape, generator=g, device="cuda", dtype=torch.uint8)
    c.scales()[:] = 127
    js = torch.arange(piece, n, device="cuda")
    page = c.table[0].long()[js // 64]
    c.codes()[page, js % 64, 0] = 0x7E                   # 448 * 2^127 is an infinity
    c.scales()[page, js % 64, 0] = 254
    c.codes()[page, js % 64, 1:128] = 0
    q = randn(g, q_len, H, D)
    q[..., 0] = -1
    out, lse = attention(m, c, q, [q_len], [n])
    assert m.csa_read_device_status() == 0
    assert bool(torch.isfinite(lse).all()) and bool(torch.isnan(out[..., 0]).all()) and bool(torch.isfinite(out[..., 1:]).all())
    c.scales()[c.table[0, 9], 3, 1] = 255
    out, lse = attention(m, c, q, [q_len], [n])
    assert bool(torch.isnan(lse).all()) and bool(torch.isnan(out).all())


@pytest.mark.parametrize("rows", [1, 40, 5000])
def test_merge_over_any_list(m, rows):  # noqa: F811
    """The merge's list of runs as a call whose waits ran out may leave it: what an earlier call or nobody wrote.  It merges
    what names rows and partial results that there are, and writes nowhere else."""
    slots, QR = min(128, rows), 76
    need = m.csa_quant_attn_workspace_size(1, 1, slots, slots, 1, 0)
    r = random.Random(rows)
    big = [-1, 0, 1, QR, QR + 1, 127, 128, 129, rows - 1, rows, rows + 1, 1 << 20, (1 << 31) - 1, -(1 << 31), 0x7F7F7F7F]
    for turn in range(40):
        ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
        at = (-ws.data_ptr()) % 256
        lst = []
        for k in range(QR + 1):
            if r.random() < 0.5:  # one that may be right
                n = r.randint(0, slots)
                lst.append([r.randint(0, rows - n), n, min(QR - 1, k + r.randint(0, 3))])
            else:
                lst.append([r.choice(big), r.choice(big), r.choice(big)])
        lst[QR][0] = r.choice([QR, QR, QR, 5, *big])
        ws[at: at + 12 * (QR + 1)] = torch.tensor(lst, dtype=torch.int32).view(torch.uint8).view(-1).cuda()
        if turn == 0:  # all bits set
            ws.fill_(255)
            lst = [[-1, -1, -1]] * (QR + 1)
        guard = 300
        buf = torch.full((rows + 2 * guard, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((rows + 2 * guard,), 7.0, device="cuda")
        m.csa_selftest_quant_merge(ws[at:], need, rows, buf[guard: guard + rows], lse[guard: guard + rows])
        assert m.csa_read_device_status() == 0
        runs = lst[QR][0] if 0 <= lst[QR][0] <= QR else 0
        named = torch.zeros(rows + 2 * guard, dtype=torch.bool, device="cuda")
        for k, (row0, n, last) in enumerate(lst[:runs]):
            if k < last < runs and 0 < n <= slots and 0 <= row0 <= rows - n:
                named[guard + row0: guard + row0 + n] = True
        assert turn == 0 or runs < 20 or bool(named.any())
        assert bool((buf[~named] == 7).all()) and bool((lse[~named] == 7).all())
        assert not bool((lse[named] == 7).any())


def test_unwritten_runs_are_empty(m, capped):  # noqa: F811
    """The list of runs in the workspace of a call with few row tiles: whatever it held, every run is named in it, those without
    a row tile that is cut as empty."""
    g = gen(33)
    n, QR = [3000, 40], 76
    c = Cache(g, n, 64)
    q = randn(g, 2, 16, D)
    need = m.csa_quant_attn_workspace_size(2, 16, 2, 1, ALL, 0)
    for pairs in (0, 1, 13):
        capped(pairs)
        ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
        at = (-ws.data_ptr()) % 256
        attention(m, c, q, [1, 1], n, workspace=ws[at:], ws_bytes=need)
        lst = ws[at: at + 12 * (QR + 1)].clone().view(torch.int32).view(-1, 3).tolist()
        # 24 + 3 places and 1 + 3, two to a run
        assert lst[QR][0] == 16
        assert lst[0] == [0, 16, 11] and all(lst[k] == [0, 0, k] for k in range(1, QR))
    assert m.csa_read_device_status() == 0


@pytest.mark.parametrize("B,pairs", [(200, 1), (200, 3), (280, 1), (280, 0)])
def test_many_short_items(m, capped, B, pairs):  # noqa: F811
    """Row tiles of a key tile or two, or of none, one behind the other: the next items' queries come while an item is worked
    on.  The same bits every time."""
    g = gen(34)
    H = 128
    lens = [(1, 1, 2, 0, 1)[i % 5] for i in range(B)]
    n = [(1, 130, 17, 9, 0, 128, 3)[i % 7] for i in range(B)]
    c = Cache(g, n, 64)
    q = randn(g, sum(lens), H, D)
    capped(pairs)
    out, lse = attention(m, c, q, lens, n)
    assert m.csa_read_device_status() == 0
    check_tokens(c, q, out, lse, lens, n, ALL, 0, [(b, i) for b in (*range(0, 14), *range(B - 7, B)) for i in range(lens[b])])
    for _ in range(100):
        got = attention(m, c, q, lens, n)
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)
    assert m.csa_read_device_status() == 0


def test_codes_that_are_no_numbers_beside_infinite_rows(m):  # noqa: F811
    """A query with a logit of -infinity has NaN where the rows that it sees are not finite, whole where one of its own logits is
    NaN: the same for a code of NaN in a run of its own."""
    g = gen(35)
    n, H = 3000, 16
    c = Cache(g, [n], 64)
    c.codes()[:] = c.codes() % 128 % 0x38 + c.codes() // 128 * 128  # values below 1
    c.scales()[:] = 127
    page, slot = places(c, 0, n)
    c.codes()[page[5], slot[5], :128] = 0
    c.codes()[page[5], slot[5], 3] = 0x7E
    c.scales()[page[5], slot[5], 0] = 254                # an infinity in dim 3 of row 5
    c.codes()[page[2900], slot[2900], 400] = 0xFF
    q = randn(g, 120, H, D)
    q[..., 3] = -1
    out, lse = attention(m, c, q, [120], [n])
    assert m.csa_read_device_status() == 0
    for i in (0, 19, 20, 21, 119):                       # row 2900 is the 21st token's own
        kv = c.rows(0, range(n - 120 + i + 1))
        if i >= 20:
            kv[2900, 400] = math.nan
        nan = torch.isnan(torch.softmax(SCALE * (q[i].double() @ kv.t()), -1) @ kv)
        assert torch.equal(torch.isnan(out[i]), nan), i
        assert bool(torch.isnan(lse[i]).all()) == (i >= 20)
    assert bool(torch.isfinite(out[:20, :, 4:]).all()) and bool(torch.isnan(out[:, :, 3]).all())


@pytest.mark.parametrize("B", [257, 5000, 65535])
def test_batches_of_very_many_sequences(m, B):  # noqa: F811
    """A row of each sequence, and batches that have next to no rows; whichever sequence is outside is reported."""
    g = gen(B)
    pool = torch.zeros(B, page_bytes(1), dtype=torch.uint8, device="cuda")
    table = torch.randperm(B, generator=g, device="cuda").to(torch.int32).view(B, 1)
    kv = m.paged(pool, 1, 516, table, page_stride_bytes=pool.shape[1], n_pages=B)
    x = randn(g, B, D)
    at, n = torch.arange(B + 1, device="cuda"), torch.ones(B, dtype=torch.int64, device="cuda")
    m.csa_quant_write(x, kv, 1, B, at, n, B, 1)
    out = torch.full((B, D), 7.0, dtype=torch.bfloat16, device="cuda")
    m.csa_quant_read(kv, 1, B, at, n, B, 1, out)
    assert m.csa_read_device_status() == 0
    assert torch.equal(out.double(), values(*quantised(x)))
    # one row, the last sequence's; then a sequence without rows that is too long
    at = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
    at[B] = 1
    out.fill_(7.0)
    m.csa_quant_read(kv, 1, B, at, n, 1, 1, out)
    assert m.csa_read_device_status() == 0
    assert torch.equal(out[0].double(), values(*quantised(x[-1:]))[0]) and bool((out[1:] == 7).all())
    for b in (0, 31, 32, 255, 256, B // 2, B - 2):
        n[b] = 1 << 31
        m.csa_quant_read(kv, 1, B, at, n, 1, 1, out)
        assert m.csa_read_device_status() == BOUNDS, b
        m.csa_quant_write(x, kv, 1, B, at, n, 1, 1)
        assert m.csa_read_device_status() == BOUNDS, b
        n[b] = 1


def test_values_next_to_the_largest_number(m):  # noqa: F811
    """Means of values of 1.75 * 2^127 in every partial result: their sum would be none."""
    for H, q_len, n in FORMS:
        c = Cache(gen(36), [n], 64)
        c.codes()[:] = 0x7E                              # 448
        c.codes()[..., ::2] = 0xFE
        c.scales()[:] = 127 + 119
        q = torch.zeros(q_len, H, D, dtype=torch.bfloat16, device="cuda")
        out, lse = attention(m, c, q, [q_len], [n])
        assert m.csa_read_device_status() == 0
        v = 1.75 * 2.0**127
        assert bool(((out[..., 1::2].double() - v).abs() <= 2.0**-7 * v).all())  # (2^-8 of the values, 2^-8 of the rounding)
        assert bool(((out[..., ::2].double() + v).abs() <= 2.0**-7 * v).all())
        check_tokens(c, q, out, lse, [q_len], [n], ALL, 0, [(0, q_len - 1)])


def check_any_scales(c, b, q, out, lse, n, where):
    """Rows of any finite scales.  Beside what attend() counts: a row's values are kept in fp16 as 2^7 times their ratio to its unit,
    the power of two of its tile's largest scale or, where the tile's rows are more than 2^15 apart, of its own largest.  So
    they are known to 2^-32 of the unit (half of fp16's least step, 2^-25, over 2^7); a block whose scale is 2^32 and
    more below has no such ratio (2^-25 is no fp16 number) and may count as 0.  A query's values are known to 2^-39 of its
    largest, and a weight times its unit to 2^-32 of the largest such product
    (test_small_queries_of_large_rows_and_the_other_way_round).  A logit's error moves a weight by twice that."""
    js = torch.arange(n, device="cuda")
    page = c.table[b].long()[js // c.rpp]
    scale = c.scales()[page, js % c.rpp].long()
    top = scale.amax(-1)
    unit = top.clone()
    for t in range(0, n, 128):
        rows = top[t: t + 128]
        some = rows[rows > 10]
        if len(some) and int(rows.max() - some.min()) <= 15:
            unit[t: t + 128] = rows.max()
    lost = (unit[:, None] - scale >= 32).repeat_interleave(128, 1)
    unit = power(unit - 127)
    kv = c.rows(b, range(n))
    off = torch.where(lost, kv.abs(), 2.0**-32 * unit[:, None])
    x = SCALE * (q @ kv.t())
    full = torch.logsumexp(x, -1)
    w = torch.exp(x - full[:, None])
    o, a = w @ kv, w @ kv.abs()
    d = 2.0**-14 * SCALE * (q.abs() @ kv.abs().t()).amax(-1)
    if float(d.max()) > 2.0**8:
        return False                                     # no defined result
    d = d + SCALE * ((q.abs() @ off.t()).amax(-1) + 2.0**-39 * q.abs().amax(-1) * kv.abs().sum(-1).amax())
    ok = d < 0.25                                        # (e^(2 d) - 1 <= 3 d)
    to = 2.0**-8 * (a + o.abs()) + (3 * d[:, None] + 2.0**-20) * a + 2.0**-133
    to = to + w @ off + (2.0**-32 * (w * unit).amax(-1) * (kv.abs() / unit[:, None]).sum(0).amax())[:, None]
    assert float(((out.double() - o).abs() - to)[ok].max() if bool(ok.any()) else -1) <= 0, where
    assert float(((lse.double() - full).abs() - d - 2.0**-20 * (1 + full.abs())).max()) <= 0, where
    return True


@pytest.mark.parametrize("seed", range(40))
def test_drawn_scales(m, seed):  # noqa: F811
    """Scales drawn for the cache, its tiles, its rows and their blocks; queries as large as they may be for them."""
    r, g = random.Random(seed), gen(seed)
    H, q_len, n = r.choice(FORMS + [(24, 7, 500), (128, 320, 400), (1, 1, 130)])
    c = Cache(g, [n], r.choice((64, 16, 17, 1)))
    js = torch.arange(n, device="cuda")

    def spread(count, most):
        return torch.randint(-most, most + 1, (count,), generator=g, device="cuda")

    s = torch.full((n, 4), r.randint(0, 246), device="cuda")
    s += spread(n // 128 + 1, r.choice((0, 0, 3, 20, 60, 120)))[js // 128][:, None]
    s += spread(n, r.choice((0, 0, 2, 7, 16, 40)))[:, None]
    s += spread(4 * n, r.choice((0, 1, 4, 12))).view(n, 4)
    s = s.clamp(0, 246)
    set_scales(c, 0, s)
    if r.random() < 0.3:
        set_scales(c, 0, torch.where((js % r.choice((2, 50, 300)) == 1)[:, None], torch.full_like(s, r.choice((0, 10, 11))), s))
    if r.random() < 0.3:
        set_codes(c, 0, torch.where((js % r.choice((2, 50, 300)) == 0)[:, None], 0, c.codes()[places(c, 0, n)]))
    big = float(c.rows(0, range(n)).abs().max()) or 1.0
    size = math.floor(math.log2(2.0 ** r.choice((-20, 0, 3, 6)) / big))
    q = (randn(g, q_len, H, D).double() * power(torch.tensor(max(-126, min(size, 126)), device="cuda"))).to(torch.bfloat16)
    if r.random() < 0.3:
        q[:, :, r.randrange(512):] = 0
    out, lse = attention(m, c, q, [q_len], [n])
    assert m.csa_read_device_status() == 0
    for i in {0, q_len // 2, q_len - 1}:
        check_any_scales(c, 0, q[i].double(), out[i], lse[i], n - q_len + i + 1, (seed, i))


@pytest.mark.parametrize("H,q_len,n", FORMS)
def test_buffers_and_workspaces_that_are_16_byte_aligned_and_no_more(m, H, q_len, n):  # noqa: F811
    g = gen(37)
    c = Cache(g, [n], 64)
    q = randn(g, q_len, H, D)
    want = attention(m, c, q, [q_len], [n])
    q2 = torch.empty(q.numel() + 8, dtype=torch.bfloat16, device="cuda")[8:].view_as(q).copy_(q)
    out = torch.empty(q.numel() + 8, dtype=torch.bfloat16, device="cuda")[8:].view_as(q)
    lse = torch.empty(q_len * H + 1, device="cuda")[1:].view(q_len, H)
    need = m.csa_quant_attn_workspace_size(1, H, q_len, q_len, ALL, 0)
    ws = torch.full((need + 32,), 255, dtype=torch.uint8, device="cuda")[16:]
    assert q2.data_ptr() % 32 == 16 and out.data_ptr() % 32 == 16 and lse.data_ptr() % 8 == 4 and ws.data_ptr() % 32 == 16
    m.csa_quant_attn(q2, H, SCALE, c.paged(m), c.width, 1, torch.tensor([0, q_len], device="cuda"),
                     torch.tensor([n], device="cuda"), q_len, q_len, ALL, 0, out, lse, ws, need)
    assert m.csa_read_device_status() == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert bool((ws[need:] == 255).all())


@pytest.mark.parametrize("H,q_len,n", [(1, 20, 60), (1, 64, 90), (1, 100, 300), (16, 3, 90), (16, 4, 1000), (16, 5, 200), (24, 2, 2),
                                       (64, 3, 140), (100, 2, 130), (128, 3, 129)])
@pytest.mark.parametrize("scale", [255, 254])
def test_no_numbers_that_later_tokens_see(m, H, q_len, n, scale):  # noqa: F811
    """A row that is no number, or infinite, among a batch's new tokens: those before it are not touched, in any block of
    dims, however few query rows there are."""
    for block in range(4):
        g = gen(38 + block)
        c = Cache(g, [n], 64)
        c.codes()[:] = c.codes() % 128 % 0x38 + c.codes() // 128 * 128
        c.scales()[:] = 127
        at = n - 1 - q_len // 2 if q_len > 2 else n - 1
        page, slot = places(c, 0, n)
        c.scales()[page[at], slot[at], block] = scale
        c.codes()[page[at], slot[at], 128 * block: 128 * block + 128: 3] = 0x7E
        q = randn(g, q_len, H, D)
        out, lse = attention(m, c, q, [q_len], [n])
        assert m.csa_read_device_status() == 0
        check_tokens(c, q, out, lse, [q_len], [n], ALL, 0, [(0, i) for i in range(q_len)])
        before = q_len - (n - at)
        assert before >= 1 and bool(torch.isfinite(out[:before]).all()) and not bool(torch.isfinite(out[before]).all())


@pytest.mark.parametrize("H,q_len,n", FORMS)
@pytest.mark.parametrize("below", [14, 15, 16, 21, 22, 24, 25, 28, 31])
def test_blocks_far_below_their_rows_largest(m, H, q_len, n, below):  # noqa: F811
    """Three blocks of a row below the other, up to 2^31: queries in those three see them, and outputs have them."""
    g = gen(39)
    c = Cache(g, [n], 64)
    js = torch.arange(n, device="cuda")
    big = js * 7 % 4                                     # the large block differs from row to row
    s = torch.full((n, 4), 110 - below, device="cuda")
    s[js, big] = 110
    codes = torch.randint(0x40, 0x7F, (n, D), generator=g, device="cuda") + 128 * torch.randint(0, 2, (n, D), generator=g, device="cuda")
    codes.view(n, 4, 128)[js, big] = 0x00                # and has nothing in it but one value
    codes.view(n, 4, 128)[js, big, 5] = 0x7E
    set_scales(c, 0, s)
    set_codes(c, 0, codes)
    q = (randn(g, q_len, H, D).double() * power(torch.tensor(17 + below - 8, device="cuda"))).to(torch.bfloat16)
    q.view(q_len, H, 4, 128)[..., 5] = 0                 # (which no query meets)
    out, lse = attention(m, c, q, [q_len], [n])
    assert m.csa_read_device_status() == 0
    for i in {0, q_len // 2, q_len - 1}:
        assert check_any_scales(c, 0, q[i].double(), out[i], lse[i], n - q_len + i + 1, i)
