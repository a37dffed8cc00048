"""The attention operators where the device, the arguments or the cache are at an edge: fewer SMs than the plan
counts on, infinities in rows that are attended, lengths out of range, streams given by the caller."""
import math

import pytest

from test_gpu_5_operators import (BOUNDS, D, RUNS, SCALE, Cache, attend, check, check_window, gen, m, prefix,  # noqa: F401
                                  randn, window)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# ------------------------------------------------------------------ fewer pairs of SMs than the plan counts on
@pytest.fixture
def capped(m):  # noqa: F811
    yield m.csa_selftest_pairs
    m.csa_selftest_pairs(0)


def dirty(need):
    """A workspace of NaN: what no item wrote shows."""
    return torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("pairs", [1, 13, 75])
@pytest.mark.parametrize("H,shared,n_rows,rpp", RUNS + [
    (16, 9001, [9001 + (i * 53) % 400 for i in range(32)], 48),   # splits
    (20, 130, [131, 200, 130, 177, 900], 17),
])
def test_prefix_attention_on_fewer_pairs(m, capped, H, shared, n_rows, rpp, pairs):  # noqa: F811
    g = gen(41)
    c = Cache(g, [max(n, shared) for n in n_rows], rpp, min(shared, max(n_rows)))
    q = randn(g, len(n_rows), H, D)
    need = m.csa_prefix_attn_workspace_size(len(n_rows), H, shared, max(max(n_rows), shared))
    want, lse = prefix(m, q, c, shared, n_rows, workspace=dirty(need), ws_bytes=need)
    capped(pairs)
    out, lse2 = prefix(m, q, c, shared, n_rows, workspace=dirty(need), ws_bytes=need)
    assert torch.equal(out, want) and torch.equal(lse, lse2)
    assert m.csa_read_device_status() == 0


@pytest.mark.parametrize("pairs", [1, 13, 75])
@pytest.mark.parametrize("H,q_len,n_tokens,W,S", [(24, [300, 41], [300, 900], 100, 5), (16, [1, 1], [3000, 70], 2000, 4)])
def test_window_attention_on_fewer_pairs(m, capped, H, q_len, n_tokens, W, S, pairs):  # noqa: F811
    g = gen(42)
    c = Cache(g, n_tokens, 64)
    q = randn(g, sum(q_len), H, D)
    need = m.csa_window_attn_workspace_size(len(q_len), H, sum(q_len), max(q_len), W, S)
    want, lse = window(m, q, c, q_len, n_tokens, W, S, workspace=dirty(need), ws_bytes=need)
    capped(pairs)
    out, lse2 = window(m, q, c, q_len, n_tokens, W, S, workspace=dirty(need), ws_bytes=need)
    assert torch.equal(out, want) and torch.equal(lse, lse2)
    assert m.csa_read_device_status() == 0


# ------------------------------------------------------------------ a stream given with the call
@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("call", ["prefix", "window", "pages"])
def test_scratch_of_a_call_on_another_stream(m, call, as_handle):  # noqa: F811
    """Memory that was given back with a copy from it still pending on the current stream is no scratch for a call on
    another one."""
    g = gen(49)
    n_rows = [2000, 2100]
    c = Cache(g, n_rows, 64, 1900)
    q = randn(g, 2, 16, D)
    n, off = (torch.tensor(x, dtype=torch.int64, device="cuda") for x in (n_rows, [0, 1, 2]))
    out, lse = torch.zeros_like(q), torch.zeros(2, 16, dtype=torch.float32, device="cuda")
    pages = 1 << 20
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table, first, count = torch.full((1, 9), -1, dtype=torch.int32, device="cuda"), refs.new_zeros(1), refs.new_ones(1)
    need = {"prefix": m.csa_prefix_attn_workspace_size(2, 16, 1900, 2100),
            "window": m.csa_window_attn_workspace_size(2, 16, 2, 1, 900, 4),
            "pages": m.csa_pages_workspace_size(pages)}[call]
    assert need > 1 << 16
    side = torch.cuda.Stream()
    held = torch.full((need,), 1, dtype=torch.uint8, device="cuda")
    copy = torch.zeros_like(held)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    copy.copy_(held)
    del held
    s = side.cuda_stream if as_handle else side
    if call == "prefix":
        m.csa_prefix_attn(q, 2, 16, SCALE, c.paged(m), c.width, 1900, n, 2100, out, lse, stream=s)
    elif call == "window":
        m.csa_window_attn(q, 16, SCALE, c.paged(m), c.width, 2, off, n, 2, 1, 900, 4, out, lse, stream=s)
    else:
        m.csa_pages_alloc(refs, pages, table, 9, 1, first, count, stream=s)
    torch.cuda.synchronize()
    assert bool((copy == 1).all())
    if call == "pages":
        assert table.tolist() == [[0] + [-1] * 8] and int(refs.sum()) == 1
    for b in range(2) if call != "pages" else ():
        keys = range(n_rows[b]) if call == "prefix" else list(range(4)) + list(range(n_rows[b] - 900, n_rows[b]))
        check(out[b], lse[b], attend(q[b].double(), c.rows(b, keys)), f"request {b}")
    assert m.csa_read_device_status() == 0


def test_scratch_of_a_call_on_the_default_stream(m):  # noqa: F811
    """The handle 0 is the default stream, whatever stream is the current one."""
    g = gen(50)
    c = Cache(g, [700], 64)
    q = randn(g, 1, 16, D)
    n, out = torch.tensor([700], dtype=torch.int64, device="cuda"), torch.zeros_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        m.csa_prefix_attn(q, 1, 16, SCALE, c.paged(m), c.width, 600, n, 700, out, stream=0)
    torch.cuda.synchronize()
    w = attend(q[0].double(), c.rows(0, range(700)))
    check(out[0], w[1].float(), w, "prefix")


# ------------------------------------------------------------------ lengths out of range, no rows of their own
@pytest.mark.parametrize("B,H,shared", [(3, 16, 100), (12, 128, 6000), (5, 7, 1)])
@pytest.mark.parametrize("n", [1, 1 << 31, (1 << 63) - 1, -1, -(1 << 63)])
def test_prefix_attention_reports_lengths_where_every_row_is_shared(m, B, H, shared, n):  # noqa: F811
    """max_rows = n_shared: a length above it (by 1 and more) or below 0 is reported, and taken for the nearest one."""
    g = gen(48)
    c = Cache(g, [shared] * B, 64, shared)
    n_rows = [shared] * B
    q = randn(g, B, H, D)
    want, lse = prefix(m, q, c, shared, n_rows)
    assert m.csa_read_device_status() == 0
    n_rows[B - 1] = n if n < 0 or n > 1 else shared + n
    out, lse2 = prefix(m, q, c, shared, n_rows, max_rows=shared)
    assert m.csa_read_device_status() == BOUNDS
    last = B - 1 if n < 0 else B
    assert torch.equal(out[:last], want[:last]) and torch.equal(lse[:last], lse2[:last])
    assert n > 0 or (bool((out[last] == 0).all()) and bool((lse2[last] == -math.inf).all()))


# ------------------------------------------------------------------ infinities in rows that are attended
def check_readers(out, lse, q, kv, where):
    """Against the formula, element for element: a logit of +inf or NaN leaves nothing but NaN; one of -inf has the
    weight 0, and 0 times what its row holds is NaN where that is not finite.  What stays finite is what the other
    rows give."""
    x = SCALE * (q @ kv.t())
    w = torch.exp(x - torch.logsumexp(x, -1, keepdim=True))
    nan = torch.isnan(w @ kv)
    assert torch.equal(torch.isnan(out), nan), f"{where}: {int((torch.isnan(out) != nan).sum())} of {nan.sum()}"
    o, l, to, tl = attend(q, kv[torch.isfinite(kv).all(1)])
    off = torch.where(nan, torch.zeros_like(o), (out.double() - o).abs() - to)
    assert float(off.max()) <= 0, where
    fin = torch.isfinite(torch.logsumexp(x, -1))
    assert bool((~torch.isfinite(lse[~fin])).all()), where
    if bool(fin.any()):
        assert float(((lse.double() - l).abs() - tl)[fin].max()) <= 0, where


@pytest.mark.parametrize("rpp", [64, 40])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
@pytest.mark.parametrize("j", [100, 650, 690, 699, 1279, 1280, 1299])
def test_prefix_attention_readers_of_an_infinity(m, rpp, value, j):  # noqa: F811
    """Rows of tiles that every request sees whole, of tiles that one sees in part, and of a request's own."""
    g = gen(43)
    shared, n_rows = 1280, [1300, 1280, 700, 1281]
    c = Cache(g, [1300] * 4, rpp, shared)
    for b in range(4):
        c.pool[c.row(0 if j < shared else b, j), 17] = value
    q = randn(g, 4, 30, D)
    out, lse = prefix(m, q, c, shared, n_rows)
    for b, n in enumerate(n_rows):
        kv = torch.cat([c.rows(0, range(min(n, shared))), c.rows(b, range(shared, n))])
        check_readers(out[b], lse[b], q[b].double(), kv, f"request {b}")
    assert m.csa_read_device_status() == 0


@pytest.mark.parametrize("bad", [[0], [30], [30, 31, 69], list(range(70))])
def test_prefix_attention_readers_of_infinities_in_one_item(m, bad):  # noqa: F811
    """A whole context of one tile, of which any row may be the only one that a request attends."""
    g = gen(44)
    n_rows = [70, 1, 33, 64]
    c = Cache(g, n_rows, 16)
    for b in range(4):
        for j in bad:
            if j < n_rows[b]:
                c.pool[c.row(b, j), 500] = math.inf
    q = randn(g, 4, 33, D)
    out, lse = prefix(m, q, c, 0, n_rows)
    for b, n in enumerate(n_rows):
        check_readers(out[b], lse[b], q[b].double(), c.rows(b, range(n)), f"request {b}")


@pytest.mark.parametrize("H,shared,n", [(128, 256, 300), (16, 2000, 2100), (40, 0, 128)])
def test_prefix_attention_readers_of_a_channel_of_infinities(m, H, shared, n):  # noqa: F811
    """Every row holds an infinity at one place: a head's logits are all +inf or all -inf, and no output is finite."""
    g = gen(45)
    c = Cache(g, [n, n], 64, shared)
    c.pool[:, 9] = math.inf
    q = randn(g, 2, H, D)
    out, lse = prefix(m, q, c, shared, [n, n])
    assert bool(torch.isnan(out).all()) and not bool(torch.isfinite(lse).any())


@pytest.mark.parametrize("rpp", [64, 24])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
@pytest.mark.parametrize("p", [1, 330, 380, 399])
@pytest.mark.parametrize("H", [16, 128])
def test_window_attention_readers_of_an_infinity(m, rpp, value, p, H):  # noqa: F811
    """A sink, rows that only earlier or only later tokens of the chunk see, the last row."""
    g = gen(46)
    c = Cache(g, [400], rpp)
    c.pool[c.row(0, p), 300] = value
    q = randn(g, 60, H, D)
    out, lse = window(m, q, c, [60], [400], 50, 3)
    for t in range(0, 60, 1 if H == 16 else 3):
        pos = 340 + t
        kv = c.rows(0, list(range(3)) + list(range(pos - 49, pos + 1)))
        check_readers(out[t], lse[t], q[t].double(), kv, f"position {pos}")
    assert m.csa_read_device_status() == 0


@pytest.mark.parametrize("H,ql,W", [(128, 3, 500), (16, 1, 2000), (8, 1, 2000)])
@pytest.mark.parametrize("back", [0, 3, 140, 300, 499])
def test_window_attention_readers_of_an_infinity_in_wide_windows(m, H, ql, W, back):  # noqa: F811
    """Tiles that every token of an item sees whole, and keys that are split."""
    g = gen(47)
    n = 2500
    c = Cache(g, [n], 64)
    c.pool[c.row(0, n - 1 - back), 0] = math.inf
    q = randn(g, ql, H, D)
    out, lse = window(m, q, c, [ql], [n], W, 0)
    for t in range(ql):
        pos = n - ql + t
        check_readers(out[t], lse[t], q[t].double(), c.rows(0, range(pos - W + 1, pos + 1)), f"position {pos}")


# ------------------------------------------------------------------ pages
@pytest.mark.parametrize("first", [0, 1, 255])
def test_pages_alloc_of_the_longest_row(m, first):  # noqa: F811
    """A table row of 2^31 - 1 entries, all of them (or all but the first ones) asked for, in a pool of seven pages."""
    width = (1 << 31) - 1
    i32 = dict(dtype=torch.int32, device="cuda")
    refs, table = torch.zeros(7, **i32), torch.full((1, width), -9, **i32)
    m.csa_pages_alloc(refs, 7, table, width, 1, torch.tensor([first], **i32), torch.tensor([width - first], **i32))
    assert m.csa_read_device_status() == 1 << 6
    assert refs.tolist() == [1] * 7
    assert table[0, :first].tolist() == [-9] * first and table[0, first:first + 7].tolist() == list(range(7))
    assert all(bool((t == -1).all()) for t in table[0, first + 7:].split(1 << 28))


def real_pools(n_pages, seed=5):
    """Pages of a cache's sizes (raw rows, compressed rows, index keys) and of one that ends inside a piece of its
    copy, in a pool whose pages lie apart; random bytes."""
    g = gen(seed)
    words = (16384, 4096, 1024, 6164 + 12)
    p = [torch.randint(-2**31, 2**31 - 1, (n_pages, w), generator=g, device="cuda", dtype=torch.int32) for w in words]
    return p[:3] + [p[3][:, 4:6168]], p[3]


def test_pages_of_real_sizes(m):  # noqa: F811
    """Copies, forks and moves of whole pages, byte for byte, every other page and byte left as it was."""
    n_pages, rpp, width = 200, 64, 40
    pools, wide = real_pools(n_pages)
    assert pools[3].stride(0) == 6176 and pools[3].shape[1] * 4 % 8192 not in (0, 16)
    d = m.page_pools(pools, n_pages)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def moved(before, src, dst):
        for p, old in zip(pools, before):
            old[dst] = old[src]
            assert torch.equal(p, old)

    gaps = wide[:, :4].clone(), wide[:, 6168:].clone()
    before = [p.clone() for p in pools]
    m.csa_pages_copy(d, i32([3, 199, 3]), i32([198, 0, 77]), 3)
    moved(before, [3, 199, 3], [198, 0, 77])

    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[::3] = 1
    table = torch.full((6, width), -1, dtype=torch.int32, device="cuda")
    tokens = [30 * rpp + 17, 5 * rpp + 63]
    m.csa_pages_alloc(refs, n_pages, table, width, 6, i32([0] * 6), i32([31, 6, 0, 0, 0, 0]))
    nt = torch.tensor(tokens + [0] * 4, dtype=torch.int64, device="cuda")
    free = [p for p, r in enumerate(refs.tolist()) if r == 0]
    before = [p.clone() for p in pools]
    last = [int(table[0, 30]), int(table[1, 5])]
    m.csa_pages_fork(d, refs, table, width, 6, i32([0, 1, 1, 0]), i32([2, 3, 4, 5]), 4, nt, rpp)
    moved(before, [last[0], last[1], last[1], last[0]], free[:4])
    assert [int(table[2, 30]), int(table[3, 5]), int(table[4, 5]), int(table[5, 30])] == free[:4]

    m.csa_pages_free(refs, n_pages, table, width, 6, i32([0, 4]), 2)
    before = [p.clone() for p in pools]
    n = torch.zeros(1, dtype=torch.int64, device="cuda")
    refs[::3] += 1  # (pages that no table names move too)
    used = [p for p, r in enumerate(refs.tolist()) if r > 0]
    holes = [p for p in range(len(used)) if p not in used]
    m.csa_pages_compact(d, refs, refs, table, table, width, 6, n)
    far = [p for p in used if p >= len(used)]
    assert n.item() == len(used) and 0 < len(far) == len(holes)
    moved(before, far, holes)
    assert torch.equal(wide[:, :4], gaps[0]) and torch.equal(wide[:, 6168:], gaps[1])
    assert m.csa_read_device_status() == 0


# ------------------------------------------------------------------ scales
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-45, -1e-45])
@pytest.mark.parametrize("call", ["prefix", "window"])
def test_attention_of_no_scale_over_large_rows(m, call, scale):  # noqa: F811
    """Logits before scaling of 1e33 to 1e35: every weight is the same (off by 1e35 * 1.4e-45, far below 2^-20)."""
    g = gen(51)
    n_rows, H = [300, 190], 20
    c = Cache(g, n_rows, 32, 160)
    c.pool.mul_(1e16)
    q = randn(g, 2, H, D) * 1e16
    n, off = (torch.tensor(x, dtype=torch.int64, device="cuda") for x in (n_rows, [0, 1, 2]))
    out, lse = torch.zeros_like(q), torch.zeros(2, H, dtype=torch.float32, device="cuda")
    if call == "prefix":
        m.csa_prefix_attn(q, 2, H, scale, c.paged(m), c.width, 160, n, 300, out, lse)
    else:
        m.csa_window_attn(q, H, scale, c.paged(m), c.width, 2, off, n, 2, 1, 70, 3, out, lse)
    for b, x in enumerate(n_rows):
        kv = c.rows(b, range(x) if call == "prefix" else list(range(3)) + list(range(x - 70, x)))
        o, a = kv.mean(0).expand(H, D), kv.abs().mean(0)
        want = torch.full((H,), math.log(len(kv)), dtype=torch.float64, device="cuda")
        check(out[b], lse[b], (o, want, 2.0**-8 * (a + o.abs()) + 2.0**-20 * a, 2.0**-20 * (1 + want)), f"request {b}")
    assert m.csa_read_device_status() == 0


# ------------------------------------------------------------------ bounds and batches
@pytest.mark.parametrize("max_q", [1 << 31, (1 << 63) - 1])
def test_window_attention_with_any_bound_on_new_tokens(m, max_q):  # noqa: F811
    g = gen(52)
    q_len, n_tokens = [40, 1, 3], [300, 2000, 3]
    c = Cache(g, n_tokens, 64)
    q = randn(g, 44, 20, D)
    want, lse = window(m, q, c, q_len, n_tokens, 700, 3, max_q=(1 << 31) - 1)
    out, lse2 = window(m, q, c, q_len, n_tokens, 700, 3, max_q=max_q)
    assert torch.equal(out, want) and torch.equal(lse, lse2)
    check_window(q, c, q_len, n_tokens, 700, 3, out, lse2, every=7)
    assert m.csa_read_device_status() == 0


@pytest.mark.parametrize("H,B", [(1, 300), (2, 131), (3, 90)])
def test_prefix_attention_of_many_requests_with_few_heads(m, H, B):  # noqa: F811
    """Query-row tiles of up to 128 requests, whose lengths lie on both sides of the prefix's end."""
    g = gen(53)
    shared = 333
    n_rows = [(b * 29) % 420 for b in range(B)]
    c = Cache(g, [max(n, shared) for n in n_rows], 16, shared)
    q = randn(g, B, H, D)
    out, lse = prefix(m, q, c, shared, n_rows)
    for b, n in enumerate(n_rows):
        kv = torch.cat([c.rows(0, range(min(n, shared))), c.rows(b, range(shared, n))])
        check(out[b], lse[b], attend(q[b].double(), kv), f"request {b}")
    assert m.csa_read_device_status() == 0


@pytest.mark.parametrize("H,seqs,W,S,rpp", [
    (1, [(500, 500), (1, 2), (130, 900)], 60, 3, 64),
    (2, [(1, 1 + 37 * i) for i in range(140)], 128, 4, 40),   # more sequences than are looked at together
    (127, [(5, 5), (0, 9), (4, 300)], 33, 0, 16),
])
def test_window_attention_of_few_heads_and_many_sequences(m, H, seqs, W, S, rpp):  # noqa: F811
    g = gen(54)
    q_len, n_tokens = [s[0] for s in seqs], [s[1] for s in seqs]
    c = Cache(g, n_tokens, rpp)
    q = randn(g, sum(q_len), H, D)
    out, lse = window(m, q, c, q_len, n_tokens, W, S)
    check_window(q, c, q_len, n_tokens, W, S, out, lse, every=3)
    assert m.csa_read_device_status() == 0


@pytest.mark.parametrize("at", [10, 600, 1900])
@pytest.mark.parametrize("call", ["prefix", "window"])
def test_attention_of_one_dominant_key(m, call, at):  # noqa: F811
    """A key of the first tile far above all others, and one behind it that weighs up to 2^7.9 times as much: no more than
    the running maximum lets pass, so that its weight is far above 1 and rounded."""
    g = gen(55)
    n, H = 2000, 16
    c = Cache(g, [n], 64)
    c.pool.mul_(2.0**-6)
    u = randn(g, D)
    up = torch.linspace(0.05, 0.97, H, device="cuda").view(H, 1)
    q = (u.float() * up).to(torch.bfloat16).view(1, H, D)
    c.pool[c.row(0, 3)] = u * 2
    c.pool[c.row(0, at)] = (u.float() * (2 + 7.9 * math.log(2) / (SCALE * float(u.double() @ u.double())))).to(torch.bfloat16)
    out, lse = prefix(m, q, c, n, [n]) if call == "prefix" else window(m, q, c, [1], [n], n, 0)
    check(out[0], lse[0], attend(q[0].double(), c.rows(0, range(n))), call)
    assert m.csa_read_device_status() == 0


@pytest.mark.parametrize("W,S", [(1 << 30, 0), (1 << 20, 3), (1, 1 << 30), (1 << 30, 1 << 30)])
def test_window_attention_over_everything(m, W, S):  # noqa: F811
    """Windows (or sinks) far wider than the cache, without a workspace given: as many bytes as the cache needs, and
    for a prompt the same bits as under a window of its own length."""
    g = gen(56)
    c = Cache(g, [300, 5000], 64)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    base = torch.cuda.memory_allocated()
    q = randn(g, 300, 128, D)
    out, lse = window(m, q, c, [299, 1], [300, 5000], W, S)
    want, lse2 = window(m, q, c, [299, 1], [300, 5000], 5000, 0)
    assert torch.cuda.max_memory_allocated() - base < 1 << 30
    assert torch.equal(out, want) and torch.equal(lse, lse2)
    check_window(q, c, [299, 1], [300, 5000], 5000, 0, out, lse, every=40)
    q1 = q[:1].contiguous()
    c.table = c.table[1:].contiguous()
    out, lse = window(m, q1, c, [1], [5000], W, S)
    check_window(q1, c, [1], [5000], 5000, 0, out, lse)
    assert m.csa_read_device_status() == 0
