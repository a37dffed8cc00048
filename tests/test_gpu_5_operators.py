"""Shared-prefix attention, windowed attention with sinks, and the page calls (csa_prefix_attn,
csa_window_attn, csa_pages_*) against plain restatements in 64 bits (attention) and in Python
integers (pages)."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

D = 512
SCALE = 1.0 / math.sqrt(D)
NO_PAGES, BOUNDS = 1 << 6, 1 << 4


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import deepseek_v4_hybrid_c4_gb300 as mod
    mod.csa_read_device_status()
    return mod


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def attend(q, kv):
    """q [H, 512], kv [n, 512] in 64 bits -> o, lse, and the bounds on both of a computation with bf16
    weights: a weight is off by at most half a bf16 step, 2^-8 of it, the result's own rounding by 2^-8
    of the result, and a logit by 2^-14 of scale * sum |q_i k_i| (which covers any order of fp32
    accumulation of 512 terms, 511 * 2^-24, twice over) -- the latter moves every weight by at most twice
    that relative amount, and lse by that amount itself; 2^-20 covers exp, log and the fp32 sums."""
    if kv.shape[0] == 0:
        z = torch.zeros_like(q)
        return z, torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device="cuda"), z, torch.zeros_like(q[:, 0])
    x = SCALE * (q @ kv.t())
    lse = torch.logsumexp(x, -1)
    w = torch.exp(x - lse[:, None])
    o, a = w @ kv, w @ kv.abs()
    d = 2.0**-14 * SCALE * (q.abs() @ kv.abs().t()).amax(-1)
    return o, lse, 2.0**-8 * (a + o.abs()) + (2 * d[:, None] + 2.0**-20) * a, d + 2.0**-20 * (1 + lse.abs())


class Cache:
    """A paged pool, a table with random page ids, and a [rows, 512] view of each request's rows."""

    def __init__(self, g, lengths, rpp, shared=0, spare=3, pitch=None, fill=None):
        B, width = len(lengths), max(1, -(-max(lengths) // rpp)) + 1
        self.rpp, self.width, self.B = rpp, width, B
        full = shared // rpp
        n_pages = full + B * (width - full) + spare
        self.n_pages, self.pitch = n_pages, pitch or rpp
        perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        self.table = torch.empty(B, width, dtype=torch.int32, device="cuda")
        self.table[:, :full] = perm[:full]
        self.table[:, full:] = perm[full: full + B * (width - full)].view(B, -1)
        self.pool = randn(g, n_pages * self.pitch, D)
        if fill is not None:
            self.pool.fill_(fill)
        if shared % rpp:
            for b in range(1, B):
                for j in range(full * rpp, shared):
                    self.pool[self.row(b, j)] = self.pool[self.row(0, j)]
        for b, n in enumerate(lengths):  # entries behind a request's pages: never read
            self.table[b, -(-n // rpp):] = 1 << 30

    def row(self, b, j):
        return int(self.table[b, j // self.rpp]) * self.pitch + j % self.rpp

    def at(self, b, js):
        js = torch.as_tensor(js, dtype=torch.int64, device="cuda")
        return self.table[b].long()[js // self.rpp] * self.pitch + js % self.rpp

    def rows(self, b, js):
        return self.pool[self.at(b, js)].double() if len(js) else torch.zeros(0, D, dtype=torch.float64, device="cuda")

    def paged(self, m):
        return m.paged(self.pool, self.rpp, 1024, self.table, page_stride_bytes=self.pitch * 1024, n_pages=self.n_pages)


def check(got, lse, want, where):
    o, l, to, tl = want
    off = (got.double() - o).abs() - to
    assert float(off.max()) <= 0, f"{where}: out of bound by {float(off.max()):.3e}"
    same = torch.isinf(l) & (lse.double() == l)
    off = torch.where(same, torch.zeros_like(l), (lse.double() - l).abs() - tl)
    assert float(off.max()) <= 0, f"{where}: lse out of bound by {float(off.max()):.3e}"


def prefix(m, q, c, shared, n_rows, max_rows=None, **kw):
    B, H = q.shape[:2]
    out = torch.full_like(q, 7.0)
    lse = torch.full((B, H), 7.0, dtype=torch.float32, device="cuda")
    n = torch.tensor(n_rows, dtype=torch.int64, device="cuda")
    m.csa_prefix_attn(q, B, H, SCALE, c.paged(m), c.width, shared, n, max_rows or max(max(n_rows), shared), out, lse, **kw)
    return out, lse


# ------------------------------------------------------------------ shared prefix
PREFIX = [  # H, shared, rows of each request, rows per page
    (1, 0, [1], 64),
    (1, 1, [1], 1),
    (16, 500, [500, 540], 64),
    (128, 64, [64, 65, 200], 64),
    (20, 130, [131, 200, 130, 177, 900], 17),
    (64, 1000, [0, 1, 999, 1300], 64),           # an empty request, requests shorter than the prefix
    (3, 127, [127, 128, 129, 255, 256, 257, 300], 16),
    (128, 4100, [4100 + 37 * i for i in range(8)], 64),
    (16, 9001, [9001 + (i * 53) % 400 for i in range(32)], 48),
    (7, 0, [5, 0, 129, 33], 128),                # nothing shared
    (128, 700, [700], 40),
    (100, 2049, [2100, 2049, 2301], 32),
]


@pytest.mark.parametrize("H,shared,n_rows,rpp", PREFIX)
def test_prefix_attention(m, H, shared, n_rows, rpp):
    g = gen(1)
    c = Cache(g, [max(n, shared) for n in n_rows], rpp, min(shared, max(n_rows)))
    q = randn(g, len(n_rows), H, D)
    out, lse = prefix(m, q, c, shared, n_rows)
    assert m.csa_read_device_status() == 0
    for b, n in enumerate(n_rows):
        check(out[b], lse[b], attend(q[b].double(), c.rows(b, range(n))), f"request {b}")
    again, lse2 = prefix(m, q, c, shared, n_rows)
    assert torch.equal(out, again) and torch.equal(lse, lse2)  # the same bits


RUNS = [  # H, shared, rows of each request, rows per page: many tiles, cut in runs of one length
    (16, 20000, [20000 + (i * 97) % 2000 for i in range(32)], 64),
    (128, 3000, [3000 + 13 * i for i in range(20)], 32),
    (128, 6000, [6000] * 12, 64),                       # nothing of their own
    (64, 0, [1200 + 31 * i for i in range(40)], 64),    # nothing shared
    (33, 5000, [0, 700, 5000, 5001] + [5000 + 300 * i for i in range(30)], 40),
]


@pytest.mark.parametrize("H,shared,n_rows,rpp", RUNS)
def test_prefix_attention_in_runs(m, H, shared, n_rows, rpp):
    test_prefix_attention(m, H, shared, n_rows, rpp)


def test_attention_over_nothing(m):
    """No rows at all: outputs of zero and lse -inf; no new tokens: nothing is written."""
    g = gen(7)
    c = Cache(g, [10, 10], 16)
    q = randn(g, 2, 5, D)
    out, lse = prefix(m, q, c, 0, [0, 0])
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    out, lse = prefix(m, q, c, 9, [0, 0])
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    out, lse = window(m, q[:0], c, [0, 0], [10, 0], 16, 2)
    out, lse = window(m, q, c, [0, 0], [10, 0], 16, 2)
    assert bool((out == 7).all()) and bool((lse == 7).all())
    assert m.csa_read_device_status() == 0


def test_prefix_attention_with_page_gaps_and_without_lse(m):
    """Pages 1.25 rows' pitch apart; no lse wanted; large logits (weights close to one-hot)."""
    g = gen(2)
    n_rows = [300, 257, 410]
    c = Cache(g, n_rows, 16, 256, pitch=20)
    q = (randn(g, 3, 24, D).float() * 12).to(torch.bfloat16)
    out = torch.empty_like(q)
    n = torch.tensor(n_rows, dtype=torch.int64, device="cuda")
    m.csa_prefix_attn(q, 3, 24, SCALE, c.paged(m), c.width, 256, n, 410, out)
    for b in range(3):
        w = attend(q[b].double(), c.rows(b, range(n_rows[b])))
        check(out[b], w[1].float(), w, f"request {b}")


@pytest.mark.parametrize("scale", [-0.07, 0.0, 1.5])
def test_attention_with_other_scales(m, scale):
    """A negative scale, a scale of zero (every row the same weight), logits of hundreds; outputs and
    workspace at addresses that are 16-byte aligned and no more."""
    g = gen(6)
    n_rows, H, W, S = [300, 190], 20, 70, 3
    c = Cache(g, n_rows, 32, 160)
    q = randn(g, 2, H, D)
    n = torch.tensor(n_rows, dtype=torch.int64, device="cuda")
    off = torch.tensor([0, 1, 2], dtype=torch.int64, device="cuda")
    need = max(m.csa_prefix_attn_workspace_size(2, H, 160, 300), m.csa_window_attn_workspace_size(2, H, 2, 1, W, S))
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")[16:]
    for call in range(2):
        out = torch.empty(2 * H * D + 8, dtype=torch.bfloat16, device="cuda")[8:].view(2, H, D)
        assert out.data_ptr() % 32 == 16 and ws.data_ptr() % 32 == 16
        lse = torch.empty(2, H, dtype=torch.float32, device="cuda")
        if call == 0:
            m.csa_prefix_attn(q, 2, H, scale, c.paged(m), c.width, 160, n, 300, out, lse, ws, need)
        else:
            m.csa_window_attn(q, H, scale, c.paged(m), c.width, 2, off, n, 2, 1, W, S, out, lse, ws, need)
        for b in range(2):
            keys = range(n_rows[b]) if call == 0 else list(range(S)) + list(range(n_rows[b] - W, n_rows[b]))
            kv = c.rows(b, keys)
            x = scale * (q[b].double() @ kv.t())
            want_lse = torch.logsumexp(x, -1)
            w = torch.exp(x - want_lse[:, None])
            o, av = w @ kv, w @ kv.abs()
            d = 2.0**-14 * abs(scale) * (q[b].double().abs() @ kv.abs().t()).amax(-1)
            check(out[b], lse[b], (o, want_lse, 2.0**-8 * (av + o.abs()) + (2 * d[:, None] + 2.0**-20) * av,
                                   d + 2.0**-20 * (1 + want_lse.abs())), f"call {call} request {b}")


def test_prefix_attention_rising_logits(m):
    """Each tile's largest logit far above the ones before it: the running maximum moves at every tile."""
    g = gen(3)
    n = 1500
    c = Cache(g, [n, n], 64, n)
    q = randn(g, 2, 16, D)
    u = q[0, 0].double() / q[0, 0].double().norm()
    at = c.at(0, range(n))
    ramp = torch.linspace(-30, 30, n, device="cuda", dtype=torch.float64)
    c.pool[at] = (c.pool[at].double() * 0.1 + ramp[:, None] * u).to(torch.bfloat16)
    out, lse = prefix(m, q, c, n, [n, n])
    for b in range(2):  # every row is shared: read through row 0 of the table
        check(out[b], lse[b], attend(q[b].double(), c.rows(0, range(n))), f"request {b}")


def test_prefix_attention_nan_reaches_only_its_readers(m):
    """A NaN and an infinity in rows that only some requests attend, in the shared part (behind a shorter
    request's end), in a request's own part, and behind every request's end."""
    g = gen(4)
    n_rows = [200, 130, 64, 201, 0]
    c = Cache(g, [256] * 5, 64, 192)
    c.pool[c.row(0, 150), 5] = math.nan        # shared: requests 0 and 3 attend it
    c.pool[c.row(3, 200), 300] = math.inf      # request 3's own
    c.pool[c.row(1, 130):c.row(1, 130) + 1] = math.nan
    for b in range(5):
        for j in range(max(n_rows[b], 192), 256):
            c.pool[c.row(b, j)] = math.inf
    q = randn(g, 5, 40, D)
    out, lse = prefix(m, q, c, 192, n_rows)
    assert torch.isnan(out[0]).any() and torch.isnan(out[3]).any()
    for b in (1, 2, 4):
        check(out[b], lse[b], attend(q[b].double(), c.rows(b, range(n_rows[b]))), f"request {b}")


def test_prefix_attention_bad_pages(m):
    """Page ids outside the pool leave their rows out and are reported; rows above max_rows are not read."""
    g = gen(5)
    c = Cache(g, [320, 400], 64, 128)
    c.table[0, 1] = c.n_pages          # rows 64..127 of the shared part
    c.table[1, 1] = -5
    c.table[1, 3] = -1                 # rows 192..255 of request 1
    q = randn(g, 2, 30, D)
    out, lse = prefix(m, q, c, 128, [320, 5000], max_rows=400)
    assert m.csa_read_device_status() == BOUNDS
    keep = [j for j in range(400) if not 64 <= j < 128]
    c.table[:, 1] = 0
    check(out[0], lse[0], attend(q[0].double(), c.rows(0, [j for j in keep if j < 320])), "request 0")
    check(out[1], lse[1], attend(q[1].double(), c.rows(1, [j for j in keep if not 192 <= j < 256])), "request 1")


# ------------------------------------------------------------------ window and sinks
def window(m, q, c, q_len, n_tokens, W, S, max_q=None, total_q=None, **kw):
    H = q.shape[1]
    off = torch.tensor(np.concatenate([[0], np.cumsum(q_len)]), dtype=torch.int64, device="cuda")
    n = torch.tensor(n_tokens, dtype=torch.int64, device="cuda")
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device="cuda")
    m.csa_window_attn(q, H, SCALE, c.paged(m), c.width, len(q_len), off, n, total_q or q.shape[0],
                      max_q or max(max(q_len), 1), W, S, out, lse, **kw)
    return out, lse


def check_window(q, c, q_len, n_tokens, W, S, out, lse, every=1):
    t = 0
    for b, (ql, n) in enumerate(zip(q_len, n_tokens)):
        for i in range(ql):
            p = n - ql + i
            if i % every == 0 or i == ql - 1:
                keys = [j for j in range(min(S, p + 1)) if j <= p - W] + list(range(max(0, p - W + 1), p + 1))
                check(out[t], lse[t], attend(q[t].double(), c.rows(b, keys)), f"sequence {b} token {i} (position {p})")
            t += 1


WINDOW = [  # H, (new tokens, tokens) of each sequence, window, sinks, rows per page
    (1, [(1, 1)], 1, 0, 64),
    (128, [(1, 1000)], 128, 4, 64),
    (16, [(1, 5), (1, 128), (1, 129), (1, 133), (1, 700), (1, 64)], 128, 16, 64),
    (128, [(70, 70)], 128, 4, 64),
    (24, [(33, 400), (1, 1), (0, 50), (100, 100), (7, 2000)], 100, 5, 40),
    (5, [(300, 300), (41, 90)], 17, 1, 16),
    (64, [(150, 150)], 1, 3, 64),
    (100, [(9, 600)], 257, 40, 32),
    (48, [(20, 20), (20, 21), (20, 3000)], 2000, 64, 128),
    (3, [(200, 200)], 1000, 500, 1),             # the sinks reach into the window
    (128, [(3, 3), (2, 900)], 512, 0, 17),
]


@pytest.mark.parametrize("H,seqs,W,S,rpp", WINDOW)
def test_window_attention(m, H, seqs, W, S, rpp):
    g = gen(11)
    q_len, n_tokens = [s[0] for s in seqs], [s[1] for s in seqs]
    c = Cache(g, n_tokens, rpp)
    q = randn(g, sum(q_len), H, D)
    out, lse = window(m, q, c, q_len, n_tokens, W, S)
    assert m.csa_read_device_status() == 0
    check_window(q, c, q_len, n_tokens, W, S, out, lse, every=1 if sum(q_len) < 200 else 7)
    again, lse2 = window(m, q, c, q_len, n_tokens, W, S)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("rpp", [1, 3, 20, 24])
def test_attention_over_pages_in_memory_order(m, rpp):
    """Pages of any size one behind the other in memory, with one page elsewhere: rows of several pages are
    neighbours in memory too."""
    g = gen(18)
    n = 333
    c = Cache(g, [n], rpp)
    first = (n + rpp - 1) // rpp
    c.table[0, :first] = torch.arange(first, dtype=torch.int32, device="cuda")
    c.table[0, 100 // rpp] = first  # one page elsewhere
    q = randn(g, 7, 33, D)
    out, lse = window(m, q, c, [7], [n], 200, 5)
    check_window(q, c, [7], [n], 200, 5, out, lse)
    out, lse = prefix(m, q[:1].contiguous(), c, n, [n])
    check(out[0], lse[0], attend(q[0].double(), c.rows(0, range(n))), "prefix")
    assert m.csa_read_device_status() == 0


def test_window_attention_leaves_other_rows_alone(m):
    """Rows behind the last sequence and before the first, and sequences that leave their buffers."""
    g = gen(12)
    c = Cache(g, [50, 60, 70], 64)
    q = randn(g, 40, 16, D)
    out, lse = window(m, q, c, [5, 6, 7], [50, 60, 70], 32, 2)
    check_window(q, c, [5, 6, 7], [50, 60, 70], 32, 2, out, lse)
    assert (out[18:] == 7).all() and (lse[18:] == 7).all() and m.csa_read_device_status() == 0
    out, lse = window(m, q, c, [5, 6, 7], [50, 60, 70], 32, 2, max_q=6)  # the third has too many new tokens
    check_window(q, c, [5, 6], [50, 60], 32, 2, out, lse)
    assert (out[11:] == 7).all() and m.csa_read_device_status() == BOUNDS
    out, lse = window(m, q, c, [5, 6, 7], [50, 60, 70], 32, 2, total_q=12)  # the third ends behind the buffers
    check_window(q, c, [5, 6], [50, 60], 32, 2, out, lse)
    assert (out[11:] == 7).all() and m.csa_read_device_status() == BOUNDS


def test_window_attention_tokens_before_the_first_position(m):
    g = gen(13)
    c = Cache(g, [4, 60], 16)
    q = randn(g, 20, 33, D)
    out, lse = window(m, q, c, [10, 10], [4, 60], 32, 2)
    assert (out[:6] == 0).all() and torch.isinf(lse[:6]).all() and (lse[:6] < 0).all()
    check_window(q[6:], c, [4, 10], [4, 60], 32, 2, out[6:], lse[6:])


def test_window_attention_with_given_back_pages(m):
    """Pages behind the window (not those of the sinks) are -1 in the table and never read."""
    g = gen(14)
    for rpp in (16, 24):
        n_tokens, q_len, W, S = [1000, 777], [20, 1], 64, 6
        c = Cache(g, n_tokens, rpp)
        for b in range(2):
            first = (n_tokens[b] - q_len[b] + 1 - W) // rpp
            c.table[b, 1:first] = -1
        q = randn(g, 21, 16, D)
        out, lse = window(m, q, c, q_len, n_tokens, W, S)
        assert m.csa_read_device_status() == 0
        check_window(q, c, q_len, n_tokens, W, S, out, lse)


@pytest.mark.parametrize("rpp", [64, 24])
def test_window_attention_nan_reaches_only_its_readers(m, rpp):
    """A row of NaN, an infinity and rows behind the end of the sequence: tokens that do not see them
    are as if they were not there."""
    g = gen(15)
    c = Cache(g, [400], rpp)
    c.pool[c.row(0, 200), 17] = math.nan
    c.pool[c.row(0, 390), 400] = -math.inf
    last = c.row(0, 399)
    c.pool[last + 1: last + rpp - 399 % rpp] = math.nan
    q = randn(g, 300, 16, D)
    out, lse = window(m, q, c, [300], [400], 50, 3)
    t = 0
    for p in range(100, 400):
        keys = list(range(3)) + list(range(p - 49, p + 1))
        if 200 in keys:
            assert torch.isnan(out[t]).all(), p
        elif 390 not in keys and p % 5 == 0:
            check(out[t], lse[t], attend(q[t].double(), c.rows(0, keys)), f"position {p}")
        t += 1


@pytest.mark.parametrize("H,rpp", [(128, 64), (128, 40), (24, 64), (24, 40)])
def test_window_attention_nan_in_masked_rows_of_every_kind(m, H, rpp):
    """Windows whose tiles are a full one and a short one: NaN behind the last position, infinity between the sinks
    and the window and in the sinks' own unit, in every sequence; and a NaN that only the later tokens of one
    sequence have left behind."""
    g = gen(27)
    n_tokens, q_len, W, S = [1000, 641, 333, 150, 2000], [1, 2, 1, 6, 3], 128, 4
    c = Cache(g, [n + 16 for n in n_tokens], rpp)
    for b, n in enumerate(n_tokens):
        c.pool[c.at(b, range(n, n + 16))] = math.nan
        c.pool[c.at(b, range(S, n - q_len[b] - W))] = math.inf
    p = n_tokens[3] - q_len[3] - W + 2             # the first two tokens of sequence 3 still see it
    clean = c.pool[c.row(3, p)].clone()
    c.pool[c.row(3, p)] = math.nan
    q = randn(g, sum(q_len), H, D)
    out, lse = window(m, q, c, q_len, n_tokens, W, S)
    t = 0
    for b, (ql, n) in enumerate(zip(q_len, n_tokens)):
        for i in range(ql):
            pos = n - ql + i
            keys = list(range(S)) + list(range(max(S, pos - W + 1), pos + 1))
            if b == 3 and p in keys:
                assert bool(torch.isnan(out[t]).all()) and bool(torch.isnan(lse[t]).all())
            else:
                check(out[t], lse[t], attend(q[t].double(), c.rows(b, keys)), f"sequence {b} token {i}")
            t += 1
    c.pool[c.row(3, p)] = clean
    assert m.csa_read_device_status() == 0


def test_window_attention_bad_pages(m):
    g = gen(16)
    c = Cache(g, [300, 300], 32)
    c.table[0, 8] = c.n_pages + 3      # positions 256..287
    q = randn(g, 12, 20, D)
    out, lse = window(m, q, c, [6, 6], [300, 300], 60, 4)
    assert m.csa_read_device_status() == BOUNDS
    for i in range(12):
        b, p = i // 6, 294 + i % 6
        keys = list(range(4)) + [j for j in range(p - 59, p + 1) if b or not 256 <= j < 288]
        check(out[i], lse[i], attend(q[i].double(), c.rows(b, keys)), f"sequence {b} position {p}")
    c.width = 9                        # tokens behind the table's pages
    t = c.table[:, :9].contiguous()
    c.table = t
    c.table[0, 8] = 0
    window(m, q, c, [6, 6], [300, 300], 60, 4)
    assert m.csa_read_device_status() == BOUNDS


def test_window_attention_matches_the_decode_step(m):
    """Without sinks a single token is the decode step's sliding window (csa_sparse_attn, no selection)."""
    g = gen(17)
    for H in (16, 128):
        c = Cache(g, [900], 64)
        q = randn(g, 1, H, D)
        out, lse = window(m, q, c, [1], [900], 128, 0)
        o2, l2 = torch.empty_like(q), torch.empty(H, dtype=torch.float32, device="cuda")
        ws = torch.empty(m.csa_sparse_attn_workspace_size(H, 0, 128) + 16, dtype=torch.uint8, device="cuda")
        m.csa_sparse_attn(q, H, SCALE, c.paged(m), None, 0, c.paged(m), 900, 128, o2, l2, ws, ws.numel())
        want = attend(q[0].double(), c.rows(0, range(772, 900)))
        check(out[0], lse[0], want, "window")
        # both are within the bound of the same value (csa_sparse_attn's sum is over the rounded weights)
        assert ((out[0] - o2[0]).abs().double() <= 2 * want[2] + 2.0**-8 * want[2]).all()


# ------------------------------------------------------------------ streams, graphs, workspaces
def test_attention_on_a_side_stream_and_in_graphs(m):
    """Both calls on a stream of their own, and captured: two graphs that share one workspace, replayed in
    turn with inputs changed in place, and an eager call between them."""
    g = gen(21)
    n_rows = [3000 + 11 * b for b in range(4)]
    c = Cache(g, n_rows, 64, 2900)
    q, q2 = randn(g, 4, 16, D), randn(g, 4, 16, D)
    n = torch.tensor(n_rows, dtype=torch.int64, device="cuda")
    need = max(m.csa_prefix_attn_workspace_size(4, 16, 2900, 3100), m.csa_window_attn_workspace_size(4, 16, 4, 1, 900, 4), 16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    off = torch.arange(5, dtype=torch.int64, device="cuda")
    o1, o2 = torch.zeros_like(q), torch.zeros_like(q)
    kv = c.paged(m)

    def one():
        m.csa_prefix_attn(q, 4, 16, SCALE, kv, c.width, 2900, n, 3100, o1, None, ws, need)

    def two():
        m.csa_window_attn(q, 16, SCALE, kv, c.width, 4, off, n, 4, 1, 900, 4, o2, None, ws, need)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        one()
        two()
    torch.cuda.current_stream().wait_stream(s)
    e1, e2 = o1.clone(), o2.clone()
    for b in range(4):
        w = attend(q[b].double(), c.rows(b, range(n_rows[b])))
        check(e1[b], w[1].float(), w, "prefix")
        w = attend(q[b].double(), c.rows(b, list(range(4)) + list(range(n_rows[b] - 900, n_rows[b]))))
        check(e2[b], w[1].float(), w, "window")
    graphs = []
    for f in (one, two):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            f()
        graphs.append(gr)
    o1.zero_(), o2.zero_()
    for _ in range(2):
        graphs[0].replay()
        graphs[1].replay()
    assert torch.equal(o1, e1) and torch.equal(o2, e2)
    q.copy_(q2)
    graphs[1].replay()
    graphs[0].replay()
    r1, r2 = o1.clone(), o2.clone()
    one()
    two()
    assert torch.equal(o1, r1) and torch.equal(o2, r2)
    torch.cuda.synchronize()
    assert m.csa_read_device_status() == 0


def test_attention_calls_on_two_streams_at_once(m):
    """Both calls, each on its own stream with its own workspace, in flight together: the same bits as alone."""
    g = gen(22)
    n_rows = [5000 + 70 * b for b in range(8)]
    c = Cache(g, n_rows, 64, 4500)
    q, qw = randn(g, 8, 128, D), randn(g, 600, 24, D)
    kv, n = c.paged(m), torch.tensor(n_rows, dtype=torch.int64, device="cuda")
    off = torch.tensor([0, 100, 101, 101, 400, 401, 402, 500, 600], dtype=torch.int64, device="cuda")
    sizes = (m.csa_prefix_attn_workspace_size(8, 128, 4500, 5500), m.csa_window_attn_workspace_size(8, 24, 600, 300, 2000, 9))
    ws = [torch.empty(max(x, 16), dtype=torch.uint8, device="cuda") for x in sizes]
    outs = [torch.zeros_like(q), torch.zeros_like(qw)]

    def one():
        m.csa_prefix_attn(q, 8, 128, SCALE, kv, c.width, 4500, n, 5500, outs[0], None, ws[0], ws[0].numel())

    def two():
        m.csa_window_attn(qw, 24, SCALE, kv, c.width, 8, off, n, 600, 300, 2000, 9, outs[1], None, ws[1], ws[1].numel())

    one()
    two()
    torch.cuda.synchronize()
    alone = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for f, s in zip((one, two), streams):
            with torch.cuda.stream(s):
                f()
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) for o, a in zip(outs, alone)) and m.csa_read_device_status() == 0


@pytest.mark.parametrize("rpp", [64, 24])
def test_attention_beyond_4_gb(m, rpp):
    """A pool of 6 GB whose used pages are its last ones: row offsets that pass 32 bits."""
    g = gen(23)
    n = 700
    pages = -(-n // rpp)
    n_pages = (6 << 30) // (rpp * 1024)
    c = Cache.__new__(Cache)
    c.rpp, c.pitch, c.width, c.B, c.n_pages = rpp, rpp, pages, 1, n_pages
    c.pool = torch.zeros(n_pages * rpp, D, dtype=torch.bfloat16, device="cuda")
    c.table = (n_pages - 1 - torch.arange(pages, dtype=torch.int32, device="cuda")).view(1, -1)
    c.pool[c.at(0, range(n))] = randn(g, n, D)
    q = randn(g, 5, 24, D)
    out, lse = window(m, q, c, [5], [n], 600, 3)
    check_window(q, c, [5], [n], 600, 3, out, lse)
    out, lse = prefix(m, q[:1].contiguous(), c, 650, [n])
    check(out[0], lse[0], attend(q[0].double(), c.rows(0, range(n))), "prefix")
    assert m.csa_read_device_status() == 0


@pytest.mark.parametrize("call", ["prefix", "window"])
def test_attention_over_the_longest_context(m, call):
    """2^31 - 128 rows over three pages of 4,096 rows, named again and again; all rows, and a window of 2^30.  Beside
    the bounds of attend(): a split of 4,096 tiles adds eight times a tile to its output, each losing up to
    2^-23 of the sum (2^-8 in all), and once a tile to its row sums, and up to 4,096 splits are merged in fp32 (2^-24 an
    addition: 2^-11 for both)."""
    g = gen(26)
    n, rpp, H = (1 << 31) - 128, 4096, 16
    pages = -(-n // rpp)
    c = Cache.__new__(Cache)
    c.rpp, c.pitch, c.width, c.B, c.n_pages = rpp, rpp, pages, 1, 3
    c.pool = (randn(g, 3 * rpp, D).float() + 0.5).to(torch.bfloat16)
    c.table = (torch.arange(pages, dtype=torch.int32, device="cuda") % 3).view(1, -1).contiguous()
    q = randn(g, 1, H, D)
    if call == "prefix":
        first = 0
        out, lse = prefix(m, q, c, 64, [n])
    else:
        first = n - (1 << 30)
        out, lse = window(m, q, c, [1], [n], 1 << 30, 0)
    assert m.csa_read_device_status() == 0
    count = torch.zeros(3 * rpp, dtype=torch.float64, device="cuda")  # how often a row is attended
    whole, last = first // rpp + 1, pages - 1                         # pages attended as a whole: [whole, last)
    for p in range(3):
        count[p * rpp:(p + 1) * rpp] = (last - p + 2) // 3 - (whole - p + 2) // 3
    count[whole % 3 * rpp - rpp + first % rpp if whole % 3 else 2 * rpp + first % rpp:
          whole % 3 * rpp if whole % 3 else 3 * rpp] += 1             # page whole - 1 from `first` on
    count[last % 3 * rpp:last % 3 * rpp + (n - last * rpp)] += 1
    assert int(count.sum()) == n - first
    kv, qd = c.pool.double(), q[0].double()
    x = SCALE * (qd @ kv.t()) + torch.log(count)
    want = torch.logsumexp(x, -1)
    w = torch.exp(x - want[:, None])
    o, a = w @ kv, w @ kv.abs()
    d = 2.0**-14 * SCALE * (qd.abs() @ kv.abs().t()).amax(-1)
    check(out[0], lse[0], (o, want, 2.0**-8 * (2 * a + o.abs()) + (2 * d[:, None] + 2.0**-11) * a,
                           d + 2.0**-20 * (1 + want.abs()) + 2.0**-11), call)


def test_window_attention_offsets_that_fall_and_rise(m):
    """Offsets that are not non-decreasing are reported, and the call ends: sequences that overlap because of
    them are not all computed."""
    g = gen(24)
    B = 300
    c = Cache(g, [40] * B, 64)
    q = randn(g, 64, 128, D)
    off = torch.tensor([0, 32] * (B // 2) + [0], dtype=torch.int64, device="cuda")
    n = torch.full((B,), 40, dtype=torch.int64, device="cuda")
    out = torch.full_like(q, 7.0)
    m.csa_window_attn(q, 128, SCALE, c.paged(m), c.width, B, off, n, 64, 32, 8, 0, out)
    torch.cuda.synchronize()
    assert (out[32:] == 7).all() and m.csa_read_device_status() == BOUNDS


def test_window_attention_lengths_out_of_range(m):
    """A token count behind the largest is reported and its sequence skipped; the others are as if alone."""
    g = gen(25)
    c = Cache(g, [50, 60, 70], 64)
    q = randn(g, 9, 16, D)
    for n in ((1 << 31) - 1, 1 << 31, (1 << 63) - 1):
        out, lse = window(m, q, c, [3, 3, 3], [50, n, 70], 32, 2)
        assert m.csa_read_device_status() == BOUNDS
        assert (out[3:6] == 7).all() and (lse[3:6] == 7).all()
        check_window(q[:3], c, [3], [50], 32, 2, out[:3], lse[:3])
        for i in range(3):
            p = 67 + i
            check(out[6 + i], lse[6 + i], attend(q[6 + i].double(), c.rows(2, [0, 1] + list(range(p - 31, p + 1)))), f"{p}")


# ------------------------------------------------------------------ pages
class Model:
    """The page calls on Python integers."""

    def __init__(self, refs, table):
        self.refs, self.table = list(refs), [list(r) for r in table]

    def take(self):
        for p, r in enumerate(self.refs):
            if r == 0:
                self.refs[p] = 1
                return p
        return -1

    def alloc(self, first, count):
        for b in range(len(self.table)):
            for j in range(first[b], first[b] + count[b]):
                self.table[b][j] = self.take()

    def free(self, rows):
        for b in rows:
            for j, p in enumerate(self.table[b]):
                if p >= 0:
                    self.refs[p] -= 1
                self.table[b][j] = -1

    def fork(self, src, dst, n_tokens, rpp):
        copies = []
        for a, d in zip(src, dst):
            full, w = n_tokens[a] // rpp, len(self.table[0])
            row = self.table[a][:full] + [-1] * (w - full)
            for p in row[:full]:
                if p >= 0:
                    self.refs[p] += 1
            n_tokens[d] = n_tokens[a]
            if n_tokens[a] % rpp and self.table[a][full] >= 0:
                row[full] = self.take()
                if row[full] >= 0:
                    copies.append((self.table[a][full], row[full]))
                else:
                    n_tokens[d] = full * rpp
            self.table[d] = row
        return copies

    def compact(self):
        U = sum(r > 0 for r in self.refs)
        holes = [p for p in range(U) if self.refs[p] == 0]
        to = {p: holes.pop(0) for p in range(U, len(self.refs)) if self.refs[p] > 0}
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        self.table = [[to.get(p, p) for p in r] for r in self.table]
        return U, to


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def fragmented(n_pages, B, width, used, seed):
    """A table whose requests name `used` random pages, some of them twice, and its counts."""
    rng = np.random.default_rng(seed)
    table = np.full((B, width), -1, np.int64)
    at = rng.permutation(B * width)[:min(used, B * width)]
    ids = rng.permutation(n_pages)[:len(at)]
    table.reshape(-1)[at] = ids
    twice = rng.permutation(B * width)[:B]
    table.reshape(-1)[twice] = ids[0] if len(ids) else -1
    refs = np.zeros(n_pages, np.int64)
    np.add.at(refs, table[table >= 0], 1)
    return refs.tolist(), table.tolist()


@pytest.mark.parametrize("n_pages,B,width,used", [(1, 1, 1, 0), (100, 3, 7, 15), (4096, 5, 300, 1000), (4097, 2, 9, 12),
                                                  (9000, 4, 2000, 7000), (70000, 3, 20000, 50000)])
def test_pages_alloc_and_free(m, n_pages, B, width, used):
    refs, table = fragmented(n_pages, B, width, used, 1)
    mod = Model(refs, table)
    r, t = i32(refs), i32(table)
    rows = [B - 1, 0, B - 1]                       # one of them twice
    m.csa_pages_free(r, n_pages, t, width, B, i32(rows), 3)
    mod.free(sorted(set(rows)))
    assert r.tolist() == mod.refs and t.tolist() == mod.table
    first, count = [0] * B, [0] * B
    count[0] = min(width, 5)
    first[B - 1], count[B - 1] = width // 2, width - width // 2
    if B == 1:
        first, count = [0], [1]
    m.csa_pages_alloc(r, n_pages, t, width, B, i32(first), i32(count))
    mod.alloc(first, count)
    assert r.tolist() == mod.refs and t.tolist() == mod.table
    assert m.csa_read_device_status() == 0


def test_pages_alloc_runs_out(m):
    refs = [1, 0, 2, 0, 1, 0]
    r, t = i32(refs), i32([[-1] * 4, [-1] * 4, [-1] * 4])
    m.csa_pages_alloc(r, 6, t, 4, 3, i32([0, 3, 0]), i32([2, 2, 3]))  # request 1's range leaves the table
    assert t.tolist() == [[1, 3, -1, -1], [-1] * 4, [5, -1, -1, -1]] and r.tolist() == [1, 1, 2, 1, 1, 1]
    assert m.csa_read_device_status() == NO_PAGES | BOUNDS


def test_pages_free_reports_what_is_wrong(m):
    r, t = i32([1, 0, 3]), i32([[0, 1, 7], [2, -1, -1]])
    m.csa_pages_free(r, 3, t, 3, 2, i32([0, 5, -1]), 3)
    assert r.tolist() == [0, 0, 3] and t.tolist() == [[-1, -1, -1], [2, -1, -1]]
    assert m.csa_read_device_status() == BOUNDS


def pools_of(n_pages, seed=3):
    g = gen(seed)
    shapes = ((48,), (2, 24), (8,))               # 16-bit values of a page
    return [torch.randint(-30000, 30000, (n_pages, *s), generator=g, device="cuda", dtype=torch.int16) for s in shapes]


@pytest.mark.parametrize("n_pages,tokens,src,rpp", [
    (64, [70, 64, 1, 0], [0, 1, 2, 3, 0, 0], 16),
    (9000, [4000, 3999], [1, 0, 1, 1], 1),
    (5000, [5 * 64 + 3, 64 * 40, 64 * 1500 + 63], [2, 2, 0, 1, 2], 64),
])
def test_pages_fork(m, n_pages, tokens, src, rpp):
    P, F = len(tokens), len(src)
    B, width = P + F + 1, max(tokens) // rpp + 2
    mod = Model([0] * n_pages, [[-1] * width for _ in range(B)])
    mod.refs[::3] = [1] * len(mod.refs[::3])      # pages that others hold
    mod.alloc([0] * B, [-(-t // rpp) for t in tokens] + [0] * (B - P))
    if width > 20:
        p, mod.table[0][3] = mod.table[0][3], -1  # a page given back
        mod.refs[p] = 0
    n = tokens + [-9] * (B - P)
    pools = pools_of(n_pages)
    before = [p.clone() for p in pools]
    r, t, nt = i32(mod.refs), i32(mod.table), torch.tensor(n, dtype=torch.int64, device="cuda")
    dst = list(range(P + 1, P + 1 + F))
    m.csa_pages_fork(m.page_pools(pools, n_pages), r, t, width, B, i32(src), i32(dst), F, nt, rpp)
    copies = mod.fork(src, dst, n, rpp)
    assert r.tolist() == mod.refs and t.tolist() == mod.table and nt.tolist() == n
    for p, old in zip(pools, before):
        for a, d in copies:
            old[d] = old[a]
        assert torch.equal(p, old)
    assert m.csa_read_device_status() == 0


@pytest.mark.parametrize("n_pages,F", [(64, 1), (64, 8), (500, 9), (500, 16), (500, 17), (3000, 100), (32768, 3),
                                       (32769, 3), (40000, 16)])
def test_pages_fork_of_any_number(m, n_pages, F):
    """Pools that every scan CTA counts by itself (up to 32,768 pages) and larger ones, one child and many."""
    test_pages_fork(m, n_pages, [40, 33], [i % 2 for i in range(F)], 16)


@pytest.mark.parametrize("n_pages,free", [(32768, 3), (32768, 2), (20000, 16), (8193, 1), (70000, 5), (31, 0)])
def test_pages_fork_in_a_pool_almost_full(m, n_pages, free):
    """The free pages are the last ones of the pool, and there are as many as children, fewer, or more."""
    F = 4
    refs = [1] * (n_pages - free) + [0] * free
    mod = Model(refs, [[0, 1, -1]] + [[-1] * 3 for _ in range(F)])
    n = [6] + [0] * F
    r, t, nt = i32(mod.refs), i32(mod.table), torch.tensor(n, dtype=torch.int64, device="cuda")
    pools = pools_of(n_pages)
    m.csa_pages_fork(m.page_pools(pools, n_pages), r, t, 3, F + 1, i32([0] * F), i32([1, 2, 3, 4]), F, nt, 4)
    for f in range(F):
        mod.refs[0] += 1
        if f < free:
            mod.refs[n_pages - free + f] = 1
        mod.table[1 + f] = [0, n_pages - free + f if f < free else -1, -1]
        n[1 + f] = 6 if f < free else 4
    assert r.tolist() == mod.refs and t.tolist() == mod.table and nt.tolist() == n
    for p in pools:
        for f in range(min(free, F)):
            assert torch.equal(p[n_pages - free + f], p[1])
    assert m.csa_read_device_status() == (0 if free >= F else NO_PAGES)


def test_pages_fork_refusals_on_the_device(m):
    """Rows outside the table, a child that is a parent, a row twice, tokens that do not fit, a page id
    outside the pool, no free page: reported, and the other children are as if alone."""
    pools = pools_of(12)
    d = m.page_pools(pools, 12)

    def go(refs, table, src, dst, n):
        r, t, nt = i32(refs), i32(table), torch.tensor(n, dtype=torch.int64, device="cuda")
        m.csa_pages_fork(d, r, t, 3, len(table), i32(src), i32(dst), len(src), nt, 4)
        return r.tolist(), t.tolist(), nt.tolist(), m.csa_read_device_status()

    refs, e = [1, 1] + [0] * 10, [-1] * 3
    base = [[0, 1, -1], e, e, e]
    n = [6, -7, -7, -7]
    assert go(refs, base, [0, 9], [1, 2], n) == ([2, 1, 1] + [0] * 9, [[0, 1, -1], [0, 2, -1], e, e], [6, 6, -7, -7], BOUNDS)
    assert go(refs, base, [0, 0], [2, -1], n)[3] == BOUNDS
    assert go(refs, base, [0, 0], [0, 3], n) == ([2, 1, 0, 1] + [0] * 8, [[0, 1, -1], e, e, [0, 3, -1]], [6, -7, -7, 6], BOUNDS)
    assert go(refs, base, [0, 0], [3, 3], n) == (refs, base, n, BOUNDS)
    assert go(refs, base, [0], [1], [13, -7, -7, -7]) == (refs, base, [13, -7, -7, -7], BOUNDS)
    assert go(refs, [[0, 50, 1], e, e, e], [0], [1], [9, 0, 0, 0]) == (
        [2, 1, 1] + [0] * 9, [[0, 50, 1], [0, -1, 2], e, e], [9, 9, 0, 0], BOUNDS)
    full = [1] * 12
    assert go(full, base, [0], [1], n) == ([2] + [1] * 11, [[0, 1, -1], [0, -1, -1], e, e], [6, 4, -7, -7], NO_PAGES)


def test_pages_fork_token_counts_out_of_range(m):
    """Token counts that no table row holds, up to the largest integer: skipped and reported."""
    pools = pools_of(8)
    d = m.page_pools(pools, 8)
    for n in (12, 13, (1 << 40) + 1, (1 << 63) - 1, (1 << 63) - 4, -1, -(1 << 63)):
        r, t, nt = i32([1, 1, 1, 0, 0, 0, 0, 0]), i32([[0, 1, 2], [-1] * 3]), torch.tensor([n, 5], device="cuda")
        m.csa_pages_fork(d, r, t, 3, 2, i32([0]), i32([1]), 1, nt, 4)
        if n == 12:
            assert t.tolist() == [[0, 1, 2]] * 2 and nt.tolist() == [12, 12] and m.csa_read_device_status() == 0
        else:
            assert t.tolist() == [[0, 1, 2], [-1] * 3] and nt.tolist() == [n, 5]
            assert r.tolist() == [1, 1, 1, 0, 0, 0, 0, 0] and m.csa_read_device_status() == BOUNDS


def test_pages_beyond_4_gb(m):
    """A pool of 6 GB: a fork copies into its last page, a compaction moves pages from its end to its front."""
    n_pages, words = 400000, 2048
    pool = torch.zeros(n_pages, words, dtype=torch.int64, device="cuda")
    d = m.page_pools([pool], n_pages)
    refs = torch.ones(n_pages, dtype=torch.int32, device="cuda")
    refs[-1] = 0
    table = i32([[5, n_pages - 2, -1], [-1] * 3])
    pool[n_pages - 2] = 77
    nt = torch.tensor([7, 0], dtype=torch.int64, device="cuda")
    m.csa_pages_fork(d, refs, table, 3, 2, i32([0]), i32([1]), 1, nt, 4)
    assert table.tolist() == [[5, n_pages - 2, -1], [5, n_pages - 1, -1]] and nt.tolist() == [7, 7]
    assert bool((pool[n_pages - 1] == 77).all()) and int(refs[5]) == 2 and int(refs.sum()) == n_pages + 1
    pool[n_pages - 1] = 78
    refs.zero_()
    refs[5], refs[n_pages - 2:] = 2, 1
    used = torch.zeros(1, dtype=torch.int64, device="cuda")
    pool[5] = 76
    m.csa_pages_compact(d, refs, refs, table, table, 3, 2, used)
    assert used.item() == 3 and table.tolist() == [[0, 1, -1], [0, 2, -1]] and refs[:3].tolist() == [2, 1, 1]
    assert bool((pool[:3] == torch.tensor([[76], [77], [78]], device="cuda")).all())
    assert int(refs.sum()) == 4 and m.csa_read_device_status() == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_pages,B,width,used", [(1, 1, 1, 1), (10, 1, 3, 0), (100, 3, 17, 40), (4096, 5, 300, 1000),
                                                  (4097, 2, 2100, 4097), (9000, 4, 2000, 6000), (70000, 3, 20000, 50000)])
def test_pages_compact(m, n_pages, B, width, used, in_place):
    refs, table = fragmented(n_pages, B, width, used, 2)
    mod = Model(refs, table)
    pools = pools_of(n_pages)
    before = [p.clone() for p in pools]
    r, t, n = i32(refs), i32(table), torch.zeros(1, dtype=torch.int64, device="cuda")
    ro, to = (r, t) if in_place else (torch.empty_like(r), torch.empty_like(t))
    m.csa_pages_compact(m.page_pools(pools, n_pages), r, ro, t, to, width, B, n)
    U, moved = mod.compact()
    assert n.item() == U and ro.tolist() == mod.refs and to.tolist() == mod.table
    if not in_place:
        assert r.tolist() == refs and t.tolist() == table
    s, d = list(moved), list(moved.values())
    for p, old in zip(pools, before):
        old[d] = old[s]
        assert torch.equal(p, old)
    assert m.csa_read_device_status() == 0


def test_pages_compact_reports_dangling_entries(m):
    r, t = i32([0, 1, 0, 1]), i32([[3, 1, 2], [-1, 9, -4]])
    pools = pools_of(4)
    m.csa_pages_compact(m.page_pools(pools, 4), r, r, t, t, 3, 2, None)
    assert t.tolist() == [[0, 1, 2], [-1, 9, -4]] and r.tolist() == [1, 1, 0, 0]
    assert m.csa_read_device_status() == BOUNDS


def test_pages_copy(m):
    pools = pools_of(40)
    before = [p.clone() for p in pools]
    src, dst = [3, 3, 39, 0, 50, 2, -1], [7, 8, 1, 20, 30, 40, 9]
    m.csa_pages_copy(m.page_pools(pools, 40), i32(src), i32(dst), 7)
    for p, old in zip(pools, before):
        for a, d in zip(src[:4], dst[:4]):
            old[d] = old[a]
        assert torch.equal(p, old)
    assert m.csa_read_device_status() == BOUNDS


def test_pages_of_a_pool_with_gaps(m):
    """Pools that are slices of wider pages: only the slice is copied."""
    wide = torch.randint(-9, 9, (30, 64), generator=gen(4), device="cuda", dtype=torch.int16)
    before = wide.clone()
    m.csa_pages_copy(m.page_pools([wide[:, 16:40]], 30), i32([1, 2]), i32([10, 11]), 2)
    before[[10, 11], 16:40] = before[[1, 2], 16:40]
    assert torch.equal(wide, before)


def test_pages_calls_in_a_graph(m):
    """free + fork captured once and replayed: each replay takes the children back and forks them again."""
    n_pages, width, B = 600, 40, 6
    mod = Model([0] * n_pages, [[-1] * width for _ in range(B)])
    mod.alloc([0] * B, [30, 0, 0, 0, 0, 0])
    n = [29 * 16 + 5] + [0] * 5
    r, t, nt = i32(mod.refs), i32(mod.table), torch.tensor(n, dtype=torch.int64, device="cuda")
    pools = pools_of(n_pages)
    d, src, dst = m.page_pools(pools, n_pages), i32([0] * 4), i32([1, 2, 3, 5])
    ws = torch.empty(m.csa_pages_workspace_size(n_pages), dtype=torch.uint8, device="cuda")

    def step():
        m.csa_pages_free(r, n_pages, t, width, B, dst, 4)
        m.csa_pages_fork(d, r, t, width, B, src, dst, 4, nt, 16, ws, ws.numel())

    step()
    torch.cuda.synchronize()
    mod.fork([0] * 4, [1, 2, 3, 5], n, 16)
    assert r.tolist() == mod.refs and t.tolist() == mod.table
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step()
    for _ in range(3):
        gr.replay()
    assert r.tolist() == mod.refs and t.tolist() == mod.table and nt.tolist() == n
    assert m.csa_read_device_status() == 0


# ------------------------------------------------------------------ the operators together
@pytest.mark.parametrize("H", [16, 128])
def test_a_prompt_sampled_forked_and_compacted(m, H):
    """A prompt is attended in chunks (window and sinks), forked into four samples, each sample grows by its
    own tokens, the batch attends the shared prompt once, two samples end, the pages are
    compacted: every output is right, and the compaction changes no bit of the survivors'."""
    g = gen(31)
    rpp, n0, B, width, n_pages = 64, 1000, 5, 24, 90
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[::4] = 1                                  # pages of others
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    pool = torch.zeros(n_pages * rpp, D, dtype=torch.bfloat16, device="cuda")
    kidx = torch.randint(-9, 9, (n_pages, 2048), generator=g, device="cuda", dtype=torch.int16)
    desc = m.page_pools([pool.view(n_pages, rpp * D), kidx], n_pages)
    n_tokens = torch.tensor([n0, 0, 0, 0, 0], dtype=torch.int64, device="cuda")
    m.csa_pages_alloc(refs, n_pages, table, width, B, i32([0] * B), i32([-(-n0 // rpp), 0, 0, 0, 0]))
    c = Cache.__new__(Cache)
    c.rpp, c.pitch, c.width, c.B, c.n_pages, c.table, c.pool = rpp, rpp, width, B, n_pages, table, pool
    pool[c.at(0, range(n0))] = randn(g, n0, D)
    q = randn(g, 30, H, D)
    out, lse = window(m, q, c, [30], [n0], 128, 4)
    check_window(q, c, [30], [n0], 128, 4, out, lse, every=9)
    m.csa_pages_fork(desc, refs, table, width, B, i32([0] * 4), i32([1, 2, 3, 4]), 4, n_tokens, rpp)
    assert n_tokens.tolist() == [n0] * 5 and int((refs > 1).sum()) == n0 // rpp
    grow = [3, 100, 24, 25, 200]
    have = torch.full((B,), -(-n0 // rpp), dtype=torch.int32, device="cuda")
    want = i32([-(-(n0 + x) // rpp) for x in grow])
    m.csa_pages_alloc(refs, n_pages, table, width, B, have, want - have)
    for b, x in enumerate(grow):
        pool[c.at(b, range(n0, n0 + x))] = randn(g, x, D)
    rows = [n0 + x for x in grow]
    q = randn(g, B, H, D)
    out, lse = prefix(m, q, c, n0, rows)
    for b in range(B):
        check(out[b], lse[b], attend(q[b].double(), c.rows(b, range(rows[b]))), f"sample {b}")
    m.csa_pages_free(refs, n_pages, table, width, B, i32([1, 3]), 2)
    used = torch.zeros(1, dtype=torch.int64, device="cuda")
    m.csa_pages_compact(desc, refs, refs, table, table, width, B, used)
    assert int((refs > 0).sum()) == used.item() and bool((refs[:used.item()] > 0).all())
    assert int(table.max()) < used.item()
    keep = [0, 2, 4]
    c.table = table[keep].contiguous()
    after, lse2 = prefix(m, q[keep].contiguous(), c, n0, [rows[b] for b in keep], max_rows=max(rows))
    for i, b in enumerate(keep):
        check(after[i], lse2[i], attend(q[b].double(), c.rows(i, range(rows[b]))), f"sample {b} after the move")
    assert m.csa_read_device_status() == 0
