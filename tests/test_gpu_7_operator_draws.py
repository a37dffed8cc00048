"""csa_prefix_attn and csa_window_attn on drawn calls: sizes, page sizes and gaps, lengths on both sides of their
bounds, pages that are not there, values that are not finite, few SMs -- together, against the formula in 64 bits."""
import math
import random

import pytest

from test_gpu_5_operators import BOUNDS, D, attend, gen, m, randn  # noqa: F401
from test_gpu_6_operator_edges import capped, dirty  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def log_uniform(r, lo, hi):
    return int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))


class Drawn:
    """A cache with what can be wrong with one: gaps of NaN between pages, entries that name no page, and rows with a
    NaN or an infinity."""

    def __init__(self, r, g, B, positions):
        self.rpp = rpp = r.choice((1, 3, 16, 17, 32, 40, 48, 64, 64, 64, 128, 250))
        self.width = max(1, -(-positions // rpp) + r.choice((0, 0, 2)))
        self.pitch = rpp + r.choice((0, 0, 0, 1, 3, 16))
        self.n_pages = B * self.width + r.randint(0, 4)
        self.pool = randn(g, self.n_pages * self.pitch, D)
        if r.random() < 0.3:
            self.pool.view(self.n_pages, self.pitch, D)[:, rpp:] = math.nan
        order = torch.randperm(self.n_pages, generator=g, device="cuda")
        if r.random() < 0.3:
            order = order.sort().values
        self.table = order[:B * self.width].to(torch.int32).view(B, -1).clone()
        for _ in range(r.choice((0, 0, 1, 3, 20))):
            self.pool[r.randrange(len(self.pool)), r.randrange(D)] = r.choice((math.inf, -math.inf, math.nan))
        if r.random() < 0.05:
            self.pool[:, r.randrange(D)] = math.inf
        for _ in range(r.choice((0, 0, 0, 0, 2))):
            self.table[r.randrange(B), r.randrange(self.width)] = r.choice((-1, -7, 1 << 30, self.n_pages))

    def rows(self, b, js):
        js = torch.as_tensor(list(js), dtype=torch.int64, device="cuda")
        js = js[js < self.width * self.rpp]
        page = self.table[b].long()[js // self.rpp]
        there = (page >= 0) & (page < self.n_pages)
        return self.pool[page[there] * self.pitch + js[there] % self.rpp].double()

    def paged(self, m):  # noqa: F811
        return m.paged(self.pool, self.rpp, 1024, self.table, page_stride_bytes=self.pitch * 1024, n_pages=self.n_pages)


def check_formula(out, lse, q, kv, where):
    """NaN where the formula has it and nowhere else; the rest within attend()'s bounds over the finite rows."""
    scale = 1 / math.sqrt(D)
    if not len(kv):
        assert bool((out == 0).all()) and bool((lse == -math.inf).all()), where
        return
    x = scale * (q @ kv.t())
    full = torch.logsumexp(x, -1)
    nan = torch.isnan(torch.exp(x - full[:, None]) @ kv)
    assert torch.equal(torch.isnan(out), nan), where
    o, l, to, tl = attend(q, kv[torch.isfinite(kv).all(1)])
    assert float(torch.where(nan, -to, (out.double() - o).abs() - to).max()) <= 0, where
    fin = torch.isfinite(full)
    assert not bool(torch.isfinite(lse[~fin]).any()), where
    assert not bool(fin.any()) or float(((lse.double() - l).abs() - tl)[fin].max()) <= 0, where


@pytest.mark.parametrize("seed", range(32))
def test_drawn_prefix_attention(m, capped, seed):  # noqa: F811
    r, g = random.Random(seed), gen(seed)
    B, H = log_uniform(r, 1, 60), r.choice((1, 2, 16, 128, r.randint(1, 128)))
    shared = r.choice((0, log_uniform(r, 1, 4000)))
    most = max(shared, 1) + r.choice((0, 0, log_uniform(r, 1, 1200)))
    c = Drawn(r, g, B, most)
    n = [r.choice((r.randint(0, most), most, shared, r.randint(shared, most), -5, most + 3)) for _ in range(B)]
    q = randn(g, B, H, D)
    out, lse = torch.full_like(q, 7.0), torch.full((B, H), 7.0, dtype=torch.float32, device="cuda")
    need = m.csa_prefix_attn_workspace_size(B, H, shared, most)
    capped(r.choice((0, 0, 1, 5, 40)))
    m.csa_prefix_attn(q, B, H, 1 / math.sqrt(D), c.paged(m), c.width, shared, torch.tensor(n, device="cuda"), most, out, lse,
                      dirty(need), need)
    status = m.csa_read_device_status()
    assert status in (0, BOUNDS) and (status or all(0 <= x <= most for x in n))
    for b in range(B) if B <= 12 else r.sample(range(B), 12):
        k = min(max(n[b], 0), most)
        kv = torch.cat([c.rows(0, range(min(k, shared))), c.rows(b, range(shared, k))])
        check_formula(out[b], lse[b], q[b].double(), kv, f"request {b} of {n[b]} rows")


@pytest.mark.parametrize("seed", range(32))
def test_drawn_window_attention(m, capped, seed):  # noqa: F811
    r, g = random.Random(1000 + seed), gen(1000 + seed)
    B, H = log_uniform(r, 1, 30), r.choice((1, 16, 24, 128, r.randint(1, 128)))
    W, S = r.choice((1, log_uniform(r, 1, 3000), 128, 1 << 29)), r.choice((0, 1, 4, r.randint(0, 300), 1 << 29))
    q_len = [r.choice((0, 1, 1, log_uniform(r, 1, 150))) for _ in range(B - 1)] + [1]
    before = r.choice((0, log_uniform(r, 1, 3000)))
    n = [max(0, x + r.randint(0, before) - r.choice((0, 0, 0, 2))) for x in q_len]
    c = Drawn(r, g, B, max(n + [1]) - r.choice((0, 0, 0, 1)))
    for b in range(B):  # pages behind every window given back
        for p in range(c.width if r.random() < 0.5 else 0):
            if p * c.rpp >= S and (p + 1) * c.rpp <= n[b] - q_len[b] + 1 - W:
                c.table[b, p] = r.choice((-1, 1 << 29))
    T, extra = sum(q_len), r.choice((0, 5))
    q = randn(g, T + extra, H, D)
    out, lse = torch.full_like(q, 7.0), torch.full((T + extra, H), 7.0, dtype=torch.float32, device="cuda")
    at = [sum(q_len[:b]) for b in range(B + 1)]
    capped(r.choice((0, 0, 1, 5, 40)))
    m.csa_window_attn(q, H, 1 / math.sqrt(D), c.paged(m), c.width, B, torch.tensor(at, device="cuda"),
                      torch.tensor(n, device="cuda"), T + extra, max(q_len), W, S, out, lse)
    assert m.csa_read_device_status() in (0, BOUNDS)
    assert bool((out[T:] == 7).all()) and bool((lse[T:] == 7).all())
    tokens = [(b, i) for b in range(B) for i in range(q_len[b])]
    for b, i in tokens if len(tokens) <= 40 else r.sample(tokens, 40):
        p, t = n[b] - q_len[b] + i, at[b] + i
        lo = max(0, p - W + 1)
        kv = c.rows(b, [*range(min(S, lo)), *range(lo, p + 1)] if p >= 0 else [])
        check_formula(out[t], lse[t], q[t].double(), kv, f"sequence {b} token {i} at {p}")
