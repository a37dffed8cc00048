"""The attention operators where the device, the arguments or the cache are at an edge: fewer SMs than the plan
counts on, infinities in rows that are attended, lengths out of range, streams given by the caller."""
import math

import pytest

from test_gpu_5_operators import (BOUNDS, D, RUNS, SCALE, Cache, attend, check, gen, m, prefix, randn,  # noqa: F401
                                  window)

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
