"""What csa_quant_write, csa_quant_read and csa_quant_attn refuse on the host, before anything is enqueued (no GPU: the
pointers below are never dereferenced)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def csa():
    from deepseek_v4_hybrid_c4_gb300 import build
    build.build()
    import deepseek_v4_hybrid_c4_gb300 as m
    return m


A16, A8, A4, A2 = (ctypes.c_void_p(0x10000 + x) for x in (0, 8, 4, 2))
PAGE = 64 * 516


def kv(csa, base=0x20000, table=0x30000, rpp=64, stride=PAGE, pages=100):
    return csa.csa_paged(base, table, rpp, stride, pages)


BAD_CACHE = [{"base": None}, {"base": 0x20008}, {"table": None}, {"table": 0x30002}, {"rpp": 0}, {"rpp": 65},
             {"stride": PAGE - 16}, {"stride": PAGE + 8}, {"pages": 0}]


def test_write_and_read_refusals(csa):
    L = csa.lib()
    inv, uns = csa.CSA_ERR_INVALID_ARG, csa.CSA_ERR_UNSUPPORTED

    def write(data=A16, cache=None, stride=10, B=2, off=A8, n=A8, total=50, most=30):
        return L.csa_quant_write(data, cache or kv(csa), stride, B, off, n, total, most, None)

    def read(data=A16, cache=None, stride=10, B=2, off=A8, n=A8, total=50, most=30):
        return L.csa_quant_read(cache or kv(csa), stride, B, off, n, total, most, data, None)

    for f in (write, read):
        for kw in ({"B": 0}, {"B": 65536}, {"total": 1 << 31}, {"cache": kv(csa, pages=1 << 31)}):
            assert f(**kw) == uns, (f.__name__, kw)
        for kw in ({"data": None}, {"data": A8}, {"off": None}, {"off": A4}, {"n": None}, {"n": A4}, {"total": -1},
                   {"most": 0}, {"stride": 0}):
            assert f(**kw) == inv, (f.__name__, kw)
        for kw in BAD_CACHE:
            assert f(cache=kv(csa, **kw)) == inv, (f.__name__, kw)
        assert f(total=0) == csa.CSA_OK and f(total=0, data=None) == csa.CSA_OK
        assert f(total=0, cache=kv(csa, rpp=65)) == inv


def test_attn_refusals(csa):
    f = csa.lib().csa_quant_attn

    def go(q=A16, H=16, cache=None, stride=10, B=2, off=A8, n=A8, total=50, max_q=30, window=128, sink=4, out=A16, lse=A4,
           ws=A16, ws_bytes=1 << 40):
        return f(q, H, 0.04, cache or kv(csa), stride, B, off, n, total, max_q, window, sink, out, lse, ws, ws_bytes, None)

    inv, uns = csa.CSA_ERR_INVALID_ARG, csa.CSA_ERR_UNSUPPORTED
    for kw in ({"H": 0}, {"H": 129}, {"B": 0}, {"B": 65536}, {"window": (1 << 30) + 1}, {"sink": (1 << 30) + 1},
               {"total": 1 << 28}, {"cache": kv(csa, pages=1 << 31)}):
        assert go(**kw) == uns, kw
    for kw in ({"q": None}, {"q": A8}, {"out": None}, {"out": A8}, {"lse": A2}, {"off": None}, {"off": A4}, {"n": None},
               {"n": A4}, {"window": 0}, {"sink": -1}, {"total": -1}, {"max_q": 0}, {"stride": 0}):
        assert go(**kw) == inv, kw
    for kw in BAD_CACHE:
        assert go(cache=kv(csa, **kw)) == inv, kw
    assert go(total=0) == csa.CSA_OK and go(total=0, q=None, out=None, ws=None, ws_bytes=0) == csa.CSA_OK
    need = csa.csa_quant_attn_workspace_size(1, 16, 1, 1, 1 << 30, 0)
    assert need > 0
    for kw in ({"ws": None}, {"ws": A8}, {"ws_bytes": 16}):
        assert go(B=1, total=1, max_q=1, window=1 << 30, sink=0, stride=5000, **kw) == csa.CSA_ERR_WORKSPACE, kw
    assert csa.csa_quant_attn_workspace_size(0, 16, 1, 1, 128, 0) == 0


def test_merge_selftest_refusals(csa):
    f = csa.lib().csa_selftest_quant_merge
    need = csa.csa_quant_attn_workspace_size(1, 1, 40, 40, 1, 0)

    def go(ws=A16, ws_bytes=need, rows=40, out=A16, lse=A4):
        return f(ws, ws_bytes, rows, out, lse, None)

    for kw in ({"ws": None}, {"ws": A8}, {"rows": 0}, {"rows": -1}, {"out": None}, {"out": A8}, {"lse": A2}):
        assert go(**kw) == csa.CSA_ERR_INVALID_ARG, kw
    assert go(ws_bytes=need - 1) == csa.CSA_ERR_WORKSPACE and go(rows=41) == csa.CSA_ERR_WORKSPACE
