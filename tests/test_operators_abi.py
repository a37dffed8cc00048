"""What csa_prefix_attn, csa_window_attn and the csa_pages_* calls refuse on the host, before anything is
enqueued (no GPU: the pointers below are never dereferenced)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def csa():
    from deepseek_v4_hybrid_c4_gb300 import build
    build.build()
    import deepseek_v4_hybrid_c4_gb300 as m
    return m


A16, A4, A2 = (ctypes.c_void_p(0x10000 + x) for x in (0, 4, 2))


def kv(csa, base=0x20000, table=0x30000, rpp=64, stride=64 * 1024, pages=100):
    return csa.csa_paged(base, table, rpp, stride, pages)


def test_prefix_attn_refusals(csa):
    f = csa.lib().csa_prefix_attn

    def go(q=A16, B=2, H=16, cache=None, stride=10, shared=100, n_rows=A16, max_rows=200, out=A16, lse=A4, ws=A16,
           ws_bytes=1 << 40):
        return f(q, B, H, 0.04, cache or kv(csa), stride, shared, n_rows, max_rows, out, lse, ws, ws_bytes, None)

    inv, uns = csa.CSA_ERR_INVALID_ARG, csa.CSA_ERR_UNSUPPORTED
    for kw in ({"H": 0}, {"H": 129}, {"B": 0}, {"B": 65536}, {"max_rows": 1 << 31},
               {"cache": kv(csa, stride=64 * 1024 + 16)}, {"cache": kv(csa, pages=1 << 26)}):
        assert go(**kw) == uns, kw
    for kw in ({"q": None}, {"q": A4}, {"out": None}, {"out": A4}, {"lse": A2}, {"n_rows": None}, {"n_rows": A4},
               {"shared": -1}, {"shared": 201}, {"stride": 3}, {"stride": 0}, {"cache": kv(csa, base=None)},
               {"cache": kv(csa, base=0x20008)}, {"cache": kv(csa, table=None)}, {"cache": kv(csa, table=0x30002)},
               {"cache": kv(csa, rpp=0)}, {"cache": kv(csa, rpp=65)}, {"cache": kv(csa, pages=0)}):
        assert go(**kw) == inv, kw
    need = csa.csa_prefix_attn_workspace_size(2, 16, 100, 200)
    assert need > 0
    for kw in ({"ws": None}, {"ws": A4}, {"ws_bytes": need - 1}):
        assert go(**kw) == csa.CSA_ERR_WORKSPACE, kw
    assert csa.csa_prefix_attn_workspace_size(0, 16, 100, 200) == 0
    assert csa.csa_prefix_attn_workspace_size(2, 16, 300, 200) == 0


def test_prefix_attn_longest_context(csa):
    assert csa.csa_prefix_attn_workspace_size(2, 16, 100, (1 << 31) - 128) > 0
    assert csa.csa_prefix_attn_workspace_size(2, 16, 100, (1 << 31) - 127) == 0


def test_window_attn_refusals(csa):
    f = csa.lib().csa_window_attn

    def go(q=A16, H=16, cache=None, stride=10, B=2, off=A16, n=A16, total=50, max_q=30, window=128, sink=4, out=A16,
           lse=A4, ws=A16, ws_bytes=1 << 40):
        return f(q, H, 0.04, cache or kv(csa), stride, B, off, n, total, max_q, window, sink, out, lse, ws, ws_bytes,
                 None)

    inv, uns = csa.CSA_ERR_INVALID_ARG, csa.CSA_ERR_UNSUPPORTED
    for kw in ({"H": 0}, {"H": 129}, {"B": 0}, {"B": 65536}, {"window": (1 << 30) + 1}, {"sink": (1 << 30) + 1},
               {"total": 1 << 28}, {"cache": kv(csa, stride=64 * 1024 + 16)}, {"cache": kv(csa, pages=1 << 26)}):
        assert go(**kw) == uns, kw
    for kw in ({"q": None}, {"q": A4}, {"out": None}, {"out": A4}, {"lse": A2}, {"off": None}, {"off": A4}, {"n": None},
               {"n": A4}, {"window": 0}, {"sink": -1}, {"total": -1}, {"max_q": 0}, {"stride": 0},
               {"cache": kv(csa, table=None)}, {"cache": kv(csa, rpp=65)}):
        assert go(**kw) == inv, kw
    assert go(total=0) == csa.CSA_OK  # no rows: nothing to do
    need = csa.csa_window_attn_workspace_size(1, 16, 1, 1, 4096, 4)
    if need:
        for kw in ({"ws": None}, {"ws": A4}, {"ws_bytes": need - 1}):
            assert go(B=1, total=1, max_q=1, window=4096, **kw) == csa.CSA_ERR_WORKSPACE, kw


def pools(csa, n_pools=2, n_pages=100, base=0x40000, nbytes=256, stride=512):
    d = csa.csa_page_pools()
    d.n_pools, d.n_pages = n_pools, n_pages
    for i in range(min(max(n_pools, 0), csa.CSA_POOLS_MAX)):
        d.base[i], d.page_bytes[i], d.page_stride[i] = base, nbytes, stride
    return d


BAD_POOLS = [{"n_pools": 0}, {"n_pools": 5}, {"n_pages": 0}, {"base": None}, {"base": 0x40008}, {"nbytes": 0},
             {"nbytes": 24}, {"stride": 24}, {"stride": 240}]
BAD_TABLE = [{"refs": None}, {"refs": A2}, {"table": None}, {"table": A2}, {"B": 0}, {"stride": 0}]


def test_pages_refusals(csa):
    L = csa.lib()
    inv, uns, wsp = csa.CSA_ERR_INVALID_ARG, csa.CSA_ERR_UNSUPPORTED, csa.CSA_ERR_WORKSPACE
    need = csa.csa_pages_workspace_size(100)
    assert need > 0 and csa.csa_pages_workspace_size(0) == 0 and csa.csa_pages_workspace_size((1 << 28) + 1) == 0

    def alloc(refs=A4, pages=100, table=A4, stride=7, B=3, first=A4, count=A4, ws=A16, nb=need):
        return L.csa_pages_alloc(refs, pages, table, stride, B, first, count, ws, nb, None)

    def free(refs=A4, pages=100, table=A4, stride=7, B=3, rows=A4, R=2):
        return L.csa_pages_free(refs, pages, table, stride, B, rows, R, None)

    def fork(p=None, refs=A4, table=A4, stride=7, B=3, src=A4, dst=A4, F=2, n=A16, rpp=64, ws=A16, nb=need):
        return L.csa_pages_fork(ctypes.byref(p or pools(csa)), refs, table, stride, B, src, dst, F, n, rpp, ws, nb, None)

    def compact(p=None, refs=A4, refs_out=A4, table=A4, table_out=A4, stride=7, B=3, n=A16, ws=A16, nb=need):
        return L.csa_pages_compact(ctypes.byref(p or pools(csa)), refs, refs_out, table, table_out, stride, B, n, ws, nb,
                                   None)

    for call in (alloc, free, fork, compact):
        for kw in BAD_TABLE:
            assert call(**kw) == inv, (call.__name__, kw)
        for kw in ({"B": 65536}, {"stride": 1 << 31}):
            assert call(**kw) == uns, (call.__name__, kw)
    for call in (fork, compact):
        for kw in BAD_POOLS:
            assert call(p=pools(csa, **kw)) == inv, (call.__name__, kw)
        assert call(p=pools(csa, n_pages=(1 << 28) + 1)) == uns
    for call in (alloc, fork, compact):
        for kw in ({"ws": None}, {"ws": A4}, {"nb": need - 1}):
            assert call(**kw) == wsp, (call.__name__, kw)
    assert alloc(first=None) == inv and alloc(count=A2) == inv and alloc(B=4097) == uns and alloc(pages=0) == inv
    assert free(rows=None) == inv and free(R=-1) == inv and free(R=65536) == uns and free(R=0) == csa.CSA_OK
    for kw in ({"src": None}, {"dst": A2}, {"n": None}, {"n": A4}, {"rpp": 0}, {"F": -1}):
        assert fork(**kw) == inv, kw
    assert fork(F=1025) == uns and fork(F=0) == csa.CSA_OK
    assert compact(refs_out=None) == inv and compact(table_out=A2) == inv and compact(n=A4) == inv
    cp = L.csa_pages_copy
    assert cp(ctypes.byref(pools(csa)), None, A4, 1, None) == inv and cp(ctypes.byref(pools(csa)), A4, A4, -1, None) == inv
    assert cp(None, A4, A4, 1, None) == inv and cp(ctypes.byref(pools(csa)), None, None, 0, None) == csa.CSA_OK


def test_calls_of_nothing(csa):
    """Empty tensors have null pointers: nothing to do is no error."""
    L = csa.lib()
    pools = csa.csa_page_pools(1, 10, (0x10000,), (1024,), (1024,))
    assert L.csa_window_attn(None, 16, 0.04, kv(csa), 10, 2, A16, A16, 0, 1, 128, 4, None, None, None, 0, None) == 0
    assert L.csa_pages_free(A16, 10, A16, 5, 2, None, 0, None) == 0
    assert L.csa_pages_fork(ctypes.byref(pools), A16, A16, 5, 2, None, None, 0, A16, 64, A16, 1 << 20, None) == 0
    assert L.csa_pages_copy(ctypes.byref(pools), None, None, 0, None) == 0
    assert L.csa_pages_free(A16, 10, A16, 5, 2, None, 1, None) == csa.CSA_ERR_INVALID_ARG


def test_page_pools_struct_matches_the_header(csa, tmp_path):
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    st = csa.csa_page_pools
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "csa.h"', "int main(void) {",
             'printf("%zu\\n", sizeof(csa_page_pools));']
    lines += [f'printf("%zu\\n", offsetof(csa_page_pools, {f}));' for f, _ in st._fields_] + ["return 0;", "}"]
    (tmp_path / "l.c").write_text("\n".join(lines))
    subprocess.check_call([cc, "-I", os.path.join(root, "include"), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")])
    got = [int(x) for x in subprocess.check_output([str(tmp_path / "l")], text=True).split()]
    assert got == [ctypes.sizeof(st)] + [getattr(st, f).offset for f, _ in st._fields_]


def test_page_pools_helper_refuses(csa):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        csa.page_pools([], 4)
    with pytest.raises(ValueError):
        csa.page_pools([torch.zeros(3, 8)], 4)
    with pytest.raises(ValueError):
        csa.page_pools([torch.zeros(4, 8, 8).transpose(1, 2)], 4)
    assert csa.status_string(csa.CSA_ERR_NO_PAGES) == "no free page left in the pool"


def test_window_attn_takes_any_bound_on_new_tokens(csa):
    """max_q is a bound, up to the largest integer: beyond the rows of the buffers it bounds nothing."""
    f = csa.lib().csa_window_attn
    for args in ((1, 16, 1, 4096, 4), (7, 128, 9000, 128, 4), (3, 5, 40, 1 << 17, 0)):
        B, H, total, window, sink = args
        want = csa.csa_window_attn_workspace_size(B, H, total, (1 << 31) - 1, window, sink)
        for max_q in (1 << 31, 1 << 40, (1 << 63) - 1):
            assert csa.csa_window_attn_workspace_size(B, H, total, max_q, window, sink) == want
            if want:
                assert f(A16, H, 0.04, kv(csa), 10, B, A16, A16, total, max_q, window, sink, A16, A4, A16, want - 1,
                         None) == csa.CSA_ERR_WORKSPACE
    assert csa.csa_window_attn_workspace_size(1, 16, 1, (1 << 31) - 1, 4096, 4) > 0


def test_page_pools_helper_refuses_empty_pools(csa):
    torch = pytest.importorskip("torch")
    for n in (0, -1):
        with pytest.raises(ValueError):
            csa.page_pools([torch.zeros(0, 8)], n)


def test_window_attn_workspace_of_a_window_over_everything(csa):
    """A window wider than the page table's positions needs the workspace of one that reaches over them, whatever
    csa_window_attn_workspace_size says for its width."""
    f = csa.lib().csa_window_attn
    size = csa.csa_window_attn_workspace_size

    def go(window, sink, nbytes, stride=128, rpp=64):
        return f(A16, 128, 0.04, kv(csa, rpp=rpp, stride=rpp * 1024), stride, 1, A16, A16, 8192, 8192, window, sink, A16, A4,
                 A16 if nbytes else None, nbytes, None)

    for window in (1 << 17, 1 << 19, (1 << 19) + 1, 1 << 20, 1 << 30):
        for sink in (0, 4, 1 << 30):
            assert go(window, sink, 0) != csa.CSA_ERR_WORKSPACE, (window, sink)
    # a table row of 2^21 positions: as much as for a window of them
    need = size(1, 128, 8192, 8192, 1 << 21, 0)
    assert need > 0
    for window in (1 << 21, 1 << 22, 1 << 30):
        assert go(window, 0, need - 1, stride=1 << 15) == csa.CSA_ERR_WORKSPACE
        assert go(window, 0, need, stride=1 << 15) != csa.CSA_ERR_WORKSPACE
