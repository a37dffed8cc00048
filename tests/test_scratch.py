"""Where the scratch of a call without a workspace comes from (no GPU: the allocator and the streams are fakes)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


class Like:
    is_cuda, device = True, "a device"

    def data_ptr(self):
        return 0x1000


@pytest.fixture
def calls(monkeypatch):
    """The package over a library that takes every call; [(entry point, stream of the call, stream its scratch was
    allocated on)]."""
    import deepseek_v4_hybrid_c4_gb300 as m
    current, got, scratch = [Stream(7)], [], []

    @contextlib.contextmanager
    def on(s):
        current.append(s)
        yield
        current.pop()

    def empty(n, dtype=None, device=None):
        scratch.append(current[-1].cuda_stream)
        return Like()

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return lambda *a: 4096

            def call(*a):
                got.append((name, a[-1], scratch.pop() if scratch else None))
                return 0
            return call

    monkeypatch.setattr(m, "lib", Lib)
    monkeypatch.setattr(m, "_current_stream", lambda: current[-1].cuda_stream)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(Like, "record_stream", lambda self, s: None, raising=False)
    x = Like()
    kv = m.csa_paged(0x1000, 0x2000, 64, 65536, 10)
    pools = m.csa_page_pools(1, 10, (0x1000,), (1024,), (1024,))

    def go(stream):
        got.clear()
        m.csa_prefix_attn(x, 2, 16, 0.04, kv, 10, 100, x, 200, x, stream=stream)
        m.csa_window_attn(x, 16, 0.04, kv, 10, 2, x, x, 50, 30, 128, 4, x, stream=stream)
        m.csa_pages_alloc(x, 10, x, 5, 2, x, x, stream=stream)
        m.csa_pages_fork(pools, x, x, 5, 2, x, x, 1, x, 64, stream=stream)
        m.csa_pages_compact(pools, x, x, x, x, 5, 2, stream=stream)
        m.csa_topk(x, 100, 10, x, stream=stream)
        m.csa_topk_batched(x, x, 2, 100, 10, x, stream=stream)
        m.csa_topk_merge(x, x, x, 2, 10, stream=stream)
        m.csa_sparse_attn_partial(x, 16, 0.04, kv, x, 10, kv, 100, 128, x, x, stream=stream)
        return list(got)
    return go


@pytest.mark.parametrize("stream,handle", [(None, 7), (Stream(99), 99), (99, 99), (0, 0)])
def test_scratch_is_allocated_on_the_stream_of_the_call(calls, stream, handle):
    """A block from another stream's pool may still be read by work that is pending there."""
    got = calls(stream)
    assert len(got) == 9
    for name, used, allocated in got:
        assert (used, allocated) == (handle, handle), name
