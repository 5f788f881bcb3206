"""Handles may be destroyed at any time, e.g. by a garbage collector during a graph's capture."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("method", ["knorm", "curdkv"])
@pytest.mark.parametrize("own_stream", [False, True])
def test_a_handle_destroyed_during_a_capture(method, own_stream):
    from kv_cache_token_bf16_gb300 import binding
    stream, other = torch.cuda.Stream(), torch.cuda.Stream()
    kw = dict(budget=64, max_block=32, n_sink=4, recent=8)
    k, v = (torch.randn(2, 2, 32, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        kept = binding.EvictCache("knorm", 2, 2, stream=stream.cuda_stream, **kw)
        kept.update_and_fetch(k, v)
    gone = binding.EvictCache(method, 2, 2, stream=other.cuda_stream if own_stream else 0, **kw)
    gone.update_and_fetch(k, v)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        kept.update_and_fetch(k, v)
        gone.close()
    g.replay()
    stream.synchronize()
    kept.sync()
    got = kept.view()[0]
    assert torch.equal(got[:, :, :32], k) and torch.equal(got[:, :, 32:64], k)


def cudart():
    """The runtime that the library uses: a capture that ends with an error is no business of torch's."""
    import ctypes
    torch.cuda.init()
    path = next(x.split()[-1] for x in open("/proc/self/maps") if "libcudart.so" in x)
    rt = ctypes.CDLL(path)
    rt.cudaStreamBeginCapture.argtypes = [ctypes.c_void_p, ctypes.c_int]
    rt.cudaStreamEndCapture.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)]
    rt.cudaGraphDestroy.argtypes = [ctypes.c_void_p]
    return rt


@pytest.mark.parametrize("method,call", [("knorm", "update"), ("curdkv", "update"), ("knorm", "group"),
                                         ("knorm", "state"), ("curdkv", "scores")])
@pytest.mark.parametrize("holds", [True, False], ids=["holds", "apart"])
def test_a_handle_destroyed_while_its_own_stream_captures(method, call, holds):
    # a graph that holds the handle's work must not come to be: it would write to freed memory
    import ctypes
    from kv_cache_token_bf16_gb300 import binding
    stream, rt = torch.cuda.Stream(), cudart()
    kw = dict(budget=64, max_block=32, n_sink=4, recent=8)
    k, v = (torch.randn(2, 2, 32, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
    pos = torch.arange(32, dtype=torch.int32, device="cuda").expand(2, 2, 32).contiguous()
    scores = torch.zeros(2, 2, 32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        kept, gone = (binding.EvictCache(method, 2, 2, stream=stream.cuda_stream, **kw) for _ in range(2))
        for c in (kept, gone):
            c.update_and_fetch(k, v)
    torch.cuda.synchronize()

    def work(c):
        if call == "update":
            binding.evict_update_and_fetch(c.handle, k.data_ptr(), v.data_ptr(), None, 8)
        elif call == "group":
            binding.evict_update_and_fetch_group([c.handle], [k.data_ptr()], [v.data_ptr()], None, 8)
        elif call == "state":
            c.set_state(k, v, pos)
        else:
            binding.evict_curdkv_scores(c.handle, scores.data_ptr(), None)

    graph = ctypes.c_void_p()
    assert rt.cudaStreamBeginCapture(stream.cuda_stream, 0) == 0
    work(kept)
    if holds:
        work(gone)
    gone.close()
    code = rt.cudaStreamEndCapture(stream.cuda_stream, ctypes.byref(graph))
    if holds:
        assert code == 901 and not graph.value              # cudaErrorStreamCaptureInvalidated
    else:
        assert code == 0 and graph.value
        assert rt.cudaGraphDestroy(graph) == 0
    assert rt.cudaGetLastError() in ((0, 901) if holds else (0,))
    # nothing else suffers: the stream, the other handle and later captures work
    with torch.cuda.stream(stream):
        kept.reset()
        kept.update_and_fetch(k, v)
    kept.sync()
    assert torch.equal(kept.view()[0], k)
    kept.close()
