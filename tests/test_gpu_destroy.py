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
