"""Prompts' attention, weights of keys and of steps: rarer calls' refusals, and what reading alone can show (no GPU needed)."""
import math
import os
import re
from types import SimpleNamespace

import pytest

from kv_cache_token_bf16_gb300 import binding
from kv_cache_token_bf16_gb300.binding import EVICT_EINVAL, EVICT_ELIMIT
from tests.test_prompt_host import A, call, refused, rows

CSRC = os.path.join(os.path.dirname(os.path.abspath(binding.__file__)), "csrc")


def body(file, head):
    """The text of the function that begins with `head`."""
    text = open(os.path.join(CSRC, file)).read()
    at = text.index("{", text.index(head))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return re.sub(r"//[^\n]*", "", text[at:i + 1])
    raise AssertionError(head)


def test_warps_that_meet_at_a_barrier_leave_it_together():
    # warps w and w + 8 sum halves of the same keys and meet at a barrier that nothing bounds. A warp that left the loop
    # on its own (a wait that gave up makes read_unit's answer differ between the two) would leave the other there for
    # good: every way out has to be a decision of both.
    text = body("weights.cu", "void sum_warp(")
    exits = [line.strip() for line in text.splitlines() if re.search(r"\b(break|return|goto)\b", line)]
    assert len(exits) == 2
    for line in exits:
        assert re.fullmatch(r"if \(!named_and\(1 \+ \(warp & 7\), 64, .+\)\) break;", line), line


# 8 query heads and as many KV heads, 100 tokens: log-sum-exps and weights are 3200 bytes each
@pytest.mark.parametrize("match,kw", [
    ("overlap lse", dict(weights=A)), ("overlap lse", dict(weights=A + 3196)), ("overlap lse", dict(weights=A - 3196)),
    ("be q or k", dict(weights=A << 3)), ("be q or k", dict(weights=A << 4))])
def test_weights_over_what_they_are_made_of_are_refused(lib, match, kw):
    base = dict(hkv=8, q=rows(8, 100, A << 3), k=rows(8, 100, A << 4), lse=A)
    refused(EVICT_EINVAL, match, binding.evict_prompt_weights, call(**dict(base, **kw)))


def test_weights_beside_their_log_sum_exps_are_not_refused(lib):
    for at in (A + 3200, A - 3200):
        with pytest.raises(binding.EvictError) as e:             # the workspace, or no GPU here
            binding.evict_prompt_weights(call(hkv=8, lse=A, weights=at))
        assert "overlap" not in str(e.value)


def test_queries_on_another_device_than_the_caches_are_refused(lib):
    # (tensors and a cache that say where they are: two devices are more than there may be)
    pytest.importorskip("torch")
    from kv_cache_token_bf16_gb300 import paged
    q = SimpleNamespace(shape=(1, 4, 1, 128), requires_grad=False, get_device=lambda: 1, device="cuda:1")
    lse = SimpleNamespace(requires_grad=False)
    with pytest.raises(ValueError, match="cache is on CUDA device 0, q on 1"):
        paged.weigh_rows(SimpleNamespace(device_index=0, handle=None), q, lse)


def fake_streams(monkeypatch, torch):
    """Device 0 is current, whose current stream has the number of the cache's; the cache is on device 1. Returns it and
    the log of who waited for whom."""
    log = []

    class Stream:
        def __init__(self, number, device=None):
            self.at = device, number

        def wait_stream(self, other):
            log.append((self.at, other.at))

    class Context:
        def __init__(self, *_):
            pass

        def __enter__(self):
            pass

        __exit__ = __init__

    monkeypatch.setattr(binding, "evict_get_stream", lambda handle: 77)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: (77, 5)[index], raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index=0: Stream((77, 5)[index], index))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    for name, fake in (("ExternalStream", Stream), ("stream", Context), ("device", Context)):
        monkeypatch.setattr(torch.cuda, name, fake)
    cache = binding.EvictCache.__new__(binding.EvictCache)
    cache.handle, cache.device_index, cache.method = None, 1, "attention"
    return cache, log


def test_streams_are_ordered_on_the_caches_device(lib, monkeypatch):
    torch = pytest.importorskip("torch")
    from kv_cache_token_bf16_gb300 import paged
    cache, log = fake_streams(monkeypatch, torch)
    monkeypatch.setattr(paged, "weigh_rows", lambda *a, **kw: log.append("weigh"))
    cache.weigh(None, None)
    assert log == [((1, 5), (1, 77)), "weigh", ((1, 77), (1, 5))]


def test_work_before_a_refusal_is_ordered_all_the_same(lib, monkeypatch):
    # the attention is on its way when the weights are refused: the cache's next update still comes behind it
    torch = pytest.importorskip("torch")
    from kv_cache_token_bf16_gb300 import paged
    cache, log = fake_streams(monkeypatch, torch)

    def refuse(*a, **kw):
        raise ValueError("refused")

    monkeypatch.setattr(paged, "shared_attention", lambda *a, **kw: log.append("attend"))
    monkeypatch.setattr(paged, "weigh_rows", refuse)
    monkeypatch.setattr(cache, "view", lambda: (None,) * 4, raising=False)
    with pytest.raises(ValueError, match="refused"):
        cache.attend(None, lse=0, weigh=True)
    assert log == [((1, 5), (1, 77)), "attend", ((1, 77), (1, 5))]


def fake_rows(monkeypatch, device_index):
    """A cache of 2 KV heads with room for 8 rows, and the devices that tensors over them are asked for on."""
    torch = pytest.importorskip("torch")
    asked = []

    def as_tensor(x, device=None):
        asked.append(str(device))
        at = x.__cuda_array_interface__
        return torch.zeros(at["shape"], dtype={"<i2": torch.int16, "<f4": torch.float32, "<i4": torch.int32}[at["typestr"]])

    monkeypatch.setattr(torch, "as_tensor", as_tensor)
    cache = binding.EvictCache.__new__(binding.EvictCache)
    cache.handle, cache.device_index, cache.batch, cache.heads, cache.dtype = None, device_index, 1, 2, "bf16"
    cache._held, cache._rows, cache._views = None, None, (-1, None)
    return cache, asked


def test_views_are_made_on_the_caches_device(lib, monkeypatch):
    cache, asked = fake_rows(monkeypatch, 3)
    cache._kept(binding.EvictView(A, A, A, A, 5, 8))
    assert asked == ["cuda:3"] * 4


def test_views_are_the_callers_own_objects(lib, monkeypatch):
    torch = pytest.importorskip("torch")
    cache, asked = fake_rows(monkeypatch, 0)
    view = binding.EvictView(A, A, A, A, 5, 8)
    first = cache._kept(view)
    first[0].requires_grad_()
    first[3].unsqueeze_(0)
    first[2].transpose_(0, 1)
    second = cache._kept(view)
    assert [x.shape for x in second] == [(1, 2, 5, 128), (1, 2, 5, 128), (1, 2, 5), (1, 2, 5)]
    assert not any(x.requires_grad for x in second) and len(asked) == 4
    second[3].fill_(3.0)                            # the same rows
    assert (first[3] == 3).all() and (cache._kept(view)[3] == 3).all()
    versions = [x._version for x in first]
    cache._kept(view)[0].add_(1.0)
    assert [x._version for x in first] == versions and (first[0] == 1).all()
    with torch.inference_mode():
        third = cache._kept(view)
    third[3].add_(1.0)
    assert (second[3] == 4).all()


# a plane of 2^20 tokens and more in short sequences, or of which a window counts: by their plane's length alone these
# would be 2^31 steps. (What they need, or without a GPU an error that there is none.)
@pytest.mark.parametrize("fn", [binding.evict_prompt_attention_workspace, binding.evict_prompt_weights_workspace])
@pytest.mark.parametrize("hq,hkv,m,n,last", [(64, 8, 1 << 20, 1024, 0), (1, 1, (1 << 23) + 77, 16385, 0), (64, 8, 1 << 21, 1, 64),
                                             (128, 128, (1 << 23) - 1, 65536, 0)])
def test_long_planes_are_no_long_sequences(lib, fn, hq, hkv, m, n, last):
    a = call(hq=hq, hkv=hkv, m=m, starts=A, n_seqs=n, last=last)
    try:
        assert 0 < fn(a) < 1 << 30
    except binding.EvictError as e:
        assert e.code == binding.EVICT_ECUDA, e


@pytest.mark.parametrize("fn", [binding.evict_prompt_attention_workspace, binding.evict_prompt_weights_workspace])
def test_too_many_units_are_refused(lib, fn):
    refused(EVICT_ELIMIT, "units", fn, call(hq=1 << 15, hkv=1 << 15, m=1000, starts=A, n_seqs=65536))


def test_scales_that_are_none_in_fp32_are_refused(lib):
    # (0 is the C calls' default)
    torch = pytest.importorskip("torch")
    from kv_cache_token_bf16_gb300 import paged, prompt
    q = SimpleNamespace(shape=(1, 4, 1, 128), requires_grad=False, get_device=lambda: 0, device="cuda:0", dtype=torch.bfloat16,
                        stride=lambda: (512, 128, 512, 1), data_ptr=lambda: A)
    lse = SimpleNamespace(requires_grad=False)
    for scale in (0, 0.0, 1e-50, -1e-46):
        with pytest.raises(ValueError, match="scale must not be 0"):
            prompt.attention(q, q, q, scale=scale, out=q)
        with pytest.raises(ValueError, match="scale must not be 0"):
            prompt.weights(q, q, lse, scale=scale)
        with pytest.raises(ValueError, match="scale must not be 0"):
            paged.weigh_rows(SimpleNamespace(device_index=0, handle=None), q, lse, scale=scale)
        with pytest.raises(ValueError, match="scale must not be 0"):
            paged.shared_attention(q, scale=scale, out=q)
    assert paged._scale(None) == 0 and paged._scale(1e-45) > 0 and paged._scale(-0.25) == -0.25
    for fn in (binding.evict_prompt_attention, binding.evict_prompt_weights):
        for scale in (math.inf, -math.inf, 2.0 ** 127, -3e38):
            refused(EVICT_EINVAL, "finite", fn, call(scale=scale))


def test_log_sum_exps_that_require_a_gradient_are_refused(lib):
    torch = pytest.importorskip("torch")
    from kv_cache_token_bf16_gb300 import prompt
    q = torch.zeros(1, 4, 3, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="no gradient"):
        prompt.attention(q, q, q, lse=torch.zeros(1, 4, 3, requires_grad=True))
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        prompt.attention(q, q, q, lse=torch.zeros(1, 4, 3, requires_grad=True))
