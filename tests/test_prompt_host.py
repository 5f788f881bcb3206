"""Prompts' attention, weights of keys and of steps: what the host decides (no GPU needed).

Every refusal runs before any CUDA call, so the pointers below are made-up addresses that nothing
dereferences."""
import ctypes
import math
import os
import subprocess

import pytest

from kv_cache_token_bf16_gb300 import binding
from kv_cache_token_bf16_gb300.binding import EVICT_EINVAL, EVICT_ELIMIT, EvictPrompt, EvictRows

HERE = os.path.dirname(os.path.abspath(__file__))
A = 0x100000                        # an aligned address


def refused(code, match, fn, *args):
    with pytest.raises(binding.EvictError, match=match) as e:
        fn(*args)
    assert e.value.code == code


def test_binding_struct_has_the_headers_layout(tmp_path):
    fields = [f[0] for f in EvictPrompt._fields_]
    src = tmp_path / "s.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "evict.h"\nint main(void){printf("%zu", sizeof('
                   'evict_prompt));' + "".join(f'printf(" %zu", offsetof(evict_prompt, {f}));' for f in fields) + "return 0;}")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(os.path.dirname(HERE), "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(EvictPrompt)] + [getattr(EvictPrompt, f).offset for f in fields]
    from kv_cache_token_bf16_gb300 import prompt
    values = [2, 7] + [x for i in range(4) for x in (A + i, 11 + i, 12 + i, 13 + i, 14 + i)] + [A, A + 1, A + 2, 3, 4, 0.5, A + 3, 99, A + 4, A + 5]
    p = EvictPrompt.from_buffer_copy(prompt._PROMPT.pack(*values))
    flat = []
    for f in fields:
        x = getattr(p, f)
        flat += [x.data, x.stride_b, x.stride_h, x.stride_m, x.heads] if isinstance(x, EvictRows) else [x]
    assert flat == values


def rows(heads, m, at=A, **kw):
    return EvictRows(**dict(dict(data=at, stride_b=heads * m * 128, stride_h=128, stride_m=heads * 128, heads=heads), **kw))


def call(**kw):
    m, hq, hkv = kw.pop("m", 100), kw.pop("hq", 8), kw.pop("hkv", 2)
    base = dict(batch=1, m=m, q=rows(hq, m), k=rows(hkv, m, A << 1), v=rows(hkv, m, A << 2), out=rows(hq, m, A << 3), lse=A << 4,
                weights=A << 5, starts=None, n_seqs=0, last=0, scale=0.0, workspace=None, workspace_bytes=0, error=None, stream=None)
    return EvictPrompt(**dict(base, **kw))


BOTH = [binding.evict_prompt_attention, binding.evict_prompt_weights]


@pytest.mark.parametrize("fn", BOTH)
@pytest.mark.parametrize("code,match,kw", [
    (EVICT_EINVAL, "batch and m", dict(batch=-1)), (EVICT_EINVAL, "batch and m", dict(m=-1)),
    (EVICT_EINVAL, "multiple of k", dict(hq=7)), (EVICT_EINVAL, "multiple of k", dict(hkv=0, k=rows(0, 100))),
    (EVICT_ELIMIT, "more than 128", dict(hq=129, hkv=1)),
    (EVICT_EINVAL, "batch of 1", dict(batch=2, starts=A, n_seqs=1)), (EVICT_EINVAL, "batch of 1", dict(starts=A, n_seqs=-1)),
    (EVICT_ELIMIT, "65537 sequences", dict(starts=A, n_seqs=65537)),
    (EVICT_ELIMIT, "2\\^30", dict(batch=1 << 14, m=1 << 16)), (EVICT_ELIMIT, "2\\^30", dict(batch=1, m=1 << 27)),
    (EVICT_EINVAL, "finite", dict(scale=math.nan)), (EVICT_EINVAL, "4-byte", dict(starts=A + 2, n_seqs=1)),
    (EVICT_EINVAL, "4-byte", dict(lse=A + 1)), (EVICT_EINVAL, "4-byte", dict(weights=A + 1)), (EVICT_EINVAL, "4-byte", dict(error=A + 1)),
    (EVICT_EINVAL, "q must not be NULL", dict(q=rows(8, 100, None))), (EVICT_EINVAL, "k must not be NULL", dict(k=rows(2, 100, None))),
    (EVICT_EINVAL, "q: addresses", dict(q=rows(8, 100, A + 8))), (EVICT_EINVAL, "k: addresses", dict(k=rows(2, 100, stride_m=260))),
    (EVICT_EINVAL, "q: strides", dict(q=rows(8, 100, stride_h=-128))),
    (EVICT_EINVAL, "q is expanded", dict(q=rows(8, 100, stride_h=0))), (EVICT_EINVAL, "k is expanded", dict(k=rows(2, 100, stride_m=0))),
    (EVICT_EINVAL, "k is expanded", dict(batch=2, k=rows(2, 100, stride_b=0))),
])
def test_bad_calls_are_refused(lib, fn, code, match, kw):
    refused(code, match, fn, call(**kw))


@pytest.mark.parametrize("match,kw", [
    ("v must not be NULL", dict(v=rows(2, 100, None))), ("v has 4 heads, not 2", dict(v=rows(4, 100))),
    ("out has 2 heads, not 8", dict(out=rows(2, 100))), ("out must not be q, k or v", dict(out=rows(8, 100, A))),
    ("on top of each other", dict(out=rows(8, 100, A << 3, stride_m=128))), ("out is expanded", dict(out=rows(8, 100, A << 3, stride_h=0))),
])
def test_bad_attention_is_refused(lib, match, kw):
    refused(EVICT_EINVAL, match, binding.evict_prompt_attention, call(**kw))


@pytest.mark.parametrize("match,kw", [("lse and weights", dict(lse=None)), ("lse and weights", dict(weights=None)), ("last", dict(last=-1))])
def test_bad_weights_are_refused(lib, match, kw):
    refused(EVICT_EINVAL, match, binding.evict_prompt_weights, call(**kw))


@pytest.mark.parametrize("fn", BOTH)
def test_nothing_to_do_needs_no_gpu(lib, fn):
    fn(call(m=0))
    fn(call(batch=0))
    fn(call(starts=A, n_seqs=0))
    refused(EVICT_EINVAL, "arguments are NULL", lambda: binding.check(getattr(binding.load(), fn.__name__)(None)))


def test_weigh_without_a_handle_is_refused(lib):
    refused(EVICT_EINVAL, "NULL", binding.evict_weigh, None, rows(8, 1), 1, 1, A, None, 0.0, None)
    assert lib.evict_update_scored(None, A, A, None, A, 1, None) == EVICT_EINVAL


def test_tensors_of_the_cpu_or_with_a_gradient_are_refused(lib):
    torch = pytest.importorskip("torch")
    from kv_cache_token_bf16_gb300 import prompt
    q = torch.zeros(1, 4, 3, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        prompt.attention(q, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        prompt.weights(q, q, torch.zeros(1, 4, 3))
    with pytest.raises(ValueError, match="no gradient"):
        prompt.attention(q.clone().requires_grad_(), q, q)
    with pytest.raises(ValueError, match="no gradient"):
        prompt.weights(q, q, torch.zeros(1, 4, 3, requires_grad=True))
    with pytest.raises(ValueError, match="starts"):
        prompt.Packing(torch.zeros(3))
    with pytest.raises(ValueError, match="CUDA"):
        prompt.Packing(torch.zeros(3, dtype=torch.int32))


def test_weights_want_log_sum_exps(lib):
    torch = pytest.importorskip("torch")
    from kv_cache_token_bf16_gb300 import paged, prompt
    x = torch.zeros(1, 1, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="lse must be given"):
        prompt.weights(x, x, None)
    with pytest.raises(ValueError, match="lse must be given"):
        paged.weigh_rows(None, x, None)
