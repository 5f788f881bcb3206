"""Rotary positions, pages and shared-prefix attention: what the host decides (no GPU needed).

Every refusal runs before any CUDA call, so the pointers below are made-up addresses that nothing
dereferences."""
import ctypes
import math
import os
import subprocess

import pytest

from kv_cache_token_bf16_gb300 import binding, paged
from kv_cache_token_bf16_gb300.binding import (EVICT_BF16, EVICT_EINVAL, EVICT_ELIMIT, EVICT_FP32, EvictAttention,
                                               EvictPages, EvictRows)

HERE = os.path.dirname(os.path.abspath(__file__))
A = 0x100000                        # an aligned address


def refused(code, match, fn, *args):
    with pytest.raises(binding.EvictError, match=match) as e:
        fn(*args)
    assert e.value.code == code


@pytest.mark.parametrize("struct", ["evict_rows", "evict_rotary_config", "evict_pages", "evict_attention"])
def test_binding_structs_have_the_headers_layout(struct, tmp_path):
    cls = {"evict_rows": EvictRows, "evict_rotary_config": binding.EvictRotaryConfig, "evict_pages": EvictPages,
           "evict_attention": EvictAttention}[struct]
    fields = [f[0] for f in cls._fields_]
    src = tmp_path / "s.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "evict.h"\nint main(void){printf("%zu", sizeof('
                   + struct + "));" + "".join(f'printf(" %zu", offsetof({struct}, {f}));' for f in fields)
                   + "return 0;}")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(os.path.dirname(HERE), "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]


# --- rotations ------------------------------------------------------------------------------
@pytest.mark.parametrize("kw,match", [
    (dict(rotary_dim=0), "rotary_dim"), (dict(rotary_dim=130), "rotary_dim"),
    (dict(rotary_dim=63, inv_freq=[1.0] * 31), "rotary_dim"),
    (dict(n_axes=0), "n_axes"), (dict(n_axes=5), "n_axes"),
    (dict(rotary_dim=4, axis=[0, 2], n_axes=2), "axis 2 of 2"),
    (dict(scale=math.inf), "scale"), (dict(scale=math.nan), "scale"),
    (dict(rotary_dim=4, inv_freq=[1.0, math.nan]), "inv_freq"), (dict(rotary_dim=4, inv_freq=[1.0, 1e6]), "inv_freq"),
])
def test_bad_rotations_are_refused(lib, kw, match):
    refused(EVICT_EINVAL, match, lambda: paged.Rotary(**kw))


@pytest.mark.parametrize("kw", [dict(pairs="other"), dict(rotary_dim=8, inv_freq=[1.0] * 3),
                                dict(rotary_dim=8, axis=[0] * 5), dict(rotary_dim=8, axis=[0] * 4, sections=[4]),
                                dict(rotary_dim=8, sections=[1, 2]), dict(rotary_dim=4, axis=[0, -1])])
def test_bad_rotation_arguments_are_refused(lib, kw):
    with pytest.raises(ValueError):
        paged.Rotary(**kw)


def test_sections_name_the_axes(lib):
    r = paged.Rotary(rotary_dim=16, sections=[4, 2, 2])
    assert r.n_axes == 3
    assert paged.Rotary(rotary_dim=16).n_axes == 1


def test_null_rotation_arguments(lib):
    assert lib.evict_rotary_init(None, None) == EVICT_EINVAL
    out = ctypes.c_void_p()
    assert lib.evict_rotary_init(None, out) == EVICT_EINVAL and out.value is None
    lib.evict_rotary_destroy(None)


def rows(data=A, heads=4, stride_m=128, stride_h=1024, stride_b=4096):
    return EvictRows(data, stride_b, stride_h, stride_m, heads)


@pytest.fixture
def rot(lib):
    return paged.Rotary(rotary_dim=64)


@pytest.mark.parametrize("kw,code,match", [
    (dict(dtype=2), EVICT_EINVAL, "dtype"), (dict(batch=-1), EVICT_EINVAL, "batch"), (dict(m=-1), EVICT_EINVAL, "m must"),
    (dict(pos=A + 2), EVICT_EINVAL, "pos"), (dict(transpose=2), EVICT_EINVAL, "transpose"),
    (dict(x=rows(None)), EVICT_EINVAL, "NULL"), (dict(out=rows(None)), EVICT_EINVAL, "NULL"),
    (dict(x=rows(A + 1)), EVICT_EINVAL, "aligned"), (dict(x=rows(heads=3)), EVICT_EINVAL, "heads"),
    (dict(x=rows(heads=0), out=rows(heads=0)), EVICT_EINVAL, "heads"),
    (dict(out=rows(A, stride_m=256)), EVICT_EINVAL, "in place"),
    (dict(batch=1 << 15, m=1 << 14), EVICT_ELIMIT, "rows"),
    (dict(n=0), EVICT_EINVAL, "tensors"), (dict(n=3), EVICT_EINVAL, "tensors"),
])
def test_bad_rotate_calls_are_refused(rot, kw, code, match):
    a = dict(dtype=EVICT_BF16, batch=2, m=8, pos=None, transpose=0, x=rows(), out=rows(2 * A), n=1)
    a.update(kw)
    refused(code, match, binding.evict_rotate, rot.handle, a["dtype"], a["batch"], a["m"], a["pos"], 0, a["transpose"],
            a["x"], a["out"], a["n"], None)


def test_nothing_to_rotate_is_no_launch(rot, lib):
    before = lib.evict_launch_count()
    binding.evict_rotate(rot.handle, EVICT_BF16, 0, 8, None, 0, 0, rows(), rows(2 * A), 1, None)
    binding.evict_rotate(rot.handle, EVICT_FP32, 2, 0, None, 0, 0, rows(), rows(2 * A), 1, None)
    assert lib.evict_launch_count() == before
    assert lib.evict_rotate(None, 0, 1, 1, None, 0, 0, rows(), rows(2 * A), 1, None) == EVICT_EINVAL


# --- pages ----------------------------------------------------------------------------------
def pages(**kw):
    a = dict(k=A, v=2 * A, page_stride=0, n_pages=8, page_size=16, n_kv_heads=4, dtype=EVICT_BF16, table=3 * A,
             table_stride=0, table_width=4, lens=4 * A, error=None)
    a.update(kw)
    return EvictPages(**a)


BAD_PAGES = [
    (dict(dtype=7), EVICT_EINVAL, "dtype"), (dict(n_pages=0), EVICT_EINVAL, "n_pages"),
    (dict(n_kv_heads=0), EVICT_EINVAL, "n_kv_heads"), (dict(table_width=0), EVICT_EINVAL, "table_width"),
    (dict(page_size=8), EVICT_EINVAL, "page_size"), (dict(page_size=48), EVICT_EINVAL, "page_size"),
    (dict(page_size=512), EVICT_EINVAL, "page_size"), (dict(table_width=1 << 27), EVICT_ELIMIT, "table_width"),
    (dict(k=None), EVICT_EINVAL, "NULL"), (dict(v=None), EVICT_EINVAL, "NULL"), (dict(table=None), EVICT_EINVAL, "NULL"),
    (dict(lens=None), EVICT_EINVAL, "NULL"), (dict(k=A + 8), EVICT_EINVAL, "16-byte"),
    (dict(lens=A + 2), EVICT_EINVAL, "4-byte"), (dict(error=A + 2), EVICT_EINVAL, "4-byte"),
    (dict(page_stride=4 * 16 * 128 - 8), EVICT_EINVAL, "page_stride"),
    (dict(page_stride=4 * 16 * 128 + 4), EVICT_EINVAL, "page_stride"), (dict(table_stride=3), EVICT_EINVAL, "table_stride"),
]


@pytest.mark.parametrize("kw,code,match", BAD_PAGES)
def test_bad_pages_are_refused_by_both_calls(lib, kw, code, match):
    refused(code, match, binding.evict_paged_append, pages(**kw), 2, 1, None, None, None, 0, rows(), rows(), None, None,
            None)
    refused(code, match, binding.evict_shared_attention, attention(pages=pages(**kw)))


@pytest.mark.parametrize("kw,code,match", [
    (dict(k=rows(heads=3)), EVICT_EINVAL, "heads"), (dict(v=rows(heads=8)), EVICT_EINVAL, "heads"),
    (dict(k=rows(None)), EVICT_EINVAL, "NULL"), (dict(v=None), EVICT_EINVAL, "NULL"),
    (dict(q=rows(5 * A)), EVICT_EINVAL, "together"), (dict(q_out=rows(5 * A)), EVICT_EINVAL, "together"),
    (dict(q=rows(5 * A), q_out=rows(6 * A, heads=2)), EVICT_EINVAL, "heads"),
    (dict(q=rows(5 * A), q_out=rows(5 * A, stride_b=8192)), EVICT_EINVAL, "in place"),
    (dict(n_new=A + 1), EVICT_EINVAL, "n_new"), (dict(pos=A + 1), EVICT_EINVAL, "pos"), (dict(m=-2), EVICT_EINVAL, "m must"),
    (dict(batch=1 << 15, m=1 << 14), EVICT_ELIMIT, "rows"),
])
def test_bad_appends_are_refused(rot, kw, code, match):
    a = dict(batch=2, m=1, n_new=None, pos=None, k=rows(5 * A), v=rows(6 * A), q=None, q_out=None)
    a.update(kw)
    refused(code, match, binding.evict_paged_append, pages(), a["batch"], a["m"], a["n_new"], rot.handle, a["pos"], 0,
            a["k"], a["v"], a["q"], a["q_out"], None)


def test_appending_nothing_is_no_launch(lib):
    before = lib.evict_launch_count()
    binding.evict_paged_append(pages(), 0, 1, None, None, None, 0, rows(), rows(), None, None, None)
    binding.evict_paged_append(pages(), 2, 0, None, None, None, 0, rows(), rows(), None, None, None)
    assert lib.evict_launch_count() == before


def test_status_needs_a_word(lib):
    assert lib.evict_pages_status(None, None) == EVICT_EINVAL
    assert lib.evict_pages_status(A + 1, None) == EVICT_EINVAL


# --- attention ------------------------------------------------------------------------------
def attention(**kw):
    a = EvictAttention(batch=4, m=2, n_q_heads=8, n_kv_heads=4, q=rows(A, heads=8), out=rows(2 * A, heads=8),
                       prefix_k=3 * A, prefix_v=4 * A, prefix_stride_b=4 * 64 * 128, prefix_stride_h=64 * 128, n_prefix=64,
                       prefix_batch=2, workspace=5 * A, workspace_bytes=1 << 40)
    g = kw.pop("pages", None)
    for k, v in kw.items():
        setattr(a, k, v)
    if g is not None:
        a.pages = ctypes.pointer(g)
    return a


@pytest.mark.parametrize("kw,code,match", [
    (dict(batch=-1), EVICT_EINVAL, "batch"), (dict(m=-1), EVICT_EINVAL, "m must"),
    (dict(n_q_heads=6), EVICT_EINVAL, "multiple|heads"), (dict(n_kv_heads=0), EVICT_EINVAL, "multiple"),
    (dict(prefix_batch=3), EVICT_EINVAL, "divide"), (dict(prefix_batch=0), EVICT_EINVAL, "divide"),
    (dict(n_prefix=-1), EVICT_EINVAL, "n_prefix"), (dict(prefix_k=None), EVICT_EINVAL, "NULL"),
    (dict(prefix_v=A + 4), EVICT_EINVAL, "16-byte"), (dict(prefix_stride_h=100), EVICT_EINVAL, "multiples"),
    (dict(prefix_stride_b=-8), EVICT_EINVAL, "multiples"),
    (dict(q=rows(None, heads=8)), EVICT_EINVAL, "NULL"), (dict(q=rows(A, heads=4)), EVICT_EINVAL, "heads"),
    (dict(q=rows(A + 8, heads=8)), EVICT_EINVAL, "16 bytes"), (dict(out=rows(A, heads=8, stride_m=132)), EVICT_EINVAL, "16 bytes"),
    (dict(scale=math.nan), EVICT_EINVAL, "scale"), (dict(lse=A + 2), EVICT_EINVAL, "4-byte"),
    (dict(batch=5000, prefix_batch=1), EVICT_ELIMIT, "4096"),
    (dict(batch=4096, m=1 << 16), EVICT_ELIMIT, "2\\^30"),
    (dict(pages=pages(dtype=EVICT_FP32)), EVICT_EINVAL, "bf16"), (dict(pages=pages(n_kv_heads=2)), EVICT_EINVAL, "KV heads"),
])
def test_bad_attention_calls_are_refused(lib, kw, code, match):
    refused(code, match, binding.evict_shared_attention, attention(**kw))


def test_attention_of_nothing_is_no_launch(lib):
    before = lib.evict_launch_count()
    binding.evict_shared_attention(attention(batch=0))
    binding.evict_shared_attention(attention(m=0))
    assert lib.evict_launch_count() == before
    assert lib.evict_shared_attention(None) == EVICT_EINVAL
    assert lib.evict_shared_attention_workspace(None, None) == EVICT_EINVAL


@pytest.mark.parametrize("kw", [dict(), dict(n_pages=4), dict(n_pages=4, page_size=16, n_kv_heads=2, batch=0, max_rows=9),
                                dict(n_pages=4, page_size=20, n_kv_heads=2, batch=1, max_rows=9),
                                dict(k_pages=object())])
def test_bad_caches_are_refused(kw):
    with pytest.raises(ValueError):
        paged.PagedCache(**kw)


def test_host_tensors_are_refused(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 2, 3, 128)
    with pytest.raises(ValueError, match="CUDA"):
        paged.rotate(paged.Rotary(), x)
    with pytest.raises(ValueError, match="CUDA"):
        paged.shared_attention(x.bfloat16(), prefix=(x, x))


# --- strides that the C structs cannot say -------------------------------------------------------
def test_shared_table_rows_and_pages_on_top_of_each_other_are_refused():
    torch = pytest.importorskip("torch")
    pool = torch.zeros(6, 2, 16, 128, dtype=torch.bfloat16)
    table = torch.zeros(3, 4, dtype=torch.int32)
    assert paged._page_strides(pool, table) == (2 * 16 * 128, 4)
    assert paged._page_strides(pool[::2], table[:, :3]) == (2 * 2 * 16 * 128, 4)
    # a stride of 0 is what the structs hold for "dense": it must never come from a tensor
    with pytest.raises(ValueError, match="table"):
        paged._page_strides(pool, table[:1].expand(3, 4))
    with pytest.raises(ValueError, match="table"):
        paged._page_strides(pool, torch.zeros(12, dtype=torch.int32).as_strided((3, 4), (2, 1)))
    with pytest.raises(ValueError, match="pages"):
        paged._page_strides(pool[:1].expand(6, 2, 16, 128), table)
    with pytest.raises(ValueError, match="pages"):
        paged._page_strides(pool.flatten().as_strided((3, 2, 16, 128), (2048, 2048, 128, 1)), table)
    # one page, one sequence: nothing is stepped over, whatever the strides say
    assert paged._page_strides(pool[:1].as_strided((1, 2, 16, 128), (8, 2048, 128, 1)), table[:1].as_strided((1, 4), (1, 1))) == (0, 0)


def test_a_handles_stream_needs_a_handle(lib):
    out = ctypes.c_void_p(7)
    assert lib.evict_get_stream(None, ctypes.byref(out)) == EVICT_EINVAL and out.value == 7


def sized(heads, b, h, m, data=2 * A):
    return EvictRows(data, b, h, m, heads)


OVERLAPPING = [sized(4, 4096, 0, 128), sized(4, 0, 1024, 128), sized(4, 4096, 1024, 0), sized(4, 4096, 1024, 64),
               sized(4, 4096, 512, 128), sized(4, 2048, 1024, 128), sized(4, -4096, 1024, -64), sized(4, 1024, 4096, 512),
               sized(2, 128, 256, 384)]
# as [2, heads, 8, 128]: token-major, heads within a wider tensor, backwards, and two interleaved by hand
APART = [sized(4, 4096, 1024, 128), sized(4, 4096, 128, 512), sized(4, 8 * 7 * 128, 128, 7 * 128), sized(4, -4096, -1024, -128),
         sized(2, 128, 2048, 256), sized(3, 384, 3072, 1 << 40), sized(1, 128, 0, 256), sized(1, 128, 7, 256)]


@pytest.mark.parametrize("x", OVERLAPPING + APART, ids=lambda x: f"{x.heads}-{x.stride_b}-{x.stride_h}-{x.stride_m}")
def test_overlapping_layouts_are_told_from_others(x):
    # what the refusals below go by, against the addresses themselves
    seen = set()
    for b in range(2):
        for h in range(x.heads):
            for t in range(8):
                at = b * x.stride_b + h * x.stride_h + t * x.stride_m
                seen.add(at)
    rows_at = sorted(seen)
    overlap = len(rows_at) < 16 * x.heads or any(b - a < 128 for a, b in zip(rows_at, rows_at[1:]))
    assert overlap == (x in OVERLAPPING)


@pytest.mark.parametrize("out", OVERLAPPING, ids=lambda x: f"{x.heads}-{x.stride_b}-{x.stride_h}-{x.stride_m}")
def test_outputs_on_top_of_each_other_are_refused(rot, out):
    n = out.heads
    refused(EVICT_EINVAL, "on top", binding.evict_rotate, rot.handle, EVICT_BF16, 2, 8, None, 0, 0, rows(heads=n), out, 1, None)
    same = EvictRows(A, out.stride_b, out.stride_h, out.stride_m, n)      # in place
    refused(EVICT_EINVAL, "on top", binding.evict_rotate, rot.handle, EVICT_FP32, 2, 8, None, 0, 0, same, same, 1, None)
    refused(EVICT_EINVAL, "on top", binding.evict_paged_append, pages(), 2, 8, None, rot.handle, None, 0, rows(5 * A),
            rows(6 * A), rows(heads=n), out, None)
    if min(out.stride_b, out.stride_h, out.stride_m) >= 0:
        refused(EVICT_EINVAL, "on top", binding.evict_shared_attention,
                attention(batch=2, m=8, n_q_heads=n, n_kv_heads=n // 2, q=rows(heads=n), out=out))


@pytest.mark.parametrize("out", APART, ids=lambda x: f"{x.heads}-{x.stride_b}-{x.stride_h}-{x.stride_m}")
def test_other_outputs_get_further(rot, out):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("made-up addresses would reach a GPU")
    with pytest.raises(binding.EvictError) as e:
        binding.evict_rotate(rot.handle, EVICT_BF16, 2, 8, None, 0, 0, rows(heads=out.heads), out, 1, None)
    assert e.value.code == binding.EVICT_ECUDA                            # there is no GPU to launch on


def test_results_on_top_of_the_queries_are_refused(lib):
    q = rows(A, heads=8, stride_b=8192)
    refused(EVICT_EINVAL, "must not be q", binding.evict_shared_attention, attention(q=q, out=q))


BIG = 0x7fffffff


@pytest.mark.parametrize("batch,m,heads,n", [(BIG, BIG, 4, 1), (1 << 16, 1 << 15, 1, 1), (1 << 30, 1 << 30, 16, 1),
                                             (1, 1, BIG, 2), (2, 1, 1 << 30, 1), (1, 1, 1 << 30, 2)])
def test_sizes_whose_product_wraps_are_refused(rot, batch, m, heads, n):
    x = (EvictRows * 2)(*[EvictRows(A, 0, 0, 0, heads)] * 2)
    out = (EvictRows * 2)(*[EvictRows(2 * A, 128, 128, 128, heads)] * 2)
    refused(EVICT_ELIMIT, "2\\^31", binding.evict_rotate, rot.handle, EVICT_BF16, batch, m, None, 0, 0, x, out, n, None)
    one, q = EvictRows(A, 0, 0, 0, 4), EvictRows(A, 0, 0, 0, heads if n == 1 else BIG - 7)
    refused(EVICT_ELIMIT, "2\\^31", binding.evict_paged_append, pages(), batch, m, None, rot.handle, None, 0, one, one, q,
            EvictRows(2 * A, 0, 128, 0, q.heads), None)


def test_tensors_that_require_a_gradient_are_refused(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 2, 3, 128)
    w = x.clone().requires_grad_()
    rot, h = paged.Rotary(), w.bfloat16()
    cache = paged.PagedCache.__new__(paged.PagedCache)      # refused before anything of it is looked at
    for call in (lambda a, b: paged.rotate(rot, a), lambda a, b: paged.rotate(rot, (b, a)),
                 lambda a, b: paged.rotate(rot, b, out=a), lambda a, b: paged.shared_attention(a, prefix=(b, b)),
                 lambda a, b: paged.shared_attention(b, prefix=(b, a)), lambda a, b: paged.shared_attention(b, prefix=(b, b), out=a),
                 lambda a, b: cache.append(a, b), lambda a, b: cache.append(b, a), lambda a, b: cache.append(b, b, q=a),
                 lambda a, b: cache.append(b, b, q=b, q_out=a),
                 lambda a, b: paged.PagedCache(k_pages=a, v_pages=b, table=b, lens=b)):
        for a, b in ((w, x), (h, x.bfloat16())):
            with pytest.raises(ValueError, match="gradient"):
                call(a, b)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        paged.rotate(rot, w)
    with pytest.raises(ValueError, match="CUDA"):
        paged.rotate(rot, w.detach())


@pytest.mark.parametrize("name", ["k_pages", "v_pages", "table", "lens"])
def test_a_caches_tensors_are_written_to_and_not_replaced(name):
    # the calls go by the addresses of the tensors that the cache was made of
    torch = pytest.importorskip("torch")
    cache = paged.PagedCache.__new__(paged.PagedCache)
    cache._tensors = tuple(torch.zeros(3, dtype=torch.int32) for _ in range(4))
    before = getattr(cache, name)
    with pytest.raises(AttributeError, match="in place"):
        setattr(cache, name, before + 1)
    cache.lens += 1
    cache.table[1] = 5
    assert getattr(cache, name) is before and cache.lens.tolist() == [1, 1, 1] and cache.table.tolist() == [0, 5, 0]


@pytest.mark.parametrize("kw", [dict(prefix_stride_b=0), dict(prefix_stride_h=0)])
def test_prefixes_in_one_place_are_refused(lib, kw):
    refused(EVICT_EINVAL, "in one place", binding.evict_shared_attention, attention(**kw))
