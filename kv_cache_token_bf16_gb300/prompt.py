"""Whole prompts before a cache: their causal attention, and the weights that it puts on every key.

The scores of an ``EvictCache`` of method "attention" are the softmax weights that queries put on a
row. For a prompt they come from here, as thin wrappers of the C calls of include/evict.h::

    lse = torch.empty(1, n_q_heads, tokens, device="cuda")
    out = prompt.attention(q, k, v, packing, lse=lse)      # [1, n_q_heads, tokens, 128]
    score = prompt.weights(q, k, lse, packing, last=64)    # [1, n_kv_heads, tokens]: what its last queries look at
    cache.update_and_fetch(k, v, score=score)              # one sequence's rows: the heaviest stay

and for every step behind it from ``EvictCache.attend(q, weigh=True)``, or ``EvictCache.weigh`` with the
log-sum-exps of an attention over these rows and others.

Tensors are [batch, heads, m, 128] bf16 with any strides whose innermost is 1, so a projection's
[batch, m, heads, 128] is passed as ``x.transpose(1, 2)``. Without a ``Packing`` every batch row is a
sequence of m tokens; with one, batch is 1 and the sequences lie behind each other. Work goes on the
current stream of the tensors' device; nothing but ``Packing.sync`` waits for it. The calls are not part
of autograd: tensors that require a gradient are refused while gradients are recorded.
"""
from __future__ import annotations

import ctypes
import struct

from . import binding
from . import paged
from .binding import HEAD_DIM, EvictPrompt

_PROMPT = struct.Struct("=2i Qqqqi4x Qqqqi4x Qqqqi4x Qqqqi4x QQQ iif4x QQ QQ")
assert _PROMPT.size == ctypes.sizeof(EvictPrompt)
_NO_ROWS = (0, 0, 0, 0, 0)

_calls = _alloc = _free = None


def _load():
    """The library's calls with packed structs as arguments."""
    global _calls, _alloc, _free
    if paged._torch is None:
        paged._load()
    _alloc = paged._torch._C._cuda_cudaCachingAllocator_raw_alloc
    _free = paged._torch._C._cuda_cudaCachingAllocator_raw_delete
    lib = ctypes.CDLL(binding.load()._name)      # function objects of their own: other argument types
    calls = {}
    for name in ("evict_prompt_attention", "evict_prompt_weights"):
        calls[name] = fn = getattr(lib, name)
        fn.restype, fn.argtypes = ctypes.c_int, [ctypes.c_char_p]
    _calls = calls


class Packing:
    """Where the sequences of a packed batch begin: ``starts`` [n + 1] int32 on the GPU, sequence i being
    the tokens starts[i] .. starts[i + 1] - 1 (some may be empty). Calls read them on the device, so a
    captured call follows what is written there in place; tokens before the first and behind the last
    sequence are left alone."""

    def __init__(self, starts):
        if paged._torch is None:
            paged._load()
        torch = paged._torch
        if starts.dim() != 1 or starts.dtype != torch.int32 or not starts.is_contiguous() or starts.shape[0] < 1:
            raise ValueError("starts must be contiguous int32 [n + 1]")
        self.index, self.n = paged._device(starts), starts.shape[0] - 1
        self._starts, self.at = starts, starts.data_ptr()
        self.error = torch.zeros(1, dtype=torch.int32, device=starts.device)
        self.error_at = self.error.data_ptr()
        self._call = self.at, self.n, self.error_at

    @property
    def starts(self):
        """The tensor itself: the calls hold its address, so write to it in place."""
        return self._starts

    def sync(self):
        """Synchronise the current stream; raises EvictError(EVICT_EDEVICE) if a call's kernel has
        reported an error (starts that fall, or leave the tensors: the call wrote nothing) since the last."""
        with paged._on(self.index):
            binding.evict_pages_status(self.error_at, paged._stream(self.index))


# Workspace bytes of a call (0: attention, 1: weights) and its sizes on a device, which alone decide.
_workspace = {}


def _run(name, key, fields, error):
    """Make a call of these sizes with its workspace, which comes from torch's allocator: reused in stream order,
    private to a graph that is being captured. (Not as a tensor: making and dropping one takes 3 us, this 0.6.)"""
    index = key[1]
    if paged._torch._C._cuda_getDevice() != index:
        with paged._on(index):
            return _run(name, key, fields, error)
    size = _workspace.get(key)
    if size is None:
        if len(_workspace) >= 4096:
            _workspace.clear()
        size = getattr(binding, name + "_workspace")(EvictPrompt.from_buffer_copy(_PROMPT.pack(*fields, 0, 0, 0, 0)))
        _workspace[key] = size
    stream = paged._stream(index)
    at = _alloc(size, stream)
    try:
        code = _calls[name](_PROMPT.pack(*fields, at, size, error, stream))
    finally:
        _free(at)
    if code:
        binding.check(code)


def _sizes(q, k, packing, scale):
    """(device index, batch, query heads, KV heads, m, scale) of a call."""
    index, shape = paged._device(q), q.shape
    if len(shape) != 4 or len(k.shape) != 4:
        raise ValueError(f"q and k must be [batch, heads, m, {HEAD_DIM}], not {tuple(shape)} and {tuple(k.shape)}")
    batch, hq, m, _ = shape
    if packing is not None:
        if packing.index != index:
            raise ValueError(f"the packing is on {packing.starts.device}, q on {q.device}")
        if batch != 1:
            raise ValueError(f"packed sequences lie in a batch of 1, not of {batch}")
    return index, batch, hq, k.shape[1], m, paged._scale(scale)


def attention(q, k, v, packing: Packing | None = None, scale=None, out=None, lse=None):
    """Causal attention of q [batch, n_q_heads, m, 128] over k, v [batch, n_kv_heads, m, 128] (bf16,
    rotated): query t of a sequence sees its keys j <= t. ``out`` must not overlap an input; tokens of no
    sequence keep their rows of ``out`` and ``lse``, and have zeros in a new ``out``. lse: fp32 [batch,
    n_q_heads, m] for the log-sum-exp. Returns out."""
    if _calls is None:
        _load()
    torch = paged._torch
    if paged._recording() and (q.requires_grad or k.requires_grad or v.requires_grad or
                               (out is not None and out.requires_grad) or (lse is not None and lse.requires_grad)):
        paged._no_history()
    index, batch, hq, hkv, m, scale = _sizes(q, k, packing, scale)
    bf16 = torch.bfloat16
    qr = paged._rows(q, "q", index, bf16, batch, m)
    kr = paged._rows(k, "k", index, bf16, batch, m)
    vr = paged._rows(v, "v", index, bf16, batch, m, hkv)
    if out is None:
        out = torch.empty_like(q) if packing is None else torch.zeros_like(q)
        outr = paged._new_rows(out)
    else:
        outr = paged._rows(out, "out", index, bf16, batch, m, hq)
    lse_at = paged._like(lse, "lse", (batch, hq, m), torch.float32, index)
    starts, n, error = packing._call if packing is not None else (0, 0, 0)
    fields = (batch, m, *qr, *kr, *vr, *outr, lse_at, 0, starts, n, 0, scale)
    _run("evict_prompt_attention", (0, index, batch, hq, hkv, m, n, packing is None), fields, error)
    return out


def weights(q, k, lse, packing: Packing | None = None, last: int = 0, scale=None, out=None):
    """The weights that a prompt's queries put on each key: fp32 [batch, n_kv_heads, m], the sums of
    exp(scale * q . k - lse) over the KV head's query heads and the queries that see the key, or of them
    the ``last`` ones of every sequence (0: all). lse: as ``attention`` leaves it. ``out`` must not overlap
    an input; tokens of no sequence keep their values of it, and have zeros in a new one. Returns out."""
    if _calls is None:
        _load()
    torch = paged._torch
    if lse is None:
        raise ValueError("lse must be given")
    if paged._recording() and (q.requires_grad or k.requires_grad or lse.requires_grad or
                               (out is not None and out.requires_grad)):
        paged._no_history()
    index, batch, hq, hkv, m, scale = _sizes(q, k, packing, scale)
    if last < 0:
        raise ValueError(f"last must be >= 0, not {last}")
    qr = paged._rows(q, "q", index, torch.bfloat16, batch, m)
    kr = paged._rows(k, "k", index, torch.bfloat16, batch, m)
    lse_at = paged._like(lse, "lse", (batch, hq, m), torch.float32, index)
    if out is None:
        make = torch.empty if packing is None else torch.zeros
        out = make(batch, hkv, m, dtype=torch.float32, device=q.device)
    out_at = paged._like(out, "out", (batch, hkv, m), torch.float32, index)
    starts, n, error = packing._call if packing is not None else (0, 0, 0)
    fields = (batch, m, *qr, *kr, *_NO_ROWS, *_NO_ROWS, lse_at, out_at, starts, n, min(last, m), scale)
    _run("evict_prompt_weights", (1, index, batch, hq, hkv, m, n, packing is None), fields, error)
    return out
