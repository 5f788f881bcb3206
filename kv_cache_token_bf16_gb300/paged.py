"""The steps around a kept cache: rotary positions, pages of a batch's own rows, attention.

An ``EvictCache`` takes keys that are already rotated and returns the rows to attend to. Here are
the calls on either side of it, as thin wrappers of the C calls of include/evict.h:

* ``Rotary`` and ``rotate``: rotary positions of one to four axes (time, height, width of a video's
  tokens), whole or partial heads, both pairings, forwards and transposed;
* ``PagedCache``: own rows of a batch's sequences in pages, appended with the rotation applied on
  the way, and the attention over them behind a prefix that the sequences share;
* ``shared_attention``: that attention on its own, e.g. over an ``EvictCache``'s kept rows.

A decode step behind a shared prompt that an ``EvictCache`` of batch 1 has absorbed::

    rotary = paged.Rotary(base=500000.0)
    own = paged.PagedCache(n_pages=4096, page_size=16, n_kv_heads=8, batch=32, max_rows=2048)
    ...
    own.grow(1)                                              # a row more for every sequence
    own.append(k, v, rotary=rotary, pos_base=prompt.stats()["offset"], q=q, q_out=q)
    out = own.attend(q, prefix=prompt.view()[:2])

Work goes on the current stream of the tensors' device; nothing but ``PagedCache.sync`` waits for it
(``grow`` and ``release`` copy from pinned memory, which torch has to make the first times). Tensors are
[batch, heads, m, 128] with any strides whose innermost is 1, so a projection's
[batch, m, heads, 128] is passed as ``x.transpose(1, 2)``. The calls are not part of autograd:
tensors that require a gradient are refused while gradients are recorded (the gradient of ``rotate``
is ``rotate(..., transpose=True)``).
"""
from __future__ import annotations

import ctypes
import struct

from . import binding
from .binding import EVICT_BF16, EVICT_FP32, HEAD_DIM, EvictAttention, EvictPages, EvictRotaryConfig, EvictRows

PAGE_SIZES = (16, 32, 64, 128, 256)

# A decode step calls these functions for every layer, in tens of microseconds in all: the argument
# structs are packed in one call each instead of field by field (evict_rows; evict_attention).
_ROWS = struct.Struct("=Qqqqi4x")
_ATTENTION = struct.Struct("=4i Qqqqi4x Qqqqi4x Q f4x QQ qq ii 6Q")
assert _ROWS.size == ctypes.sizeof(EvictRows) and _ATTENTION.size == ctypes.sizeof(EvictAttention)

_torch = None
_calls = None
_recording = None                                # torch.is_grad_enabled


def _load():
    """torch, and the library's calls with packed structs as arguments."""
    global _torch, _calls, _recording
    import torch
    _recording = torch.is_grad_enabled
    lib = binding.load()
    calls = ctypes.CDLL(lib._name)               # function objects of their own: other argument types
    p, i, q = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    packed = ctypes.c_char_p
    for name, args in (("evict_rotate", [p, i, i, i, p, q, i, packed, packed, i, p]),
                       ("evict_paged_append", [p, i, i, p, p, p, q, packed, packed, packed, packed, p]),
                       ("evict_shared_attention", [packed])):
        fn = getattr(calls, name)
        fn.restype, fn.argtypes = i, args
    _calls = calls                               # before _torch, which other threads take as the sign
    _torch = torch


def _dtype(t):
    if t is _torch.bfloat16:
        return EVICT_BF16
    if t is _torch.float32:
        return EVICT_FP32
    raise ValueError(f"bf16 or fp32 tensors only, not {t}")


def _device(t):
    """Index of a CUDA tensor's device."""
    index = t.get_device()
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    return index


def _no_history():
    """Of tensors that require a gradient, which would be lost without a word."""
    raise ValueError("no gradient is recorded for this call: make it under torch.no_grad(), or of detached tensors")


def _rows(t, name, index, dtype, batch, m, heads=None):
    """The fields of a tensor's evict_rows [batch, heads, m, 128]."""
    shape, strides = t.shape, t.stride()
    if len(shape) == 4 and strides[3] == 1:
        b, h, n, d = shape
        if d == HEAD_DIM and b == batch and n == m and t.dtype is dtype and t.get_device() == index and (
                heads is None or h == heads):
            return t.data_ptr(), strides[0], strides[1], strides[2], h
    if len(shape) != 4 or shape[3] != HEAD_DIM:
        raise ValueError(f"{name} must be [batch, heads, m, {HEAD_DIM}], not {tuple(shape)}")
    if shape[0] != batch or shape[2] != m or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} is {tuple(shape)}: batch, m or heads differ from the other tensors")
    if t.dtype is not dtype:
        raise ValueError(f"{name} is {t.dtype}, not {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on CUDA device {index}")
    raise ValueError(f"{name}: the 128 elements of a row must be adjacent")


def _new_rows(t):
    """The same of a tensor made here like one that was checked."""
    sb, sh, sm, se = t.stride()
    if se != 1:
        raise ValueError("no output can be made like this input: give one")
    return t.data_ptr(), sb, sh, sm, t.shape[1]


def _like(t, name, shape, dtype, index):
    """An int32 or fp32 side tensor: dense, of this shape, on this device. Its pointer (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on CUDA device {index}")
    return t.data_ptr()


def _stream(index):
    """The current stream of a device (as an integer)."""
    raw = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw else _torch.cuda.current_stream(index).cuda_stream


class _on:
    """Makes a device current for a call."""

    def __init__(self, index):
        self.guard = _torch.cuda.device(index)

    def __enter__(self):
        self.guard.__enter__()

    def __exit__(self, *e):
        self.guard.__exit__(*e)


def _call(index, fn, *args):
    """fn(*args) with the device current; raises the library's error."""
    if _torch.cuda.current_device() == index:
        code = fn(*args)
    else:
        with _on(index):
            code = fn(*args)
    if code:
        binding.check(code)


class Rotary:
    """The tables of a rotation (host memory; usable on any device and stream).

    Pair i of a row turns by pos[axis[i]] * inv_freq[i]. ``inv_freq`` defaults to
    base ** (-2 i / rotary_dim), rounded to fp32 as models hold it; ``axis`` names the position
    axis of every pair, or ``sections`` gives how many pairs in a row each axis has. ``pairs``:
    "half" pairs element i with i + rotary_dim / 2, "adjacent" 2 i with 2 i + 1. ``scale``
    multiplies cos and sin.
    """

    def __init__(self, rotary_dim: int = HEAD_DIM, base: float = 10000.0, inv_freq=None, axis=None, sections=None,
                 n_axes: int | None = None, pairs: str = "half", scale: float = 1.0):
        self.handle = None
        if pairs not in ("half", "adjacent"):
            raise ValueError('pairs must be "half" or "adjacent"')
        n = max(rotary_dim // 2, 0)
        if inv_freq is None:
            inv_freq = [ctypes.c_float(base ** (-2.0 * i / rotary_dim)).value for i in range(n)]
        inv_freq = [float(x) for x in inv_freq]
        if sections is not None:
            if axis is not None:
                raise ValueError("axis and sections exclude each other")
            axis = [a for a, count in enumerate(sections) for _ in range(count)]
        axis = [0] * n if axis is None else [int(a) for a in axis]
        if len(inv_freq) != n or len(axis) != n:
            raise ValueError(f"need {n} frequencies and axes, got {len(inv_freq)} and {len(axis)}")
        if any(not 0 <= a < 256 for a in axis):
            raise ValueError("axis must be >= 0")
        self.rotary_dim, self.pairs = rotary_dim, pairs
        self.n_axes = n_axes if n_axes is not None else (len(sections) if sections is not None else max(axis, default=0) + 1)
        cfg = EvictRotaryConfig(rotary_dim=rotary_dim, adjacent=int(pairs == "adjacent"), n_axes=self.n_axes, scale=scale,
                                inv_freq=(ctypes.c_double * max(n, 1))(*inv_freq), axis=(ctypes.c_uint8 * max(n, 1))(*axis))
        self.handle = binding.evict_rotary_init(cfg)

    def __del__(self):
        try:
            if self.handle:
                binding.evict_rotary_destroy(self.handle)
                self.handle = None
        except Exception:
            pass


def rotate(rotary: Rotary, x, pos=None, pos_base: int = 0, out=None, transpose: bool = False):
    """Rotate x [batch, heads, m, 128], or a pair of such tensors (queries and keys) in one launch.

    pos [n_axes, batch, m] int32 (with one axis also [batch, m]), or None: token t of every
    sequence is at pos_base + t. ``out`` (a tensor or pair; x itself rotates in place) defaults to
    new tensors with x's strides where they are dense. ``transpose`` turns by the negative angle:
    the gradient of the rotation, and with scale 1 its inverse.
    """
    if _torch is None:
        _load()
    one = isinstance(x, _torch.Tensor)
    xs = (x,) if one else tuple(x)
    outs = None if out is None else (out,) if isinstance(out, _torch.Tensor) else tuple(out)
    n = len(xs)
    if not 1 <= n <= 2 or (outs is not None and len(outs) != n):
        raise ValueError("one or two tensors, and as many outputs")
    if _recording():
        for t in xs + outs if outs else xs:
            if t.requires_grad:
                _no_history()
    first = xs[0]
    index, dtype, shape = _device(first), first.dtype, first.shape
    if len(shape) != 4:
        raise ValueError(f"x must be [batch, heads, m, {HEAD_DIM}], not {tuple(shape)}")
    batch, m = shape[0], shape[2]
    ins = b"".join([_ROWS.pack(*_rows(t, "x", index, dtype, batch, m)) for t in xs])
    if outs is None:
        outs = tuple([_torch.empty_like(t) for t in xs])
        ous = b"".join([_ROWS.pack(*_new_rows(o)) for o in outs])
    else:
        ous = b"".join([_ROWS.pack(*_rows(o, "out", index, dtype, batch, m, t.shape[1])) for t, o in zip(xs, outs)])
    _call(index, _calls.evict_rotate, rotary.handle, _dtype(dtype), batch, m, _pos(pos, rotary, batch, m, index), pos_base,
          1 if transpose else 0, ins, ous, n, _stream(index))
    return outs[0] if one else outs


def _pos(pos, rotary, batch, m, index):
    if pos is None:
        return None
    n_axes = rotary.n_axes if rotary is not None else 1
    shape = (batch, m) if n_axes == 1 and pos.dim() == 2 else (n_axes, batch, m)
    return _like(pos, "pos", shape, _torch.int32, index)


# Workspace bytes of a call's sizes, on a device (the sizes alone decide).
_workspace = {}


def _workspace_bytes(key, args):
    if len(_workspace) >= 4096:
        _workspace.clear()
    with _on(key[0]):
        n = binding.evict_shared_attention_workspace(EvictAttention.from_buffer_copy(args))
    _workspace[key] = n
    return n


def shared_attention(q, prefix=None, pages: "PagedCache | None" = None, n_new=None, scale=None, out=None, lse=None):
    """Attention of q [batch, n_q_heads, m, 128] (bf16) over a shared prefix and own pages.

    prefix: (K, V) [prefix_batch, n_kv_heads, n, 128], e.g. ``EvictCache.view()[:2]``; prefix p
    serves the batch / prefix_batch sequences from p * (batch / prefix_batch) on (one that is expanded
    over its first axis is read once for all). pages: a PagedCache whose lens count the m (or n_new[b])
    query tokens' own rows, which they see up to their own. ``out`` must not overlap an input (not even
    q). Padding queries (t >= n_new[b]) leave their rows of ``out`` and ``lse`` as they are; a new
    ``out`` has zeros there. lse: fp32 [batch, n_q_heads, m] for the log-sum-exp. Returns out.
    """
    if _torch is None:
        _load()
    k, v = prefix if prefix is not None else (None, None)
    if _recording() and (q.requires_grad or (out is not None and out.requires_grad) or
                         (k is not None and (k.requires_grad or v.requires_grad))):
        _no_history()
    index, shape = _device(q), q.shape
    if len(shape) != 4:
        raise ValueError(f"q must be [batch, heads, m, {HEAD_DIM}], not {tuple(shape)}")
    batch, hq, m, _ = shape
    bf16 = _torch.bfloat16
    qr = _rows(q, "q", index, bf16, batch, m)
    if out is None:
        out = _torch.empty_like(q) if n_new is None else _torch.zeros_like(q)
        outr = _new_rows(out)
    else:
        outr = _rows(out, "out", index, bf16, batch, m, hq)
    if scale is None:
        scale = 0.0
    elif scale == 0:
        raise ValueError("scale must not be 0")
    hkv = pages_at = error = width = page = 0
    if pages is not None:
        if pages.batch != batch or pages.index != index:
            raise ValueError(f"the pages are for {pages.batch} sequences on {pages.device}")
        hkv, pages_at, error, width, page = pages.n_kv_heads, pages.address, pages.error_at, pages.width, pages.page_size
    pk = pv = sb = sh = n = groups = 0
    if prefix is not None:
        ks = k.shape
        if k.dtype is not bf16 or v.dtype is not bf16 or len(ks) != 4 or ks[3] != HEAD_DIM or ks != v.shape:
            raise ValueError(f"the prefix must be two bf16 tensors [prefix_batch, n_kv_heads, n, {HEAD_DIM}]")
        if k.get_device() != index or v.get_device() != index:
            raise ValueError(f"the prefix is not on CUDA device {index}")
        if hkv and ks[1] != hkv:
            raise ValueError(f"the prefix has {ks[1]} KV heads, the pages {hkv}")
        hkv = ks[1]
        if ks[2] > 0:
            groups, n = ks[0], ks[2]
            strides = k.stride()
            sb, sh, sn, se = strides
            if v.stride() != strides or se != 1 or (sn != HEAD_DIM and n > 1):
                raise ValueError("the prefix's rows must be adjacent, K and V with the same strides")
            if sb == 0 and batch % groups == 0:  # expanded: one prefix for all, read once
                groups = 1
            if sh == 0 and hkv > 1:              # expanded: one KV head for all query heads
                if pages is not None:
                    raise ValueError("the prefix's heads lie in one place, the pages' do not: repeat them")
                hkv, sh = 1, n * HEAD_DIM
            pk, pv = k.data_ptr(), v.data_ptr()
    if hkv == 0:
        raise ValueError("neither a prefix nor pages: nothing to attend to")
    lse_at = _like(lse, "lse", (batch, hq, m), _torch.float32, index)
    new_at = _like(n_new, "n_new", (batch,), _torch.int32, index)
    head = (batch, m, hq, hkv, *qr, *outr, lse_at, scale, pk, pv, sb, sh, n, groups, pages_at, new_at)
    key = (index, batch, m, hq, hkv, n, groups, width, page)
    size = _workspace.get(key)
    if size is None:
        size = _workspace_bytes(key, _ATTENTION.pack(*head, 0, 0, 0, 0))
    # from torch's allocator: reused in stream order, private to a graph that is being captured
    work = _torch.empty(size, dtype=_torch.uint8, device=q.device)
    _call(index, _calls.evict_shared_attention, _ATTENTION.pack(*head, work.data_ptr(), size, error, _stream(index)))
    return out


def _page_strides(k_pages, table):
    """Elements between pages, and between the table's rows, for evict_pages (0: dense, which is what a
    single page or row is given as). Pages or rows of the table on top of each other are refused."""
    n_pages, heads, page, _ = k_pages.shape
    batch, width = table.shape
    ps, ts = k_pages.stride(0) if n_pages > 1 else 0, table.stride(0) if batch > 1 else 0
    if n_pages > 1 and ps < heads * page * HEAD_DIM:
        raise ValueError(f"pages of {heads * page * HEAD_DIM} elements are {ps} apart: they would lie on top of each other")
    if batch > 1 and ts < width:
        raise ValueError(f"the table's rows of {width} entries are {ts} apart: give every sequence a row of its own")
    return ps, ts


def _kept(i):
    """A property: one of a cache's tensors."""
    def same(self, value):
        if value is not self._tensors[i]:
            raise AttributeError("the cache holds this tensor's address: write to it in place")
    return property(lambda self: self._tensors[i], same)


class PagedCache:
    """Own rows of a batch of sequences, in pages of a pool.

    Either ``PagedCache(n_pages=, page_size=, n_kv_heads=, batch=, max_rows=, dtype=)`` makes the
    tensors (zeros, no rows), and ``grow`` / ``release`` hand out the pages; or the caller brings
    ``k_pages``, ``v_pages`` [n_pages, n_kv_heads, page_size, 128] (a page's rows dense, pages any
    stride apart), ``table`` [batch, width] int32 (a row of its own for every sequence, also where
    they name the same pages) and ``lens`` [batch] int32, and keeps the last two up to date in place:
    row j of sequence b is row j % page_size of page table[b, j // page_size], and lens counts a
    call's new rows before the call.
    """

    def __init__(self, n_pages: int | None = None, page_size: int | None = None, n_kv_heads: int | None = None,
                 batch: int | None = None, max_rows: int | None = None, dtype: str = "bf16", device=None,
                 k_pages=None, v_pages=None, table=None, lens=None):
        if _torch is None:
            _load()
        torch = _torch
        given = [x is not None for x in (k_pages, v_pages, table, lens)]
        if any(given) and not all(given):
            raise ValueError("k_pages, v_pages, table and lens go together")
        if _recording() and any(given) and (k_pages.requires_grad or v_pages.requires_grad):
            _no_history()
        self._free = self._rows = None
        if not any(given):
            if min(n_pages or 0, page_size or 0, n_kv_heads or 0, batch or 0, max_rows or 0) < 1:
                raise ValueError("n_pages, page_size, n_kv_heads, batch and max_rows must be >= 1")
            if page_size not in PAGE_SIZES:
                raise ValueError(f"page_size must be one of {PAGE_SIZES}")
            t = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
            device = torch.device("cuda" if device is None else device)
            k_pages = torch.zeros(n_pages, n_kv_heads, page_size, HEAD_DIM, dtype=t, device=device)
            v_pages = torch.zeros_like(k_pages)
            table = torch.zeros(batch, -(-max_rows // page_size), dtype=torch.int32, device=device)
            lens = torch.zeros(batch, dtype=torch.int32, device=device)
            self._free = list(range(n_pages - 1, -1, -1))
            self._rows, self._pages = [0] * batch, [[] for _ in range(batch)]
        self.index, self.device = _device(k_pages), k_pages.device
        if v_pages.device != self.device or table.device != self.device:
            raise ValueError("pages, table and lens must be on one device")
        if k_pages.dim() != 4 or k_pages.shape[3] != HEAD_DIM or v_pages.shape != k_pages.shape or \
                v_pages.dtype != k_pages.dtype or v_pages.stride() != k_pages.stride():
            raise ValueError(f"pages must be two tensors [n_pages, n_kv_heads, page_size, {HEAD_DIM}] alike")
        self.n_pages, self.n_kv_heads, self.page_size, _ = k_pages.shape
        _, sh, sr, se = k_pages.stride()
        if (sh, sr, se) != (self.page_size * HEAD_DIM, HEAD_DIM, 1) and self.n_pages * self.n_kv_heads > 0:
            raise ValueError("the rows of a page must be dense")
        if table.dim() != 2 or table.dtype != torch.int32 or table.stride(1) != 1:
            raise ValueError("table must be int32 [batch, width] with adjacent entries")
        self.batch, self.width = table.shape
        page_stride, table_stride = _page_strides(k_pages, table)
        _like(lens, "lens", (self.batch,), torch.int32, self.index)
        self._tensors = k_pages, v_pages, table, lens
        self.error = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.struct = EvictPages(k=k_pages.data_ptr(), v=v_pages.data_ptr(), page_stride=page_stride, n_pages=self.n_pages,
                                 page_size=self.page_size, n_kv_heads=self.n_kv_heads, dtype=_dtype(k_pages.dtype),
                                 table=table.data_ptr(), table_stride=table_stride, table_width=self.width,
                                 lens=lens.data_ptr(), error=self.error.data_ptr())
        self.address, self.error_at = ctypes.addressof(self.struct), self.error.data_ptr()

    # The calls hold these tensors' addresses: they can be written to (``cache.lens += 1``), not replaced.
    k_pages, v_pages, table, lens = (_kept(i) for i in range(4))

    # --- pages ------------------------------------------------------------------------------
    def _managed(self):
        if self._free is None:
            raise ValueError("the caller keeps this cache's table and lens")

    def _changes(self):
        """Before grow and release: a graph would replay today's lengths and pages for ever."""
        self._managed()
        with _on(self.index):
            if _torch.cuda.is_current_stream_capturing():
                raise ValueError("grow and release belong between replays: they cannot be captured")

    def _upload(self, taken):
        """All lens, and the pages `taken` [(place in the table, page)], to the device in stream order.
        From pinned memory, which torch hands out again once the copies are through: no wait."""
        torch = _torch
        with _on(self.index):
            self.lens.copy_(torch.tensor(self._rows, dtype=torch.int32, pin_memory=True), non_blocking=True)
            if taken:
                places, pages = torch.tensor(taken, dtype=torch.int64, pin_memory=True).to(self.device, non_blocking=True).T
                self.table.view(-1).scatter_(0, places, pages.to(torch.int32))

    def grow(self, n_new):
        """Count n_new (a number, or one for every sequence) new rows in, taking pages for them.
        Raises ValueError, with nothing changed, where the pool or the table has no room."""
        self._changes()
        new = [int(n_new)] * self.batch if isinstance(n_new, int) else [int(n) for n in n_new]
        if len(new) != self.batch or min(new, default=0) < 0:
            raise ValueError("n_new must be one number >= 0 for every sequence")
        need = [-(-(r + n) // self.page_size) - len(p) for r, n, p in zip(self._rows, new, self._pages)]
        if any(len(p) + x > self.table.shape[1] for p, x in zip(self._pages, need)):
            raise ValueError(f"a sequence would have more than {self.table.shape[1]} pages")
        if sum(need) > len(self._free):
            raise ValueError(f"{sum(need)} pages needed, {len(self._free)} free")
        taken = []
        for b, x in enumerate(need):
            for _ in range(x):
                taken.append((b * self.width + len(self._pages[b]), self._free[-1]))
                self._pages[b].append(self._free.pop())
            self._rows[b] += new[b]
        self._upload(taken)

    def release(self, b: int):
        """Sequence b ends: its pages are free and it has no rows."""
        self._changes()
        self._free += reversed(self._pages[b])
        self._pages[b], self._rows[b] = [], 0
        self._upload([])

    def rows(self):
        """Rows of every sequence, as grow and release count them."""
        self._managed()
        return list(self._rows)

    # --- calls ------------------------------------------------------------------------------
    def append(self, k, v, rotary: Rotary | None = None, pos=None, pos_base: int = 0, n_new=None, q=None, q_out=None):
        """Append k, v [batch, n_kv_heads, m, 128] (the last n_new[b], or m, of lens' rows).

        With ``rotary``, keys turn by pos ([n_axes, batch, m] int32) or by pos_base + their row's
        index in the sequence; values are copied. q [batch, n_q_heads, m, 128] is rotated alike
        in the same launch, into q_out (q itself: in place; None: a new tensor). Returns q_out.
        """
        if _recording() and (k.requires_grad or v.requires_grad or (q is not None and q.requires_grad) or
                             (q_out is not None and q_out.requires_grad)):
            _no_history()
        index, dtype, batch = self.index, self.k_pages.dtype, self.batch
        shape = k.shape
        m = shape[2] if len(shape) == 4 else -1
        kr, vr = _ROWS.pack(*_rows(k, "k", index, dtype, batch, m)), _ROWS.pack(*_rows(v, "v", index, dtype, batch, m))
        qr = qo = None
        if q is not None:
            qr = _ROWS.pack(*_rows(q, "q", index, dtype, batch, m))
            if q_out is None:
                q_out = _torch.empty_like(q) if n_new is None else _torch.zeros_like(q)
            qo = _ROWS.pack(*_rows(q_out, "q_out", index, dtype, batch, m, q.shape[1]))
        elif q_out is not None:
            raise ValueError("q_out without q")
        _call(index, _calls.evict_paged_append, self.address, batch, m, _like(n_new, "n_new", (batch,), _torch.int32, index) or None,
              rotary.handle if rotary is not None else None, _pos(pos, rotary, batch, m, index), pos_base, kr, vr, qr, qo,
              _stream(index))
        return q_out

    def attend(self, q, prefix=None, n_new=None, scale=None, out=None, lse=None):
        """shared_attention of q over ``prefix`` and these pages."""
        return shared_attention(q, prefix=prefix, pages=self, n_new=n_new, scale=scale, out=out, lse=lse)

    def sync(self):
        """Synchronise the current stream; raises EvictError(EVICT_EDEVICE) if a call's kernel has
        reported an error (a table entry outside the pool, rows outside the table) since the last."""
        with _on(self.index):
            binding.evict_pages_status(self.error_at, _stream(self.index))
