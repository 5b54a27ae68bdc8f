"""Paged KV cache of the binding: per-head norm and rotation of new rows, their
append to the cache, and attention over it (include/fkv.h, "Paged cache").

A :class:`Rope` and a :class:`PagedCache` are made once per model layer: they
check the tensors that stay (weights, frequencies, caches, page table) and keep
them alive.  The calls check and marshal the tensors of one step; a decoding
step is short enough for that to count, so they pack the C structs as bytes.
Every tensor of a call lives on the cache's device; the call runs there, on
`stream` or on that device's current stream, whatever device is current.

Nothing here is differentiable: these are serving operators, as the rest of
the library.  Tensors used on another stream than the one they were allocated
on are the caller's to keep alive (``Tensor.record_stream``).
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import Optional, Sequence

import torch

from . import _lib

_DTYPES = {torch.bfloat16: _lib.FKV_DTYPE_BF16, torch.float32: _lib.FKV_DTYPE_FP32}
# What torch.cuda.current_stream(index).cuda_stream and torch.cuda.current_device()
# return, without the objects in between.
_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_pack_rows = struct.Struct("=Qqq").pack     # fkv_rows_t
_pack_batch = struct.Struct("=QQQ").pack    # kv_len, cu_q, prefix_len of fkv_paged_t
_pack_places = struct.Struct("=Qq").pack    # positions, axis_stride of fkv_rope_t


def _call(name: str, index: int, stream, *args):
    """One library call on device `index`; its last argument is the stream."""
    if stream is None:
        handle = _current_stream(index)
    elif isinstance(stream, torch.cuda.Stream):
        if stream.device_index != index:
            raise ValueError(f"stream is on device {stream.device_index}, the call on device {index}")
        handle = stream.cuda_stream
    else:
        handle = int(stream)
    fn = getattr(_lib.load(), name)
    if index == _current_device():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            status = fn(*args, handle)
    if status != _lib.FKV_OK:
        from . import FkvError
        raise FkvError(status, name)


def _vector(t: Optional[torch.Tensor], name: str, dtype, numel: int, index: int,
            optional: bool = False) -> int:
    """Data pointer of a contiguous vector of at least numel entries; 0 for None."""
    if t is None:
        if optional:
            return 0
        raise ValueError(f"{name} is required")
    if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous() or t.numel() < numel:
        raise ValueError(f"{name} must be contiguous {dtype} with at least {numel} elements on "
                         f"device {index}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, shape, dtype, index: int) -> bytes:
    """fkv_rows_t of a [tokens, heads, D] tensor whose last dimension is contiguous."""
    if t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must be {dtype} on device {index}, got {t.dtype} on {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    ts, hs, ds = t.stride()
    if ds != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return _pack_rows(t.data_ptr(), ts, hs)


class Rope:
    """Norm and rotation of query and key rows (fkv_rope_t); see :func:`make_rope`."""

    def __init__(self, omega, axis_pairs, style, norm, eps, q_weight, k_weight):
        self.omega, self.q_weight, self.k_weight = omega, q_weight, k_weight
        self.axis_pairs = tuple(int(n) for n in axis_pairs)
        if not 1 <= len(self.axis_pairs) <= 3:
            raise ValueError("axis_pairs has one to three entries")
        self._axes, self._pairs = len(self.axis_pairs), sum(self.axis_pairs)
        tensors = [t for t in (omega, q_weight, k_weight) if t is not None]
        self._index = tensors[0].get_device() if tensors else None
        if self._index is not None and self._index < 0:
            raise ValueError("omega and the weights must be CUDA tensors")
        sizes = {t.numel() for t in (q_weight, k_weight) if t is not None}
        if len(sizes) > 1:
            raise ValueError(f"the weights have {sorted(sizes)} entries: one head size is wanted")
        self._dims = sizes.pop() if sizes else None  # of the rows that the weights are for
        c = _lib.Rope()
        c.style = {"interleaved": _lib.FKV_ROPE_ADJACENT, "half": _lib.FKV_ROPE_HALF}[style]
        c.norm = 1 if norm else 0
        c.n_axes = self._axes
        for i, m in enumerate(self.axis_pairs):
            c.axis_pairs[i] = m
        c.eps = eps
        for name in ("omega", "q_weight", "k_weight"):
            setattr(c, name, _vector(getattr(self, name), name, torch.float32,
                                     self._pairs if name == "omega" else 1, self._index,
                                     optional=name != "omega" or self._pairs == 0) or None)
        self._head = bytes(c)[:_lib.Rope.positions.offset]

    def _struct(self, head_dim: int, positions, tokens: int, index: int,
                cache_positions: bool = False) -> bytes:
        """fkv_rope_t of one call."""
        if self._index is not None and self._index != index:
            raise ValueError(f"the rope's tensors are on device {self._index}, the rows on {index}")
        if self._dims is not None and self._dims != head_dim:
            raise ValueError(f"the weights have {self._dims} entries, the rows {head_dim} dims")
        if positions is None:
            if self._pairs > 0 and not (cache_positions and self._axes == 1):
                raise ValueError("positions is required")
            return self._head + _pack_places(0, 0)
        shape = tuple(positions.shape)
        if shape != (self._axes, tokens) and not (self._axes == 1 and shape == (tokens,)):
            raise ValueError(f"positions must have the shape ({self._axes}, {tokens}), got {shape}")
        return self._head + _pack_places(
            _vector(positions, "positions", torch.int32, self._axes * tokens, index), tokens)


def make_rope(omega: Optional[torch.Tensor] = None, *, axis_pairs: Optional[Sequence[int]] = None,
              style: str = "interleaved", norm: bool = True, eps: float = 1e-6,
              q_weight: Optional[torch.Tensor] = None,
              k_weight: Optional[torch.Tensor] = None) -> Rope:
    """Norm and rotation of rows.  omega: float32 frequencies, one per rotated
    pair of dims (None: no rotation); style "interleaved" pairs dims (2i, 2i+1),
    "half" dims (i, i + n).  axis_pairs splits the pairs over up to three
    position axes (default: one axis).  norm: RMS norm of each head first, with
    eps and optional float32 weights [D]."""
    n = 0 if omega is None else int(omega.numel())
    if axis_pairs is None:
        axis_pairs = (n,)
    if sum(axis_pairs) != n or min(axis_pairs, default=0) < 0:
        raise ValueError(f"axis_pairs {tuple(axis_pairs)} do not split the {n} frequencies")
    return Rope(omega, axis_pairs, style, norm, eps, q_weight, k_weight)


def qk_norm_rope(rope: Rope, q: Optional[torch.Tensor], k: Optional[torch.Tensor],
                 positions: Optional[torch.Tensor], q_out: Optional[torch.Tensor],
                 k_out: Optional[torch.Tensor], stream=None):
    """Per-head norm and rotation of q [tokens, Hq, D] and k [tokens, Hkv, D]
    into q_out / k_out of the same shapes, any strides (fkv_qk_norm_rope), in
    one launch.  positions: int32 [axes, tokens].  q_out / k_out may be q / k.
    For the chunk step's head-major operands pass transposed views, such as
    ``q_cur[layer].transpose(0, 1)``.  Either of q and k may be None."""
    some = q if q is not None else k
    if some is None or (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("q with q_out, k with k_out, or both pairs are required")
    dt, index = some.dtype, some.get_device()
    if some.dim() != 3 or dt not in _DTYPES or index < 0:
        raise ValueError("rows are [tokens, heads, D] CUDA tensors in bfloat16 or float32")
    tokens, _, D = some.shape
    hq = hk = 0
    rq = rqo = rk = rko = None
    if q is not None:
        hq = q.shape[1]
        rq, rqo = _rows(q, "q", (tokens, hq, D), dt, index), _rows(q_out, "q_out", (tokens, hq, D), dt, index)
    if k is not None:
        hk = k.shape[1]
        rk, rko = _rows(k, "k", (tokens, hk, D), dt, index), _rows(k_out, "k_out", (tokens, hk, D), dt, index)
    _call("fkv_qk_norm_rope", index, stream, rope._struct(D, positions, tokens, index), _DTYPES[dt], D,
          tokens, hq, hk, rq, rk, rqo, rko)


class PagedCache:
    """A paged cache and how its queries read it (fkv_paged_t).

    k_cache, v_cache: [num_pages, Hkv, page_size, D], any strides with the last
    dimension contiguous, the same for both (a cache kept as [num_pages,
    page_size, Hkv, D] is passed as its ``transpose(1, 2)``).  page_table: int32
    [sequences, max_pages].  softcap, window, alibi_slopes and causal as in
    fkv_paged_t; scale defaults to 1 / sqrt(D).  The page table may be changed
    in place between calls; entries of pages that no query of a call sees (behind
    a window, say) may hold anything."""

    def __init__(self, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, *,
                 num_q_heads: int, scale: Optional[float] = None, softcap: float = 0.0,
                 window: int = 0, causal: bool = True,
                 alibi_slopes: Optional[torch.Tensor] = None):
        for name, n, least in (("num_q_heads", num_q_heads, 1), ("window", window, 0)):
            if not least <= n < 2 ** 31:  # a C int would keep the low 32 bits
                raise ValueError(f"{name} must lie in {least} .. 2^31 - 1, got {n}")
        if k_cache.dim() != 4 or k_cache.dtype not in _DTYPES:
            raise ValueError("k_cache must be [num_pages, Hkv, page_size, D] in bfloat16 or float32")
        if (v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype or
                v_cache.device != k_cache.device or v_cache.stride() != k_cache.stride()):
            raise ValueError("v_cache must have k_cache's shape, strides, type and device")
        if k_cache.stride(3) != 1:
            raise ValueError("the caches must be contiguous in their last dimension")
        dev = self.device = k_cache.device
        if dev.type != "cuda":
            raise ValueError("the caches must be CUDA tensors")
        if (page_table.dim() != 2 or page_table.dtype != torch.int32 or page_table.device != dev or
                (page_table.shape[1] > 1 and page_table.stride(1) != 1)):
            raise ValueError(f"page_table must be int32 [sequences, max_pages] on {dev}, rows contiguous")
        self.k_cache, self.v_cache, self.page_table = k_cache, v_cache, page_table
        self.alibi_slopes, self.dtype = alibi_slopes, k_cache.dtype
        self.num_q_heads, self.num_seqs = int(num_q_heads), page_table.shape[0]
        self.num_kv_heads, self.head_dim = k_cache.shape[1], k_cache.shape[3]
        self._index = k_cache.get_device()
        c = _lib.Paged()
        c.dtype = _DTYPES[self.dtype]
        c.flags = _lib.FKV_PAGED_CAUSAL if causal else 0
        c.head_dim, c.num_q_heads, c.num_kv_heads = self.head_dim, self.num_q_heads, self.num_kv_heads
        c.page_size, c.num_pages = k_cache.shape[2], k_cache.shape[0]
        c.num_seqs, c.max_pages = page_table.shape
        c.window, c.softcap = int(window), softcap
        c.scale = 1.0 / math.sqrt(self.head_dim) if scale is None else scale
        c.page_stride, c.head_stride, c.row_stride = k_cache.stride()[:3]
        c.table_stride = page_table.stride(0)
        c.k_cache, c.v_cache = k_cache.data_ptr(), v_cache.data_ptr()
        c.page_table = page_table.data_ptr()
        c.alibi_slopes = _vector(alibi_slopes, "alibi_slopes", torch.float32, self.num_q_heads,
                                 self._index, optional=True) or None
        image = bytes(c)
        self._head, self._tail = image[:_lib.Paged.kv_len.offset], image[_lib.Paged.alibi_slopes.offset:]
        n = ctypes.c_size_t()
        _lib.load().fkv_paged_workspace_size(ctypes.byref(n))
        self._ws_bytes = n.value

    def workspace(self) -> torch.Tensor:
        """A workspace for calls on this device, zeroed on its current stream; one
        per stream of calls (calls that share a workspace must not overlap on the
        GPU)."""
        return torch.zeros(self._ws_bytes, dtype=torch.uint8, device=self.device)

    def _struct(self, kv_len, cu_q=None, prefix_len=None) -> bytes:
        """fkv_paged_t of one call."""
        n, index, i32 = self.num_seqs, self._index, torch.int32
        return self._head + _pack_batch(
            _vector(kv_len, "kv_len", i32, n, index),
            0 if cu_q is None else _vector(cu_q, "cu_q", i32, n + 1, index),
            0 if prefix_len is None else _vector(prefix_len, "prefix_len", i32, n, index)) + self._tail

    def _rows(self, t, name, tokens, heads) -> bytes:
        return _rows(t, name, (tokens, heads, self.head_dim), self.dtype, self._index)

    def _ws(self, ws) -> int:
        return _vector(ws, "ws", torch.uint8, self._ws_bytes, self._index)

    def _lse(self, lse, tokens) -> Optional[int]:
        return None if lse is None else _vector(lse, "lse", torch.float32, tokens * self.num_q_heads,
                                                self._index)


def paged_append(cache: PagedCache, kv_len: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                 ws: torch.Tensor, *, cu_q: Optional[torch.Tensor] = None,
                 rope: Optional[Rope] = None, positions: Optional[torch.Tensor] = None,
                 q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                 stream=None):
    """Appends k, v [tokens, Hkv, D] at the ends of their sequences
    (fkv_paged_append).  kv_len: int32 [sequences], lengths WITH the new tokens;
    cu_q: int32 [sequences + 1] token offsets (None: one token per sequence).
    With `rope` the keys are normed and rotated on the way, at `positions` (None:
    their cache positions), and so are the queries q [tokens, Hq, D] into q_out
    (which may be q) when given."""
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if rope is None and positions is not None:
        raise ValueError("positions without a rope")
    tokens, hk, hq = k.shape[0], cache.num_kv_heads, cache.num_q_heads
    _call("fkv_paged_append", cache._index, stream, cache._struct(kv_len, cu_q),
          None if rope is None else rope._struct(cache.head_dim, positions, tokens, cache._index, True), tokens,
          None if q is None else cache._rows(q, "q", tokens, hq), cache._rows(k, "k", tokens, hk),
          cache._rows(v, "v", tokens, hk), None if q is None else cache._rows(q_out, "q_out", tokens, hq),
          cache._ws(ws))


def paged_decode(cache: PagedCache, kv_len: torch.Tensor, q: torch.Tensor, out: torch.Tensor,
                 ws: torch.Tensor, *, prefix_len: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, stream=None):
    """Attention of one token per sequence, q and out [sequences, Hq, D], over
    the cached keys (fkv_paged_decode).  prefix_len: int32 [sequences], keys that
    every query sees whatever the window; lse: float32 [sequences, Hq] output."""
    n, hq = cache.num_seqs, cache.num_q_heads
    _call("fkv_paged_decode", cache._index, stream, cache._struct(kv_len, None, prefix_len),
          cache._rows(q, "q", n, hq), cache._rows(out, "out", n, hq), cache._lse(lse, n), cache._ws(ws))


def paged_attend(cache: PagedCache, kv_len: torch.Tensor, cu_q: Optional[torch.Tensor],
                 q: torch.Tensor, out: torch.Tensor, ws: torch.Tensor, *,
                 prefix_len: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 stream=None):
    """Attention of a ragged batch of query tokens, q and out [tokens, Hq, D],
    over the cached keys (fkv_paged_attend); kv_len and cu_q as in
    :func:`paged_append`, prefix_len and lse (float32 [tokens, Hq]) as in
    :func:`paged_decode`.  In bfloat16 the probabilities are rounded to bfloat16
    before their product with the values."""
    tokens, hq = q.shape[0], cache.num_q_heads
    _call("fkv_paged_attend", cache._index, stream, cache._struct(kv_len, cu_q, prefix_len), tokens,
          cache._rows(q, "q", tokens, hq), cache._rows(out, "out", tokens, hq), cache._lse(lse, tokens),
          cache._ws(ws))
