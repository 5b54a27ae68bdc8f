"""Paged KV cache of the binding: per-head norm and rotation of new rows, their
append to the cache, and attention over it (include/fkv.h, "Paged cache").

A :class:`Rope` and a :class:`PagedCache` are made once per model layer: they
check the tensors that stay (weights, frequencies, caches, page table) and keep
them alive.  The calls check and marshal the tensors of one step.  Every tensor
of a call lives on the cache's device; the call runs there, on `stream` or on
that device's current stream, whatever device is current.

Nothing here is differentiable: these are serving operators, as the rest of
the library.  Tensors used on another stream than the one they were allocated
on are the caller's to keep alive (``Tensor.record_stream``).
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional, Sequence

import torch

from . import _lib

_DTYPES = {torch.bfloat16: _lib.FKV_DTYPE_BF16, torch.float32: _lib.FKV_DTYPE_FP32}
_HERE = contextlib.nullcontext()


def _check(status: int, where: str):
    if status != _lib.FKV_OK:
        from . import FkvError
        raise FkvError(status, where)


def _device(device: torch.device):
    """The context in which a call on `device` runs."""
    return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _stream(stream, device: torch.device) -> int:
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the call on {device}")
        return stream.cuda_stream
    return int(stream)


def _vector(t: Optional[torch.Tensor], name: str, dtype, numel: int, device,
            optional: bool = False) -> Optional[int]:
    """Data pointer of a contiguous vector of at least numel entries."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if t.dtype != dtype or t.device != device or not t.is_contiguous() or t.numel() < numel:
        raise ValueError(f"{name} must be contiguous {dtype} with at least {numel} elements on "
                         f"{device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, shape, dtype, device) -> _lib.Rows:
    """fkv_rows_t of a [tokens, heads, D] tensor whose last dimension is contiguous."""
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be {dtype} on {device}, got {t.dtype} on {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    ts, hs, ds = t.stride()
    if ds != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return _lib.Rows(t.data_ptr(), ts, hs)


class Rope:
    """Norm and rotation of query and key rows (fkv_rope_t); see :func:`make_rope`."""

    def __init__(self, omega, axis_pairs, style, norm, eps, q_weight, k_weight):
        self.omega, self.q_weight, self.k_weight = omega, q_weight, k_weight
        self.axis_pairs = tuple(int(n) for n in axis_pairs)
        if not 1 <= len(self.axis_pairs) <= 3:
            raise ValueError("axis_pairs has one to three entries")
        n = sum(self.axis_pairs)
        tensors = [t for t in (omega, q_weight, k_weight) if t is not None]
        self.device = tensors[0].device if tensors else None
        if self.device is not None and self.device.type != "cuda":
            raise ValueError("omega and the weights must be CUDA tensors")
        c = self._c = _lib.Rope()
        c.style = {"interleaved": _lib.FKV_ROPE_ADJACENT, "half": _lib.FKV_ROPE_HALF}[style]
        c.norm = 1 if norm else 0
        c.n_axes = len(self.axis_pairs)
        for i, m in enumerate(self.axis_pairs):
            c.axis_pairs[i] = m
        c.eps = eps
        c.omega = _vector(omega, "omega", torch.float32, n, self.device, optional=n == 0)
        self._image = bytes(c)

    def _call(self, head_dim, positions, tokens, device, cache_positions=False) -> _lib.Rope:
        """The struct of one call."""
        if self.device is not None and self.device != device:
            raise ValueError(f"the rope's tensors are on {self.device}, the rows on {device}")
        c = _lib.Rope.from_buffer_copy(self._image)
        if self.q_weight is not None:
            c.q_weight = _vector(self.q_weight, "q_weight", torch.float32, head_dim, device)
        if self.k_weight is not None:
            c.k_weight = _vector(self.k_weight, "k_weight", torch.float32, head_dim, device)
        axes = len(self.axis_pairs)
        if positions is not None:
            shape = tuple(positions.shape)
            if shape != (axes, tokens) and not (axes == 1 and shape == (tokens,)):
                raise ValueError(f"positions must have the shape ({axes}, {tokens}), got {shape}")
            c.positions = _vector(positions, "positions", torch.int32, axes * tokens, device)
            c.axis_stride = tokens
        elif sum(self.axis_pairs) > 0 and not (cache_positions and axes == 1):
            raise ValueError("positions is required")
        return c


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
    if sum(axis_pairs) != n:
        raise ValueError(f"axis_pairs {tuple(axis_pairs)} do not add up to the {n} frequencies")
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
    if some.dim() != 3 or some.dtype not in _DTYPES or not some.is_cuda:
        raise ValueError("rows are [tokens, heads, D] CUDA tensors in bfloat16 or float32")
    dev, dt = some.device, some.dtype
    tokens, _, D = some.shape
    hq = 0 if q is None else q.shape[1]
    hk = 0 if k is None else k.shape[1]
    rq, rqo = (None, None) if q is None else (_rows(q, "q", (tokens, hq, D), dt, dev),
                                              _rows(q_out, "q_out", (tokens, hq, D), dt, dev))
    rk, rko = (None, None) if k is None else (_rows(k, "k", (tokens, hk, D), dt, dev),
                                              _rows(k_out, "k_out", (tokens, hk, D), dt, dev))
    r = rope._call(D, positions, tokens, dev)
    with _device(dev):
        st = _lib.load().fkv_qk_norm_rope(r, _DTYPES[dt], D, tokens, hq, hk, rq, rk, rqo, rko,
                                          _stream(stream, dev))
    _check(st, "fkv_qk_norm_rope")


class PagedCache:
    """A paged cache and how its queries read it (fkv_paged_t).

    k_cache, v_cache: [num_pages, Hkv, page_size, D], any strides with the last
    dimension contiguous, the same for both (a cache kept as [num_pages,
    page_size, Hkv, D] is passed as its ``transpose(1, 2)``).  page_table: int32
    [sequences, max_pages].  softcap, window, alibi_slopes and causal as in
    fkv_paged_t; scale defaults to 1 / sqrt(D).  The page table may be changed
    in place between calls."""

    def __init__(self, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, *,
                 num_q_heads: int, scale: Optional[float] = None, softcap: float = 0.0,
                 window: int = 0, causal: bool = True,
                 alibi_slopes: Optional[torch.Tensor] = None):
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
        c.alibi_slopes = _vector(alibi_slopes, "alibi_slopes", torch.float32, self.num_q_heads, dev,
                                 optional=True)
        self._image = bytes(c)

    def workspace(self) -> torch.Tensor:
        """A zeroed workspace for calls on this device; one per stream of calls
        (calls that share a workspace must not overlap on the GPU)."""
        n = ctypes.c_size_t()
        _check(_lib.load().fkv_paged_workspace_size(ctypes.byref(n)), "fkv_paged_workspace_size")
        with _device(self.device):
            return torch.zeros(n.value, dtype=torch.uint8, device=self.device)

    def _call(self, kv_len, cu_q=None, prefix_len=None) -> _lib.Paged:
        """The struct of one call (a copy: calls from several threads do not share it)."""
        c = _lib.Paged.from_buffer_copy(self._image)
        c.kv_len = _vector(kv_len, "kv_len", torch.int32, self.num_seqs, self.device)
        if cu_q is not None:
            c.cu_q = _vector(cu_q, "cu_q", torch.int32, self.num_seqs + 1, self.device)
        if prefix_len is not None:
            c.prefix_len = _vector(prefix_len, "prefix_len", torch.int32, self.num_seqs, self.device)
        return c

    def _ws(self, ws) -> int:
        n = _WS_BYTES or _workspace_bytes()
        return _vector(ws, "ws", torch.uint8, n, self.device)


_WS_BYTES = 0


def _workspace_bytes() -> int:
    global _WS_BYTES
    n = ctypes.c_size_t()
    _check(_lib.load().fkv_paged_workspace_size(ctypes.byref(n)), "fkv_paged_workspace_size")
    _WS_BYTES = n.value
    return _WS_BYTES


def _token_rows(t, name, cache: PagedCache, tokens, heads):
    return _rows(t, name, (tokens, heads, cache.head_dim), cache.dtype, cache.device)


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
    tokens = k.shape[0]
    c = cache._call(kv_len, cu_q)
    rk = _token_rows(k, "k", cache, tokens, cache.num_kv_heads)
    rv = _token_rows(v, "v", cache, tokens, cache.num_kv_heads)
    rq = rqo = None
    if q is not None:
        rq = _token_rows(q, "q", cache, tokens, cache.num_q_heads)
        rqo = _token_rows(q_out, "q_out", cache, tokens, cache.num_q_heads)
    if rope is None and positions is not None:
        raise ValueError("positions without a rope")
    r = None if rope is None else rope._call(cache.head_dim, positions, tokens, cache.device, True)
    with _device(cache.device):
        st = _lib.load().fkv_paged_append(c, r, tokens, rq, rk, rv, rqo, cache._ws(ws),
                                          _stream(stream, cache.device))
    _check(st, "fkv_paged_append")


def paged_decode(cache: PagedCache, kv_len: torch.Tensor, q: torch.Tensor, out: torch.Tensor,
                 ws: torch.Tensor, *, prefix_len: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, stream=None):
    """Attention of one token per sequence, q and out [sequences, Hq, D], over
    the cached keys (fkv_paged_decode).  prefix_len: int32 [sequences], keys that
    every query sees whatever the window; lse: float32 [sequences, Hq] output."""
    c = cache._call(kv_len, None, prefix_len)
    n = cache.num_seqs
    rq = _token_rows(q, "q", cache, n, cache.num_q_heads)
    ro = _token_rows(out, "out", cache, n, cache.num_q_heads)
    pl = _vector(lse, "lse", torch.float32, n * cache.num_q_heads, cache.device, optional=True)
    with _device(cache.device):
        st = _lib.load().fkv_paged_decode(c, rq, ro, pl, cache._ws(ws), _stream(stream, cache.device))
    _check(st, "fkv_paged_decode")


def paged_attend(cache: PagedCache, kv_len: torch.Tensor, cu_q: torch.Tensor, q: torch.Tensor,
                 out: torch.Tensor, ws: torch.Tensor, *, prefix_len: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, stream=None):
    """Attention of a ragged batch of query tokens, q and out [tokens, Hq, D],
    over the cached keys (fkv_paged_attend); kv_len and cu_q as in
    :func:`paged_append`, prefix_len and lse (float32 [tokens, Hq]) as in
    :func:`paged_decode`."""
    tokens = q.shape[0]
    c = cache._call(kv_len, cu_q, prefix_len)
    rq = _token_rows(q, "q", cache, tokens, cache.num_q_heads)
    ro = _token_rows(out, "out", cache, tokens, cache.num_q_heads)
    pl = _vector(lse, "lse", torch.float32, tokens * cache.num_q_heads, cache.device, optional=True)
    with _device(cache.device):
        st = _lib.load().fkv_paged_attend(c, tokens, rq, ro, pl, cache._ws(ws),
                                          _stream(stream, cache.device))
    _check(st, "fkv_paged_attend")
