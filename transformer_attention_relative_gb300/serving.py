"""Rotary positions and the paged key/value cache over CUDA tensors.

Marshalling only, as in the package's other functions: checks of types, shapes
and strides, allocation of the outputs, and one call of the C entry point on the
current stream. A decode step makes these calls for every layer, so they are
kept short: what a call needs of the cache or the plan is laid out when that is
made.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import (MODE_ALIBI, MODE_T5, RELPOS_BF16, RELPOS_E4M3, RELPOS_FP32, RELPOS_NO_BIAS, RELPOS_OK,
               ROTARY_LAYOUTS, ROTARY_SCALINGS, RelposError, _output_of, _PagedCache, _RotaryPlan, _RowStrides,
               load_library, relpos_rotary_plan_init)

_DTYPES = {torch.bfloat16: RELPOS_BF16, torch.float32: RELPOS_FP32}
_byref = ctypes.byref
# what torch's own wrappers call, which saves a microsecond each; those where a torch has them no longer
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream)
_empty_like = torch.empty_like
_int32, _bf16 = torch.int32, torch.bfloat16
_MOST = 2 ** 31 - 1  # the C entry points take sizes as 32-bit integers, ctypes cuts larger ones silently
_tensor = struct.Struct("@PP6qi4x").pack  # a RelposRotaryTensor's bytes: quicker than its ctypes structure
_entries = None


@functools.lru_cache(maxsize=1024)
def _strides(batch, head, row):
    """A stride triple as the C entry points take it (read only)."""
    return _byref(_RowStrides(batch, head, row))


def _lib():
    """The C entry points, looked up once."""
    global _entries
    if _entries is None:
        lib = load_library()
        _entries = (lib.relpos_rotary, lib.relpos_paged_append, lib.relpos_paged_decode)
    return _entries


def _check_device(index, *tensors):
    """The library launches on the current device: every tensor has to be there."""
    if index < 0:
        raise ValueError("tensors must be CUDA tensors")
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors must be on one device")
    if index != _device():
        raise ValueError("tensors must be on the current CUDA device")


class RotaryPlan:
    """Frequencies and layout of rotary positions, made once and passed to each call.

    ``rot_dim`` dimensions of a head are turned, as pairs of its halves (``layout="half"``) or of neighbours
    (``"interleaved"``). ``scaling`` stretches the positions for contexts longer than the trained one: ``"linear"``,
    ``"ntk"``, or ``"yarn"`` with ``original_len`` trained positions (see ``relpos_rotary_plan_init`` in the C header).
    """

    def __init__(self, rot_dim: int, *, layout: str = "half", base: float = 10000.0, scaling: str = "none",
                 factor: float = 1.0, original_len: float = 0.0, fast_turns: float = 32.0, slow_turns: float = 1.0):
        if layout not in ROTARY_LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(ROTARY_LAYOUTS)}")
        if scaling not in ROTARY_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(ROTARY_SCALINGS)}")
        self._c = _RotaryPlan()
        self.rot_dim = rot_dim
        rc = relpos_rotary_plan_init(_byref(self._c), rot_dim, ROTARY_LAYOUTS[layout], base, ROTARY_SCALINGS[scaling],
                                     factor, original_len, fast_turns, slow_turns)
        if rc != RELPOS_OK:
            raise RelposError(rc, "relpos_rotary_plan_init")
        self._ref = _byref(self._c)


def _row_of(x, y, B, L, d):
    """(x, out, strides of both, heads) as the C entry point takes them."""
    b, H, l, e = x.shape
    if b != B or l != L or e != d:
        raise ValueError("Q and K must agree but for their heads")
    x0, x1, x2, x3 = x.stride()
    y0, y1, y2, y3 = y.stride()
    if (x3 != 1 or y3 != 1) and d > 1:
        raise ValueError("the last dimension must be contiguous")
    return x.data_ptr(), y.data_ptr(), x0, x1, x2, y0, y1, y2, H


def _rotate(Q, plan, K, positions, offset, out, stream, inverse, what):
    dtype = _DTYPES.get(Q.dtype)
    if dtype is None:
        raise TypeError(f"unsupported dtype {Q.dtype}")
    if K is not None and K.dtype != Q.dtype:
        raise TypeError("Q, K and out must have one dtype")
    B, _, L, d = Q.shape
    if B * L > _MOST or not -_MOST - 1 <= offset <= _MOST:
        raise ValueError("more rows, or positions, than 32-bit integers hold")
    index = Q.get_device()
    _check_device(index, K, positions)
    if out is None:
        if stream is None:
            outs = (_empty_like(Q),) if K is None else (_empty_like(Q), _empty_like(K))
        else:
            outs = tuple(_output_of(stream, lambda: _empty_like(x)) for x in ((Q,) if K is None else (Q, K)))
    else:
        ins, outs = ((Q,), (out,)) if K is None else ((Q, K), tuple(out))
        if len(outs) != len(ins):
            raise ValueError("out must hold one tensor for each input")
        _check_device(index, *outs)
        for x, y in zip(ins, outs):
            if y.dtype != Q.dtype:
                raise TypeError("Q, K and out must have one dtype")
            if y.shape != x.shape:
                raise ValueError("out must have its input's shape")
    ptr, step = None, 0
    if positions is not None:
        if positions.dtype != _int32:
            raise TypeError("positions must be int32")
        shape = positions.shape
        if shape != (B, L) and shape != (L,):
            raise ValueError("positions must be [L] or [B, L]")
        if L > 1 and positions.stride(-1) != 1:
            raise ValueError("positions must be contiguous along a sequence")
        ptr = positions.data_ptr()
        if len(shape) == 2:
            step = positions.stride(0)
    if K is None:
        n, desc = 1, _tensor(*_row_of(Q, outs[0], B, L, d))
    else:
        n, desc = 2, _tensor(*_row_of(Q, outs[0], B, L, d)) + _tensor(*_row_of(K, outs[1], B, L, d))
    rc = _lib()[0](plan._ref, dtype, inverse, desc, n, B, L, d, ptr, step, offset,
                   _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc != RELPOS_OK:
        raise RelposError(rc, what)
    return outs[0] if K is None else outs


def rotary(Q, plan, K=None, *, positions=None, offset: int = 0, out=None, stream=None):
    """Turn queries (and keys, in the same launch) by their positions; returns ``out``, a pair when K is given.

    Q [B,Hq,L,d] and K [B,Hk,L,d] are bf16 or fp32 with any strides but a contiguous last dimension; a [T,H,d]
    tensor of ragged rows goes in as ``x.transpose(0, 1)[None]`` with its tokens' positions. ``positions``: int32
    [L] or [B,L]; without it row l is at ``offset + l``. ``out`` is allocated like the inputs when not given, and
    may be the inputs themselves.
    """
    return _rotate(Q, plan, K, positions, offset, out, stream, 0, "relpos_rotary")


def rotary_backward(dQ, plan, dK=None, *, positions=None, offset: int = 0, out=None, stream=None):
    """Gradients of ``rotary`` with respect to its inputs, from those of its outputs (arguments as ``rotary``)."""
    return _rotate(dQ, plan, dK, positions, offset, out, stream, 1, "relpos_rotary")


class PagedCache:
    """A pool of pages for keys and values, ``k`` and ``v`` [num_pages, H, page, d]: bf16, or float8_e4m3fn with fp32
    ``k_scale`` and ``v_scale`` [num_pages, H] (a value is its code times its page's and head's scale)."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn) or v.dtype != k.dtype:
            raise TypeError("k and v must both be bfloat16 or both float8_e4m3fn")
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError("k and v must be [num_pages, H, page, d]")
        eight = k.dtype == torch.float8_e4m3fn
        if eight != (k_scale is not None) or eight != (v_scale is not None):
            raise ValueError("k_scale and v_scale come with a float8_e4m3fn cache, and only with one")
        for s in (k_scale, v_scale):
            if s is not None and (s.dtype != torch.float32 or s.shape != k.shape[:2]):
                raise TypeError("scales must be fp32 [num_pages, H]")
        for t in (k, v, k_scale, v_scale):
            if t is not None and not t.is_contiguous():
                raise ValueError("the cache's tensors must be contiguous")
        _check_device(k.get_device(), v, k_scale, v_scale)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.heads, self.page_size, self.head_dim = k.shape
        self._index = k.get_device()
        self._c = _PagedCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if eight else None,
                              v_scale.data_ptr() if eight else None, *k.shape,
                              RELPOS_E4M3 if eight else RELPOS_BF16)
        self._ref = _byref(self._c)

    @classmethod
    def empty(cls, num_pages: int, heads: int, head_dim: int, *, page_size: int = 64, dtype=torch.bfloat16,
              device="cuda"):
        """A cache of its own memory; ``dtype`` bfloat16 or float8_e4m3fn."""
        shape = (num_pages, heads, page_size, head_dim)
        if dtype != torch.float8_e4m3fn:
            return cls(*(torch.zeros(shape, dtype=dtype, device=device) for _ in range(2)))
        return cls(*(torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype) for _ in range(2)),
                   *(torch.ones(shape[:2], device=device) for _ in range(2)))


def _check_table(block_table, lens, B):
    """(stride between rows, pages of a row) of a block table."""
    if block_table.dtype != _int32 or lens.dtype != _int32:
        raise TypeError("block_table and lens must be int32")
    shape = block_table.shape
    if len(shape) != 2 or shape[0] != B or lens.shape != (B,):
        raise ValueError("block_table must be [B, max_pages] and lens [B]")
    rows, cols = block_table.stride()
    if (cols != 1 and shape[1] > 1) or (B > 1 and lens.stride(0) != 1):
        raise ValueError("block_table rows and lens must be contiguous")
    return rows, shape[1]


def paged_append(cache, K, V, block_table, lens, *, cu_new=None, plan=None, stream=None):
    """Run ``relpos_paged_append``: write each sequence's newest tokens into its pages, keys turned by ``plan``.

    K, V bf16, contiguous along d: [B,H,n,d] with n new tokens of every sequence, or ragged rows [T,H,d] with
    ``cu_new`` (int32 [B+1], first row of each sequence). block_table int32 [B, max_pages]; lens int32 [B], the
    tokens of each sequence with the new ones.
    """
    if K.dtype != _bf16 or V.dtype != _bf16:
        raise TypeError("K and V must be bf16")
    shape = K.shape
    if V.shape != shape or len(shape) != (4 if cu_new is None else 3):
        raise ValueError("K and V must be [B,H,n,d], or [T,H,d] with cu_new")
    if shape[1] != cache.heads or shape[-1] != cache.head_dim:
        raise ValueError("K and V must have the cache's heads and head dimension")
    if shape[0] * shape[-2] > _MOST:
        raise ValueError("more rows than 32-bit integers hold")
    sk, sv = K.stride(), V.stride()
    if sk[-1] != 1 or sv[-1] != 1:
        raise ValueError("the last dimension must be contiguous")
    if cu_new is None:
        B, n, rows, cu = shape[0], shape[2], 0, None
        ks, vs = _strides(sk[0], sk[1], sk[2]), _strides(sv[0], sv[1], sv[2])
    else:
        if cu_new.dtype != torch.int32 or cu_new.dim() != 1 or cu_new.shape[0] < 1:
            raise TypeError("cu_new must be int32 [B + 1]")
        if not cu_new.is_contiguous():
            raise ValueError("cu_new must be contiguous")
        B, n, rows, cu = cu_new.shape[0] - 1, 0, shape[0], cu_new.data_ptr()
        ks, vs = _strides(0, sk[1], sk[0]), _strides(0, sv[1], sv[0])
    step, pages = _check_table(block_table, lens, B)
    index = cache._index
    _check_device(index, K, V, cu_new, block_table, lens)
    rc = _lib()[1](cache._ref, None if plan is None else plan._ref, K.data_ptr(), V.data_ptr(), ks, vs,
                   cu, rows, n, B, block_table.data_ptr(), step, pages, lens.data_ptr(),
                   _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc != RELPOS_OK:
        raise RelposError(rc, "relpos_paged_append")


def paged_decode(Q, cache, block_table, lens, *, bias=None, mode=None, num_buckets: int = 32,
                 max_distance: int = 128, scale: float = 0.0, out=None, stream=None):
    """Run ``relpos_paged_decode``: attention of each sequence's newest rows over its cached tokens; returns ``out``.

    Q bf16 [B,Hq,Lq,d] (Lq <= 8; Hq a multiple of the cache's heads), any strides but a contiguous last dimension;
    its rows are the last Lq of the lens[b] tokens. ``mode``: None (no bias), ``MODE_T5`` with bias fp32
    [num_buckets, Hq] (causal buckets) or ``MODE_ALIBI`` with the slopes fp32 [Hq]. ``scale`` 0 takes 1/sqrt(d).
    """
    if Q.dtype != _bf16 or (out is not None and out.dtype != _bf16):
        raise TypeError("Q and out must be bf16")
    B, Hq, Lq, d = Q.shape
    if d != cache.head_dim:
        raise ValueError("Q must have the cache's head dimension")
    if out is None:
        out = _empty_like(Q) if stream is None else _output_of(stream, lambda: _empty_like(Q))
    elif out.shape != Q.shape:
        raise ValueError("out must have Q's shape")
    q0, q1, q2, q3 = Q.stride()
    o0, o1, o2, o3 = out.stride()
    if q3 != 1 or o3 != 1:
        raise ValueError("the last dimension must be contiguous")
    step, pages = _check_table(block_table, lens, B)
    index = cache._index
    _check_device(index, Q, out, block_table, lens, bias)
    if mode is None:
        if bias is not None:
            raise ValueError("a bias needs its mode")
        mode, ptr = RELPOS_NO_BIAS, None
    else:
        if mode != MODE_T5 and mode != MODE_ALIBI:
            raise ValueError("mode must be None, MODE_T5 or MODE_ALIBI")
        if not 0 < max_distance <= _MOST:
            raise ValueError("max_distance must be positive and fit 32 bits")
        if bias is None or bias.dtype != torch.float32 or not bias.is_contiguous():
            raise TypeError("bias must be a contiguous fp32 tensor")
        if bias.shape != ((num_buckets, Hq) if mode == MODE_T5 else (Hq,)):
            raise ValueError("bias must be [num_buckets, Hq] for MODE_T5, [Hq] for MODE_ALIBI")
        ptr = bias.data_ptr()
    rc = _lib()[2](cache._ref, Q.data_ptr(), _strides(q0, q1, q2), B, Hq, Lq, block_table.data_ptr(), step,
                   pages, lens.data_ptr(), mode, ptr, num_buckets, max_distance, scale, out.data_ptr(),
                   _strides(o0, o1, o2), _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc != RELPOS_OK:
        raise RelposError(rc, "relpos_paged_decode")
    return out
