"""Binding of what stands around the delta in a layer's step (include/sgmv.h): the norm before it, the 4-bit
base product that it is added to, and the rotated append behind it; imported by the package, whose names these are.
Argument marshalling only; calls for serving, which autograd does not see.

    sgmv_rms_norm(x, weight, eps, residual, quantise) -> Normed
    sgmv_base_pack(codes, scale, zero, K, group, format) -> BaseWeight
    sgmv_base_product(x, base)                        -> y
    sgmv_kv_append(q, k, v, batch, cache, cos_sin)    -> q (rotated; cache updated in place)
"""
from __future__ import annotations

import ctypes
import struct
from dataclasses import dataclass, field
from typing import NamedTuple, Optional

import torch

from . import SGMV_OK, _check, _dtype_code, _lib
from ._serving import KV_E4M3, KV_I8, KvBatch, KvCache, _MOST, _int32, _KvBatch, _KvCache, _on_gpu, _rows3

MAX_NORM_WIDTH = 32768
BASE_MAX_SIZE = 4194304
BASE_MAX_SPLITS = 16
BASE_I4, BASE_E2M1 = range(2)
_CODES = {torch.float8_e4m3fn: KV_E4M3, torch.int8: KV_I8}


class _Norm(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "residual", "weight", "residual_out", "out", "codes", "scale")] +
                [(f"ld{a}_{b}", ctypes.c_int64) for a in "xrsoc" for b in ("token", "head")] +
                [(n, ctypes.c_int32) for n in ("T", "heads", "width", "dtype", "format")] + [("eps", ctypes.c_float)])


class _Base(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("codes", "scale", "zero")] +
                [(n, ctypes.c_int32) for n in ("N", "K", "group", "format", "dtype", "has_zero")])


class _Rotation(ctypes.Structure):
    _fields_ = ([("cos_sin", ctypes.c_void_p), ("ld", ctypes.c_int64)] +
                [(n, ctypes.c_int32) for n in ("positions", "rotary", "interleaved", "heads")] +
                [("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p)] +
                [(n, ctypes.c_int64) for n in ("ldq_token", "ldq_head", "ldo_token", "ldo_head")])


# The same as bytes, which take a third of the time to fill (0: no pointer); calls take either.
_pack_norm, _pack_rotation = (struct.Struct(f).pack for f in ("7P10q5if", "Pq4i2P4q"))
assert struct.calcsize("7P10q5if") == ctypes.sizeof(_Norm) and struct.calcsize("Pq4i2P4q") == ctypes.sizeof(_Rotation)


def _bind():
    i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    P = ctypes.POINTER
    B = P(_Base)
    for name, args in {
        "sgmv_rms_norm": [vp, vp],
        "sgmv_base_init": [i32, i32, i32, i32, i32, i32, B, P(sz), P(sz), P(sz)],
        "sgmv_base_pack": [vp, i64, vp, vp, B, vp],
        "sgmv_base_product_workspace": [i32, B, i32, P(sz)],
        "sgmv_base_product": [vp, i64, i32, B, vp, i64, i32, vp, sz, vp],
        "sgmv_kv_append": [vp, vp, i64, i64, vp, i64, i64, i32, P(_KvBatch), P(_KvCache), vp],
    }.items():
        f = getattr(_lib, name)
        f.argtypes, f.restype = args, ctypes.c_int


_bind()


_current = torch._C._cuda_getDevice  # (the calls behind torch.cuda's, which take longer than they)
_stream = torch._C._cuda_getCurrentRawStream
_tuple = tuple.__new__
_like, _dense = torch.empty_like, torch.contiguous_format  # (allocates faster than new_empty of a shape)
_ROWS = {torch.float32: _dtype_code(torch.float32), torch.bfloat16: _dtype_code(torch.bfloat16)}


def _elsewhere(index: int, call, *args) -> int:
    """The call with GPU `index` made the current one (the default stream's handle is that of the current GPU)."""
    with torch.cuda.device(index):
        return call(*args, _stream(index))


# ---------------------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------------------
class Normed(NamedTuple):
    out: Optional[torch.Tensor]       # as x, or None
    residual: Optional[torch.Tensor]  # x + residual, or None
    codes: Optional[torch.Tensor]     # float8_e4m3fn or int8, or None
    scale: Optional[torch.Tensor]     # float32, of each row


def _refuse(t: torch.Tensor, shape, dtype: torch.dtype, index: int, what: str):
    if t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{what} must be on x's device")
    raise ValueError(f"{what} must be contiguous over the last dimension")


def _strides(t: torch.Tensor, shape, dtype: torch.dtype, index: int, what: str):
    """Token and head strides of rows [T, width] or [T, heads, width]."""
    st = t.stride()
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or (st[-1] != 1 and shape[-1] > 1):
        _refuse(t, shape, dtype, index, what)
    # a stride of a single token or head says nothing
    if len(st) == 2:
        return (st[0] if shape[0] > 1 else shape[1]), shape[1]
    head = st[1] if shape[1] > 1 else shape[2]
    return (st[0] if shape[0] > 1 else shape[1] * head), head


def sgmv_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                  residual: Optional[torch.Tensor] = None, quantise: Optional[torch.dtype] = None,
                  want_out: bool = True, out: Optional[torch.Tensor] = None,
                  residual_out: Optional[torch.Tensor] = None, codes: Optional[torch.Tensor] = None,
                  scale: Optional[torch.Tensor] = None) -> Normed:
    """Root-mean-square norm of rows x [T, width], or [T, heads, width] head by head (strided views are fine),
    times ``weight``; of x + ``residual`` where one is given, which is returned too. ``quantise``
    (float8_e4m3fn or int8) asks for the normed rows as codes with one scale per row as well, ``want_out=False``
    for those alone. Outputs are allocated unless given; ``out`` and ``residual_out`` may be x or residual
    themselves (views of the same strides, each another one). The norm is that of the fp32 sum: ``residual``
    of the result is that sum rounded."""
    shape, dtype, index = x.shape, x.dtype, x.get_device()
    if len(shape) == 2:
        T, W = shape
        heads = 1
    elif len(shape) == 3:
        T, heads, W = shape
    else:
        raise ValueError(f"x must be [T, width] or [T, heads, width], got {list(shape)}")
    code = _ROWS.get(dtype)
    if code is None:
        _dtype_code(dtype)  # says which
    if T > _MOST or heads > _MOST or W > _MOST:
        _int32("T, heads and width", T, heads, W)
    if weight.numel() != W or weight.dtype is not dtype or weight.get_device() != index or weight.dim() != 1 or (
            not weight.is_contiguous()):
        raise TypeError(f"weight must be {W} contiguous {dtype} entries on x's device")
    xt, xh = _strides(x, shape, dtype, index, "x")
    rp = sp = op = cp = fp = 0
    dense = heads * W
    rt = st = ot = ct = dense
    rh = sh = oh = ch = W
    fmt = 0
    if residual is not None:
        rt, rh = _strides(residual, shape, dtype, index, "residual")
        rp = residual.data_ptr()
        if residual_out is None:
            residual_out = _like(x, memory_format=_dense)
        else:
            st, sh = _strides(residual_out, shape, dtype, index, "residual_out")
        sp = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out goes with a residual")
    if out is not None:
        ot, oh = _strides(out, shape, dtype, index, "out")
        op = out.data_ptr()
    elif want_out:
        out = _like(x, memory_format=_dense)
        op = out.data_ptr()
    if quantise is not None:
        fmt = _CODES.get(quantise)
        if fmt is None:
            raise TypeError(f"codes are float8_e4m3fn or int8, got {quantise}")
        if codes is None:
            codes = _like(x, dtype=quantise, memory_format=_dense)
        else:
            ct, ch = _strides(codes, shape, quantise, index, "codes")
        if scale is None:
            scale = x.new_empty((T,) if len(shape) == 2 else (T, heads), dtype=torch.float32)
        elif scale.shape != shape[:-1] or scale.dtype != torch.float32 or not scale.is_contiguous() or (
                scale.get_device() != index):
            raise TypeError("scale must be a contiguous float32 tensor of one entry per row on x's device")
        cp, fp = codes.data_ptr(), scale.data_ptr()
    elif codes is not None or scale is not None:
        raise ValueError("codes and scale go with quantise")
    elif out is None:
        raise ValueError("nothing to compute: neither out nor codes are wanted")
    if index < 0:
        raise ValueError("the kernels run on GPU tensors")
    a = _pack_norm(x.data_ptr(), rp, weight.data_ptr(), sp, op, cp, fp, xt, xh, rt, rh, st, sh, ot, oh, ct, ch, T, heads, W,
                   code, fmt, eps)
    call = _lib.sgmv_rms_norm
    status = call(a, _stream(index)) if index == _current() else _elsewhere(index, call, a)
    if status != SGMV_OK:
        _check(status, "sgmv_rms_norm")
    return _tuple(Normed, (out, residual_out, codes, scale))


# ---------------------------------------------------------------------------------------
# base product
# ---------------------------------------------------------------------------------------
@dataclass
class BaseWeight:
    codes: torch.Tensor           # uint8, the library's layout
    scale: torch.Tensor           # of dtype (I4) or uint8 (E2M1)
    zero: Optional[torch.Tensor]  # uint8, I4 with zero points
    desc: _Base
    dtype: torch.dtype            # of x and y
    ref: object = field(init=False, repr=False)  # what the library takes
    index: int = field(init=False, repr=False)   # of the GPU, -1: not on one
    few: int = field(init=False, repr=False)     # rows that take no workspace

    def __post_init__(self):
        self.N, self.K, self.group, self.format = self.desc.N, self.desc.K, self.desc.group, self.desc.format
        self.ref, self.index = ctypes.byref(self.desc), self.codes.get_device()
        self.few = 16 if self.dtype is torch.float32 else 32


def sgmv_base_pack(codes: torch.Tensor, scale: torch.Tensor, zero: Optional[torch.Tensor] = None,
                   K: Optional[int] = None, group: int = 128, format: int = BASE_I4,
                   dtype: Optional[torch.dtype] = None) -> BaseWeight:
    """Pack a base weight of 4 bits for sgmv_base_product. ``codes`` uint8 [N, ceil(K / 2)], the even k in the low
    four bits; K defaults to twice their width. BASE_I4: ``scale`` [N, ceil(K / group)] of the product's dtype,
    ``zero`` uint8 alike (8 where there is none); group 32, 64 or a multiple of 128. BASE_E2M1: ``scale`` uint8
    exponents [N, ceil(K / 32)], group 32, and ``dtype`` (bfloat16 by default) says what the product takes."""
    if codes.dim() != 2 or codes.dtype != torch.uint8 or (codes.shape[1] > 1 and codes.stride(1) != 1):
        raise TypeError("codes must be row-major uint8 [N, K / 2]")
    N, index = codes.shape[0], codes.get_device()
    K = 2 * codes.shape[1] if K is None else int(K)
    if (K + 1) // 2 != codes.shape[1]:
        raise ValueError(f"codes of {K} values take {(K + 1) // 2} bytes a row, got {codes.shape[1]}")
    if format == BASE_E2M1:
        dtype = torch.bfloat16 if dtype is None else dtype
        if scale.dtype != torch.uint8:
            raise TypeError("scales of BASE_E2M1 are uint8 exponents")
    elif dtype not in (None, scale.dtype):
        raise TypeError("scales of BASE_I4 have the product's dtype")
    else:
        dtype = scale.dtype
    _int32("a weight's sizes", N, K, group, format)
    desc, sizes = _Base(), [ctypes.c_size_t() for _ in range(3)]
    _check(_lib.sgmv_base_init(N, K, int(group), int(format), _dtype_code(dtype), int(zero is not None),
                               ctypes.byref(desc), *map(ctypes.byref, sizes)), "sgmv_base_init")
    want = (N, -(-K // desc.group))
    for t, what in ((scale, "scale"), (zero, "zero")):
        if t is not None and (tuple(t.shape) != want or not t.is_contiguous() or t.get_device() != index):
            raise ValueError(f"{what} must be contiguous {list(want)} on the codes' device")
    if zero is not None and zero.dtype != torch.uint8:
        raise TypeError("zero points are uint8")
    if index < 0:
        raise ValueError("the kernels run on GPU tensors")
    parts = [torch.empty(s.value, dtype=torch.uint8, device=codes.device) if s.value else None for s in sizes]
    desc.codes, desc.scale = parts[0].data_ptr(), parts[1].data_ptr()
    desc.zero = parts[2].data_ptr() if parts[2] is not None else None
    base = BaseWeight(parts[0], parts[1] if format == BASE_E2M1 else parts[1].view(dtype), parts[2], desc, dtype)
    _check(_elsewhere(index, _lib.sgmv_base_pack, codes.data_ptr(), codes.stride(0) if N > 1 else codes.shape[1],
                      scale.data_ptr(), None if zero is None else zero.data_ptr(), base.ref), "sgmv_base_pack")
    return base


def sgmv_base_product(x: torch.Tensor, base: BaseWeight, y: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, n_split: int = 0) -> torch.Tensor:
    """y = x W^T for rows x [T, K] of the weight's dtype (strided rows are fine), into ``y`` [T, N] if given; the
    delta is then added to it. A workspace (uint8) is allocated on the current stream unless one is given;
    ``n_split`` > 0 asks for the kernel of many rows, with K split into that many ranges."""
    T, N, K, dtype, index = x.shape[0], base.N, base.K, base.dtype, base.index
    if x.dim() != 2 or x.shape[1] != K or (K > 1 and x.stride(1) != 1):
        raise ValueError(f"x must be row-major [T, {K}], got {list(x.shape)}")
    if x.dtype is not dtype or x.get_device() != index:
        raise TypeError(f"x must be {dtype} on the weight's device")
    if T > _MOST or abs(n_split) > _MOST:
        _int32("T and n_split", T, n_split)
    if y is None:
        y, ldy = x.new_empty((T, N)), N
    else:
        if tuple(y.shape) != (T, N) or y.dtype != dtype or y.get_device() != index or (N > 1 and y.stride(1) != 1):
            raise ValueError(f"y must be row-major [{T}, {N}] of {dtype} on the weight's device")
        ldy = y.stride(0) if T > 1 else N
    if index < 0:
        raise ValueError("the kernels run on GPU tensors")
    size, ptr = 0, None
    if T > base.few or n_split:
        need = ctypes.c_size_t()
        st = _lib.sgmv_base_product_workspace(T, base.ref, n_split, ctypes.byref(need))
        if st != SGMV_OK:
            _check(st, "sgmv_base_product")
        size = need.value
    if workspace is not None:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on x's device")
        size, ptr = workspace.numel() * workspace.element_size(), workspace.data_ptr()
    elif size:
        workspace = torch.empty(size, dtype=torch.uint8, device=x.device)
        ptr = workspace.data_ptr()
    args = (x.data_ptr(), x.stride(0) if T > 1 else K, T, base.ref, y.data_ptr(), ldy, n_split, ptr, size)
    call = _lib.sgmv_base_product
    st = call(*args, _stream(index)) if index == _current() else _elsewhere(index, call, *args)
    if st != SGMV_OK:
        _check(st, "sgmv_base_product")
    return y


def sgmv_base_product_workspace(T: int, base: BaseWeight, n_split: int = 0) -> int:
    """Bytes of workspace that sgmv_base_product takes for T rows."""
    _int32("T and n_split", T, n_split)
    need = ctypes.c_size_t()
    _check(_lib.sgmv_base_product_workspace(int(T), base.ref, int(n_split), ctypes.byref(need)),
           "sgmv_base_product_workspace")
    return int(need.value)


# ---------------------------------------------------------------------------------------
# rotated append
# ---------------------------------------------------------------------------------------
def sgmv_kv_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, batch: KvBatch, cache: KvCache,
                   cos_sin: torch.Tensor, interleaved: bool = False,
                   q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Write the step's keys and values [T, heads, head_dim] into the cache as sgmv_kv_write does, the keys turned
    by their positions, and turn the queries q [T, query heads, head_dim] (None: none), which are returned, in
    ``q_out`` if given (q itself: in place). ``cos_sin`` float32 [positions, rotary]: rotary / 2 cosines and then as
    many sines of each position's angles; the first ``rotary`` values of a row (a multiple of 16) are turned, in
    pairs (i, i + rotary / 2) or, ``interleaved``, (2 i, 2 i + 1). Rows of no sequence and those at negative
    positions are not written: in a ``q_out`` that the call allocates they are whatever the memory held."""
    T, index, dtype = batch.T, cache.index, k.dtype
    kt, kh = _rows3(k, T, cache.heads, cache, "k")
    vt, vh = _rows3(v, T, cache.heads, cache, "v")
    if v.dtype is not dtype:
        raise TypeError("k and v must share a dtype")
    code = _ROWS.get(dtype)
    if code is None:
        _dtype_code(dtype)  # says which
    if cos_sin.dim() != 2 or cos_sin.dtype is not torch.float32 or cos_sin.get_device() != index or (
            cos_sin.stride(1) != 1):
        raise TypeError("cos_sin must be row-major float32 [positions, rotary] on the cache's device")
    positions, rotary = cos_sin.shape
    if positions > _MOST or rotary > _MOST:
        _int32("positions and rotary", positions, rotary)
    heads = qt = qh = ot = oh = 0
    qp = op = 0
    if q is not None:
        qt, qh = _rows3(q, T, None, cache, "q")
        if q.dtype is not dtype:
            raise TypeError("q must have k's dtype")
        heads, qp = q.shape[1], q.data_ptr()
        if q_out is None:
            q_out = _like(q, memory_format=_dense)
            ot, oh = heads * cache.head_dim, cache.head_dim
        else:
            ot, oh = _rows3(q_out, T, heads, cache, "q_out")
            if q_out.dtype is not dtype:
                raise TypeError("q_out must have q's dtype")
        op = q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out goes with q")
    if batch.index != index or index < 0:
        _on_gpu(batch, cache)  # says which
    r = _pack_rotation(cos_sin.data_ptr(), cos_sin.stride(0) if positions > 1 else rotary, positions, rotary,
                       1 if interleaved else 0, heads, qp, op, qt, qh, ot, oh)
    args = (r, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, code, batch.ref, cache.ref)
    call = _lib.sgmv_kv_append
    st = call(*args, _stream(index)) if index == _current() else _elsewhere(index, call, *args)
    if st != SGMV_OK:
        _check(st, "sgmv_kv_append")
    return q_out
