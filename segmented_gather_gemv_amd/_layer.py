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
from dataclasses import dataclass, field
from typing import NamedTuple, Optional

import torch

from . import SGMV_OK, _check, _dtype_code, _lib, _raw_stream
from ._serving import KV_E4M3, KV_I8, KvBatch, KvCache, _MOST, _dense3, _int32, _KvBatch, _KvCache, _on_gpu, _rows3

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


def _bind():
    i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    P = ctypes.POINTER
    B = P(_Base)
    for name, args in {
        "sgmv_rms_norm": [P(_Norm), vp],
        "sgmv_base_init": [i32, i32, i32, i32, i32, i32, B, P(sz), P(sz), P(sz)],
        "sgmv_base_pack": [vp, i64, vp, vp, B, vp],
        "sgmv_base_product_workspace": [i32, B, i32, P(sz)],
        "sgmv_base_product": [vp, i64, i32, B, vp, i64, i32, vp, sz, vp],
        "sgmv_kv_append": [P(_Rotation), vp, i64, i64, vp, i64, i64, i32, P(_KvBatch), P(_KvCache), vp],
    }.items():
        f = getattr(_lib, name)
        f.argtypes, f.restype = args, ctypes.c_int


_bind()


def _launch(where: str, index: int, call, *args):
    """The call on the current stream of GPU `index`, which is made the current one if it is not (the default
    stream's handle is that of the current GPU)."""
    if index == torch._C._cuda_getDevice():
        st = call(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = call(*args, _raw_stream(index))
    if st != SGMV_OK:
        _check(st, where)


# ---------------------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------------------
class Normed(NamedTuple):
    out: Optional[torch.Tensor]       # as x, or None
    residual: Optional[torch.Tensor]  # x + residual, or None
    codes: Optional[torch.Tensor]     # float8_e4m3fn or int8, or None
    scale: Optional[torch.Tensor]     # float32, of each row


def _strides(t: torch.Tensor, shape, index: int, what: str):
    """Token and head strides of rows [T, width] or [T, heads, width]."""
    if t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")
    st = t.stride()
    if shape[-1] > 1 and st[-1] != 1:
        raise ValueError(f"{what} must be contiguous over the last dimension")
    if t.get_device() != index:
        raise ValueError(f"{what} must be on x's device")
    T, W, heads = shape[0], shape[-1], shape[1] if len(shape) == 3 else 1
    head = st[1] if heads > 1 else W
    # a stride of a single token says nothing
    return (st[0] if T > 1 else heads * head), head


def sgmv_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                  residual: Optional[torch.Tensor] = None, quantise: Optional[torch.dtype] = None,
                  want_out: bool = True, out: Optional[torch.Tensor] = None,
                  residual_out: Optional[torch.Tensor] = None, codes: Optional[torch.Tensor] = None,
                  scale: Optional[torch.Tensor] = None) -> Normed:
    """Root-mean-square norm of rows x [T, width], or [T, heads, width] head by head (strided views are fine),
    times ``weight``; of x + ``residual`` where one is given, which is returned too. ``quantise``
    (float8_e4m3fn or int8) asks for the normed rows as codes with one scale per row as well, ``want_out=False``
    for those alone. Outputs are allocated unless given; ``out`` and ``residual_out`` may be x or residual
    themselves."""
    shape, dtype, index = x.shape, x.dtype, x.get_device()
    if len(shape) not in (2, 3):
        raise ValueError(f"x must be [T, width] or [T, heads, width], got {list(shape)}")
    code = _dtype_code(dtype)
    W, heads = shape[-1], shape[1] if len(shape) == 3 else 1
    _int32("T, heads and width", *shape)
    if weight.shape != (W,) or weight.dtype != dtype or weight.get_device() != index or (W > 1 and weight.stride(0) != 1):
        raise TypeError(f"weight must be {W} contiguous {dtype} entries on x's device")
    a = _Norm(x=x.data_ptr(), weight=weight.data_ptr(), T=shape[0], heads=heads, width=W, dtype=code, eps=eps)
    a.ldx_token, a.ldx_head = _strides(x, shape, index, "x")
    dense = (heads * W, W)
    if residual is not None:
        if residual.dtype != dtype:
            raise TypeError("residual must have x's dtype")
        a.ldr_token, a.ldr_head = _strides(residual, shape, index, "residual")
        a.residual = residual.data_ptr()
        a.lds_token, a.lds_head = dense
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=dtype, device=x.device)
        else:
            if residual_out.dtype != dtype:
                raise TypeError("residual_out must have x's dtype")
            a.lds_token, a.lds_head = _strides(residual_out, shape, index, "residual_out")
        a.residual_out = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out goes with a residual")
    if out is not None:
        if out.dtype != dtype:
            raise TypeError("out must have x's dtype")
        a.ldo_token, a.ldo_head = _strides(out, shape, index, "out")
        a.out = out.data_ptr()
    elif want_out:
        out = torch.empty(shape, dtype=dtype, device=x.device)
        a.ldo_token, a.ldo_head = dense
        a.out = out.data_ptr()
    if quantise is not None:
        if quantise not in _CODES:
            raise TypeError(f"codes are float8_e4m3fn or int8, got {quantise}")
        a.format = _CODES[quantise]
        a.ldc_token, a.ldc_head = dense
        if codes is None:
            codes = torch.empty(shape, dtype=quantise, device=x.device)
        else:
            if codes.dtype != quantise:
                raise TypeError(f"codes must be {quantise}")
            a.ldc_token, a.ldc_head = _strides(codes, shape, index, "codes")
        if scale is None:
            scale = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
        elif scale.shape != shape[:-1] or scale.dtype != torch.float32 or not scale.is_contiguous() or (
                scale.get_device() != index):
            raise TypeError("scale must be a contiguous float32 tensor of one entry per row on x's device")
        a.codes, a.scale = codes.data_ptr(), scale.data_ptr()
    elif codes is not None or scale is not None:
        raise ValueError("codes and scale go with quantise")
    elif out is None:
        raise ValueError("nothing to compute: neither out nor codes are wanted")
    if index < 0:
        raise ValueError("the kernels run on GPU tensors")
    _launch("sgmv_rms_norm", index, _lib.sgmv_rms_norm, ctypes.byref(a))
    return Normed(out, residual_out, codes, scale)


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

    def __post_init__(self):
        self.N, self.K, self.group, self.format = self.desc.N, self.desc.K, self.desc.group, self.desc.format
        self.ref, self.index = ctypes.byref(self.desc), self.codes.get_device()


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
    _launch("sgmv_base_pack", index, _lib.sgmv_base_pack, codes.data_ptr(),
            codes.stride(0) if N > 1 else codes.shape[1], scale.data_ptr(),
            None if zero is None else zero.data_ptr(), base.ref)
    return base


def sgmv_base_product(x: torch.Tensor, base: BaseWeight, y: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, n_split: int = 0) -> torch.Tensor:
    """y = x W^T for rows x [T, K] of the weight's dtype (strided rows are fine), into ``y`` [T, N] if given; the
    delta is then added to it. A workspace (uint8) is allocated on the current stream unless one is given;
    ``n_split`` > 0 asks for the kernel of many rows, with K split into that many ranges."""
    T, N, K, dtype, index = x.shape[0], base.N, base.K, base.dtype, base.index
    if x.dim() != 2 or x.shape[1] != K or (K > 1 and x.stride(1) != 1):
        raise ValueError(f"x must be row-major [T, {K}], got {list(x.shape)}")
    if x.dtype != dtype or x.get_device() != index:
        raise TypeError(f"x must be {dtype} on the weight's device")
    if T > _MOST or abs(n_split) > _MOST:
        _int32("T and n_split", T, n_split)
    if y is None:
        y, ldy = torch.empty((T, N), dtype=dtype, device=x.device), N
    else:
        if tuple(y.shape) != (T, N) or y.dtype != dtype or y.get_device() != index or (N > 1 and y.stride(1) != 1):
            raise ValueError(f"y must be row-major [{T}, {N}] of {dtype} on the weight's device")
        ldy = y.stride(0) if T > 1 else N
    if index < 0:
        raise ValueError("the kernels run on GPU tensors")
    size, ptr = 0, None
    if T > 32 or n_split:  # (none for fewer rows)
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
    _launch("sgmv_base_product", index, _lib.sgmv_base_product, x.data_ptr(), x.stride(0) if T > 1 else K, T,
            base.ref, y.data_ptr(), ldy, n_split, ptr, size)
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
    many sines of each position's angles; the first ``rotary`` values of a row are turned, in pairs (i,
    i + rotary / 2) or, ``interleaved``, (2 i, 2 i + 1)."""
    kt, kh = _rows3(k, batch.T, cache.heads, cache, "k")
    vt, vh = _rows3(v, batch.T, cache.heads, cache, "v")
    dtype = k.dtype
    if v.dtype != dtype:
        raise TypeError("k and v must share a dtype")
    code = _dtype_code(dtype)
    if cos_sin.dim() != 2 or cos_sin.dtype != torch.float32 or cos_sin.stride(1) != 1 or (
            cos_sin.get_device() != cache.index):
        raise TypeError("cos_sin must be row-major float32 [positions, rotary] on the cache's device")
    positions, rotary = cos_sin.shape
    _int32("positions and rotary", positions, rotary)
    r = _Rotation(cos_sin.data_ptr(), cos_sin.stride(0) if positions > 1 else rotary, positions, rotary,
                  1 if interleaved else 0)
    if q is not None:
        r.ldq_token, r.ldq_head = _rows3(q, batch.T, None, cache, "q")
        if q.dtype != dtype:
            raise TypeError("q must have k's dtype")
        r.heads, r.q = q.shape[1], q.data_ptr()
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=dtype, device=q.device)
            r.ldo_token, r.ldo_head = _dense3(r.heads, cache)
        else:
            r.ldo_token, r.ldo_head = _rows3(q_out, batch.T, r.heads, cache, "q_out")
            if q_out.dtype != dtype:
                raise TypeError("q_out must have q's dtype")
        r.q_out = q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out goes with q")
    _on_gpu(batch, cache)
    _launch("sgmv_kv_append", cache.index, _lib.sgmv_kv_append, ctypes.byref(r), k.data_ptr(), kt, kh, v.data_ptr(),
            vt, vh, code, batch.ref, cache.ref)
    return q_out
