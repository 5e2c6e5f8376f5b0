"""Binding of the paged key/value cache, its attention and the draft check (include/sgmv.h);
imported by the package, whose names these are. Argument marshalling only; calls for serving, which
autograd does not see: what they return carries no gradient, whatever their inputs require.

    sgmv_kv_init(pages, page_size, heads, head_dim, format)  -> KvCache
    sgmv_kv_batch(q_start, kv_len, page_table, T, max_q, max_kv) -> KvBatch
    sgmv_kv_write(k, v, batch, cache)                        -> None (cache updated in place)
    sgmv_kv_read(batch, cache, out_start, rows, dtype)       -> k, v
    sgmv_kv_attention(q, batch, cache)                       -> out, lse
    sgmv_verify_drafts(target, draft, ids, start, ...)       -> tokens, accepted
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass, field
from typing import Optional, Tuple, Union

import torch

from . import SGMV_OK, _check, _dtype_code, _lib, _raw_stream

KV_F32, KV_BF16, KV_E4M3, KV_I8 = range(4)
KV_GROUP = 16
KV_MAX_PAGE = 4096
KV_MAX_HEAD_DIM = 256
KV_MAX_HEADS = 1024
KV_MAX_B = 65536
KV_MAX_SPLITS = 64

_FORMATS = {torch.float32: KV_F32, torch.bfloat16: KV_BF16, torch.float8_e4m3fn: KV_E4M3,
            torch.int8: KV_I8}
_DTYPES = {f: d for d, f in _FORMATS.items()}


class _KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("format", ctypes.c_int32)]


class _KvBatch(ctypes.Structure):
    _fields_ = [("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("ldp", ctypes.c_int64),
                ("table_pages", ctypes.c_int32), ("B", ctypes.c_int32), ("T", ctypes.c_int32),
                ("max_q", ctypes.c_int32), ("max_kv", ctypes.c_int32)]


class _Attention(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("ldq_token", ctypes.c_int64), ("ldq_head", ctypes.c_int64),
                ("ldo_token", ctypes.c_int64), ("ldo_head", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("window", ctypes.c_int32), ("n_split", ctypes.c_int32)]


_MOST = 2 ** 31 - 1


def _int32(what: str, *values):
    """ctypes would cut them to 32 bits."""
    for v in values:
        if not -_MOST <= v <= _MOST:
            raise ValueError(f"{what} must fit in 32 bits, got {v}")


def _bind():
    i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    P = ctypes.POINTER
    C, S, A = P(_KvCache), P(_KvBatch), P(_Attention)
    for name, args in {
        "sgmv_kv_init": [i32, i32, i32, i32, i32, C, P(sz), P(sz)],
        "sgmv_kv_write": [vp, i64, i64, vp, i64, i64, i32, S, C, vp],
        "sgmv_kv_read": [S, C, vp, i32, vp, i64, i64, vp, i64, i64, i32, vp],
        "sgmv_kv_attention_workspace": [A, S, C, P(sz)],
        "sgmv_kv_attention": [A, S, C, vp, sz, vp],
        "sgmv_verify_drafts": [vp, i64, vp, i64, i32, i32, vp, vp, i32, i32, i32, vp, vp, vp,
                               i64, vp, vp, sz, vp],
    }.items():
        f = getattr(_lib, name)
        f.argtypes, f.restype = args, ctypes.c_int
    _lib.sgmv_verify_drafts_workspace.argtypes = [i32, i32]
    _lib.sgmv_verify_drafts_workspace.restype = sz


_bind()


# ---------------------------------------------------------------------------------------
# cache and batch
# ---------------------------------------------------------------------------------------
@dataclass
class KvCache:
    k: torch.Tensor                  # [pages, heads, page_size / 16, D / c, 16, c]
    v: torch.Tensor                  # [pages, heads, page_size / 16, D, 16]
    k_scale: Optional[torch.Tensor]  # fp32 [pages, heads, page_size], 8-bit formats
    v_scale: Optional[torch.Tensor]
    desc: _KvCache
    ref: object = field(init=False, repr=False)     # what the library takes
    index: int = field(init=False, repr=False)      # of the GPU, -1: not on one

    def __post_init__(self):
        d = self.desc
        self.pages, self.page_size, self.heads, self.head_dim = (d.pages, d.page_size, d.heads,
                                                                 d.head_dim)
        self.dtype, self.ref, self.index = self.k.dtype, ctypes.byref(d), self.k.get_device()


def _kv_shapes(desc: _KvCache, elem: int):
    c, g = 16 // elem, desc.page_size // KV_GROUP
    return ((desc.pages, desc.heads, g, desc.head_dim // c, KV_GROUP, c),
            (desc.pages, desc.heads, g, desc.head_dim, KV_GROUP),
            (desc.pages, desc.heads, desc.page_size))


def _kv_desc(pages, page_size, heads, head_dim, dtype) -> _KvCache:
    if dtype not in _FORMATS:
        raise TypeError(f"a cache holds float32, bfloat16, float8_e4m3fn or int8, got {dtype}")
    _int32("a cache's sizes", pages, page_size, heads, head_dim)
    desc, data, scale = _KvCache(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(_lib.sgmv_kv_init(int(pages), int(page_size), int(heads), int(head_dim),
                             _FORMATS[dtype], ctypes.byref(desc), ctypes.byref(data),
                             ctypes.byref(scale)), "sgmv_kv_init")
    return desc


def sgmv_kv_wrap(k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None) -> KvCache:
    """A cache made of existing tensors in the library's layout (KvCache lists the shapes)."""
    if k.dim() != 6 or v.dim() != 5:
        raise ValueError("k must be [pages, heads, page_size/16, D/c, 16, c] and v "
                         "[pages, heads, page_size/16, D, 16]")
    desc = _kv_desc(v.shape[0], v.shape[2] * KV_GROUP, v.shape[1], v.shape[3], k.dtype)
    ks, vs, ss = _kv_shapes(desc, k.element_size())
    scaled = desc.format in (KV_E4M3, KV_I8)
    if tuple(k.shape) != ks or tuple(v.shape) != vs or v.dtype != k.dtype:
        raise ValueError(f"k must be {ks} and v {vs}, both {k.dtype}")
    if scaled != (k_scale is not None) or scaled != (v_scale is not None):
        raise ValueError("scales go with the 8-bit formats, and only with them")
    for t, shape in ((k_scale, ss), (v_scale, ss)) if scaled else ():
        if tuple(t.shape) != shape or t.dtype != torch.float32:
            raise ValueError(f"scales must be float32 {shape}")
    for t in (k, v, k_scale, v_scale):
        if t is not None and (not t.is_contiguous() or t.device != k.device):
            raise ValueError("a cache's tensors must be contiguous and on one device")
    desc.k, desc.v = k.data_ptr(), v.data_ptr()
    if scaled:
        desc.k_scale, desc.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
    return KvCache(k, v, k_scale, v_scale, desc)


def sgmv_kv_init(pages: int, page_size: int, heads: int, head_dim: int,
                 dtype: torch.dtype = torch.bfloat16,
                 device: Union[str, torch.device] = "cuda") -> KvCache:
    """Allocate a cache (zeroed): float32 and bfloat16 hold rows of that type as they are,
    float8_e4m3fn and int8 codes with one fp32 scale per token and head."""
    desc = _kv_desc(pages, page_size, heads, head_dim, dtype)
    elem = torch.empty(0, dtype=dtype).element_size()
    ks, vs, ss = _kv_shapes(desc, elem)
    raw = torch.int8 if desc.format == KV_E4M3 else dtype
    k, v = (torch.zeros(s, dtype=raw, device=device).view(dtype) for s in (ks, vs))
    scale = [None, None]
    if elem == 1:
        scale = [torch.zeros(ss, dtype=torch.float32, device=device) for _ in range(2)]
    return sgmv_kv_wrap(k, v, *scale)


@dataclass
class KvBatch:
    q_start: torch.Tensor     # int32 [B + 1]
    kv_len: torch.Tensor      # int32 [B]
    page_table: torch.Tensor  # int32 [B, table_pages]
    desc: _KvBatch
    ref: object = field(init=False, repr=False)
    index: int = field(init=False, repr=False)

    def __post_init__(self):
        self.B, self.T = self.desc.B, self.desc.T
        self.ref, self.index = ctypes.byref(self.desc), self.kv_len.get_device()


def sgmv_kv_batch(q_start: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor, T: int,
                  max_q: int, max_kv: int) -> KvBatch:
    """The sequences of a step (device tensors that later calls read again: refill them in
    place for another step of the same sizes). T rows of new tokens, at most max_q of one
    sequence, at most max_kv tokens in one sequence, the new ones included. Rows that q_start
    leaves over (a step padded to T rows) are neither read nor written."""
    for t, d in ((q_start, 1), (kv_len, 1), (page_table, 2)):
        if t.dtype != torch.int32 or t.dim() != d or t.device != kv_len.device:
            raise TypeError("q_start [B + 1], kv_len [B] and page_table [B, pages] must be int32 "
                            "tensors on one device")
    _int32("T, max_q and max_kv", T, max_q, max_kv)
    B = kv_len.numel()
    if q_start.numel() != B + 1 or page_table.shape[0] != B:
        raise ValueError("q_start needs B + 1 entries and page_table B rows")
    if not q_start.is_contiguous() or not kv_len.is_contiguous() or (
            page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("q_start, kv_len and the rows of page_table must be contiguous")
    cols = page_table.shape[1]
    ldp = page_table.stride(0) if B > 1 else cols
    if ldp < cols:
        raise ValueError("the rows of page_table must not share memory (an expanded table: copy it)")
    desc = _KvBatch(q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), ldp, cols, B,
                    int(T), int(max_q), int(max_kv))
    return KvBatch(q_start, kv_len, page_table, desc)


def _rows3(t: torch.Tensor, n: int, heads: Optional[int], cache: KvCache, what: str):
    """Checks rows [n, heads, head_dim]; returns their token and head strides."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != n or shape[2] != cache.head_dim or (
            heads is not None and shape[1] != heads):
        raise ValueError(f"{what} must be [{n}, {'heads' if heads is None else heads}, "
                         f"{cache.head_dim}], got {tuple(shape)}")
    st = t.stride()
    if st[2] != 1:
        raise ValueError(f"{what} must be contiguous over the head dimension")
    if t.get_device() != cache.index:
        raise ValueError(f"{what} must be on the cache's device")
    # a stride of a single token or head says nothing
    return (st[0] if n > 1 else shape[1] * shape[2] + abs(st[1]) * shape[1],
            st[1] if shape[1] > 1 else shape[2])


def _dense3(heads: int, cache: KvCache):
    """The strides of rows that a call allocates itself."""
    return heads * cache.head_dim, cache.head_dim


def _on_gpu(batch: KvBatch, cache: KvCache):
    if batch.index != cache.index:
        raise ValueError("the batch must be on the cache's device")
    if cache.index < 0:
        raise ValueError("the kernels run on GPU tensors")


# ---------------------------------------------------------------------------------------
# write, read, attention
# ---------------------------------------------------------------------------------------
def sgmv_kv_write(k: torch.Tensor, v: torch.Tensor, batch: KvBatch, cache: KvCache) -> None:
    """Write the step's keys and values [T, heads, head_dim] (strided views are fine) into the
    cache, quantised to its format."""
    kt, kh = _rows3(k, batch.T, cache.heads, cache, "k")
    vt, vh = _rows3(v, batch.T, cache.heads, cache, "v")
    if v.dtype != k.dtype:
        raise TypeError("k and v must share a dtype")
    dtype = _dtype_code(k.dtype)
    _on_gpu(batch, cache)
    st = _lib.sgmv_kv_write(k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, dtype, batch.ref,
                            cache.ref, _raw_stream(cache.index))
    if st != SGMV_OK:
        _check(st, "sgmv_kv_write")


def sgmv_kv_read(batch: KvBatch, cache: KvCache, out_start: torch.Tensor, rows: int,
                 dtype: torch.dtype = torch.bfloat16, k: Optional[torch.Tensor] = None,
                 v: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The last out_start[b + 1] - out_start[b] tokens of each sequence, as rows
    [rows, heads, head_dim]: out_start = q_start reads the step's new tokens back, running sums
    of kv_len whole sequences. Into k and v if given."""
    rows, heads = int(rows), cache.heads
    _int32("rows", rows)
    if out_start.dtype != torch.int32 or out_start.numel() != batch.B + 1 or (
            not out_start.is_contiguous() or out_start.get_device() != cache.index):
        raise TypeError("out_start must be B + 1 contiguous int32 entries on the cache's device")
    code = _dtype_code(dtype)
    (kt, kh) = (vt, vh) = _dense3(heads, cache)
    if k is None:
        k = torch.empty((rows, heads, cache.head_dim), dtype=dtype, device=out_start.device)
    else:
        kt, kh = _rows3(k, rows, heads, cache, "k")
    if v is None:
        v = torch.empty((rows, heads, cache.head_dim), dtype=dtype, device=out_start.device)
    else:
        vt, vh = _rows3(v, rows, heads, cache, "v")
    if k.dtype != dtype or v.dtype != dtype:
        raise TypeError(f"k and v must be {dtype}")
    _on_gpu(batch, cache)
    st = _lib.sgmv_kv_read(batch.ref, cache.ref, out_start.data_ptr(), rows, k.data_ptr(), kt, kh,
                           v.data_ptr(), vt, vh, code, _raw_stream(cache.index))
    if st != SGMV_OK:
        _check(st, "sgmv_kv_read")
    return k, v


def sgmv_kv_attention(q: torch.Tensor, batch: KvBatch, cache: KvCache,
                      scale: Optional[float] = None, window: int = 0,
                      out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      n_split: int = 0, workspace: Optional[torch.Tensor] = None
                      ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of the step's queries [T, query heads, head_dim] over the cache, which already
    holds the step's keys and values: causal, with ``window`` > 0 over the last ``window``
    tokens only. Returns the output and the rows' log-sum-exp [T, query heads] fp32. ``scale``
    defaults to head_dim ** -0.5. A workspace (uint8) is allocated on the current stream
    unless one is given. No gradient flows through the call."""
    T, D = batch.T, cache.head_dim
    if abs(window) > _MOST or abs(n_split) > _MOST:
        _int32("window and n_split", window, n_split)
    qt, qh = _rows3(q, T, None, cache, "q")
    heads, dtype = q.shape[1], q.dtype
    code = _dtype_code(dtype)
    if out is None:
        out = torch.empty((T, heads, D), dtype=dtype, device=q.device)
        ot, oh = _dense3(heads, cache)
    else:
        ot, oh = _rows3(out, T, heads, cache, "out")
        if out.dtype != dtype:
            raise TypeError("out must have q's dtype")
    if lse is None:
        lse = torch.empty((T, heads), dtype=torch.float32, device=q.device)
    elif tuple(lse.shape) != (T, heads) or lse.dtype != torch.float32 or (
            not lse.is_contiguous() or lse.get_device() != cache.index):
        raise TypeError("lse must be a contiguous float32 tensor of one entry per token and head")
    a = _Attention(q.data_ptr(), out.data_ptr(), lse.data_ptr(), qt, qh, ot, oh, heads, code,
                   D ** -0.5 if scale is None else scale, window, n_split)
    ref, need = ctypes.byref(a), ctypes.c_size_t()
    st = _lib.sgmv_kv_attention_workspace(ref, batch.ref, cache.ref, ctypes.byref(need))
    if st != SGMV_OK:
        _check(st, "sgmv_kv_attention")
    _on_gpu(batch, cache)
    size, ptr = need.value, None
    if workspace is not None:
        if workspace.get_device() != cache.index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on q's device")
        size = workspace.numel() * workspace.element_size()
        ptr = workspace.data_ptr()
    elif size:
        workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
        ptr = workspace.data_ptr()
    st = _lib.sgmv_kv_attention(ref, batch.ref, cache.ref, ptr, size, _raw_stream(cache.index))
    if st != SGMV_OK:
        _check(st, "sgmv_kv_attention")
    return out, lse


def sgmv_kv_attention_workspace(q_heads: int, dtype: torch.dtype, batch: KvBatch, cache: KvCache,
                                window: int = 0, n_split: int = 0) -> int:
    """Bytes of workspace that sgmv_kv_attention takes for such a call."""
    _int32("q_heads, window and n_split", q_heads, window, n_split)
    a = _Attention(None, None, None, 0, 0, 0, 0, int(q_heads), _dtype_code(dtype), 1.0, int(window),
                   int(n_split))
    need = ctypes.c_size_t()
    _check(_lib.sgmv_kv_attention_workspace(ctypes.byref(a), batch.ref, cache.ref,
                                            ctypes.byref(need)), "sgmv_kv_attention_workspace")
    return int(need.value)


# ---------------------------------------------------------------------------------------
# drafts
# ---------------------------------------------------------------------------------------
def _entries(t: torch.Tensor, n: int, dtype: torch.dtype, index: int, what: str):
    if t.dtype != dtype or t.numel() != n or t.get_device() != index or not t.is_contiguous():
        raise TypeError(f"{what} must be {n} contiguous {dtype} entries on target's device")


def sgmv_verify_drafts(target: torch.Tensor, draft: Optional[torch.Tensor],
                       draft_ids: torch.Tensor, draft_start: torch.Tensor,
                       accept_u: torch.Tensor, sample_u: torch.Tensor, max_drafts: int,
                       tokens: Optional[torch.Tensor] = None,
                       accepted: Optional[torch.Tensor] = None
                       ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Check the N drafted tokens of B sequences against the target's probabilities
    ``target`` [N + B, vocab] (a sequence's n + 1 rows follow each other), with the drafter's
    probabilities ``draft`` [N, vocab] or None for certain drafts, and the uniform numbers
    given. Returns tokens [B, max_drafts + 1] (those taken, the one drawn, then -1) and how
    many were taken [B], both int32."""
    B, N, shape = sample_u.numel(), draft_ids.numel(), target.shape
    dev, dtype = target.get_device(), target.dtype
    if len(shape) != 2 or shape[0] != N + B or shape[1] < 1 or (
            shape[1] > 1 and target.stride(1) != 1):
        raise ValueError(f"target must be row-major [{N + B}, vocab], got {tuple(shape)}")
    V = shape[1]
    if draft is not None:
        if draft.dim() != 2 or tuple(draft.shape) != (N, V) or (V > 1 and draft.stride(1) != 1):
            raise ValueError(f"draft must be row-major [{N}, {V}], got {tuple(draft.shape)}")
        if draft.dtype != dtype or draft.get_device() != dev:
            raise TypeError("draft must have target's dtype and device")
    _entries(draft_ids, N, torch.int32, dev, "draft_ids")
    _entries(draft_start, B + 1, torch.int32, dev, "draft_start")
    _entries(accept_u, N, torch.float32, dev, "accept_u")
    _entries(sample_u, B, torch.float32, dev, "sample_u")
    _int32("vocab and max_drafts", V, max_drafts)
    if max_drafts < 0:
        raise ValueError("max_drafts must not be negative")
    if tokens is None:
        tokens = torch.empty((B, max_drafts + 1), dtype=torch.int32, device=target.device)
    elif tokens.dtype != torch.int32 or tuple(tokens.shape) != (B, max_drafts + 1) or (
            tokens.get_device() != dev or (max_drafts > 0 and tokens.stride(1) != 1)):
        raise ValueError("tokens must be row-major int32 [B, max_drafts + 1] on target's device")
    if accepted is None:
        accepted = torch.empty(B, dtype=torch.int32, device=target.device)
    elif accepted.dtype != torch.int32 or accepted.numel() != B or (
            accepted.get_device() != dev or not accepted.is_contiguous()):
        raise ValueError("accepted must be B contiguous int32 entries on target's device")
    code = _dtype_code(dtype)
    if dev < 0:
        raise ValueError("the kernels run on GPU tensors")
    size = _lib.sgmv_verify_drafts_workspace(B, V)
    workspace = torch.empty(max(size, 1), dtype=torch.uint8, device=target.device)
    no_draft = draft is None or N == 0
    st = _lib.sgmv_verify_drafts(
        target.data_ptr(), target.stride(0) if N + B > 1 else V,
        None if no_draft else draft.data_ptr(), V if no_draft or N == 1 else draft.stride(0), V, code,
        draft_ids.data_ptr(), draft_start.data_ptr(), B, N, int(max_drafts), accept_u.data_ptr(),
        sample_u.data_ptr(), tokens.data_ptr(),
        tokens.stride(0) if B > 1 else max_drafts + 1, accepted.data_ptr(),
        workspace.data_ptr(), size, _raw_stream(dev))
    if st != SGMV_OK:
        _check(st, "sgmv_verify_drafts")
    return tokens, accepted
