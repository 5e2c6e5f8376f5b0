"""CPU tests of the norm, the base product and the rotated append: the oracle's pins, sizes, and the refusals of the
C-ABI and of the binding. Nothing is launched."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import segmented_gather_gemv_amd as sg
from oracle import layer_oracle as lo
from segmented_gather_gemv_amd import _layer as ly
from segmented_gather_gemv_amd import _serving as sv

E, UNS, OK = sg.SGMV_EINVAL, sg.SGMV_EUNSUPPORTED, sg.SGMV_OK
I32 = lambda *v: torch.tensor(v, dtype=torch.int32)


# ---- the oracle's pins ----------------------------------------------------------------
def test_norm_by_hand():
    out, h, codes, scale = lo.rms_norm([[3.0, 4.0]], [1.0, 2.0], 12.0 - 0.25, [[0.0, -3.0]], "i8")
    root = math.sqrt((9 + 1) / 2 + 11.75)
    assert h.tolist() == [[3.0, 1.0]] and np.allclose(out, [[3 / root, 2 / root]])
    assert codes.tolist() == [[127, 85]] and np.isclose(scale[0], 3 / 127 / root)  # 84.67
    out, _, codes, scale = lo.rms_norm([[0.0, 0.0]], [1.0, 1.0], 1e-6, None, "e4m3")
    assert (out == 0).all() and (codes == 0).all() and scale[0] == 0


def test_base_weight_by_hand():
    codes = np.array([[0x21, 0x0F], [0x98, 0x07]], np.uint8)
    assert lo.unpack(codes, 3).tolist() == [[1, 2, 15], [8, 9, 7]]
    v, a = lo.base_weight(codes, 3, np.array([[2.0, 0.5], [1.0, 4.0]]), np.array([[1, 3], [8, 0]]), 2, "i4")
    assert v.tolist() == [[0, 2, 6], [0, 1, 28]] and a.tolist() == [[4, 6, 9], [16, 17, 28]]
    v, _ = lo.base_weight(codes, 3, np.array([[2.0], [1.0]]), None, 4, "i4")
    assert v.tolist() == [[-14, -12, 14], [0, 1, -1]]
    v, a = lo.base_weight(codes, 3, np.array([[127], [129]]), None, 32, "e2m1")
    assert v.tolist() == [[0.5, 1, -6], [0, -2, 24]] and a.tolist() == [[0.5, 1, 6], [0, 2, 24]]


def test_rotate_by_hand_and_as_complex_numbers():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    c, s = np.array([[0.0, 1.0]]), np.array([[1.0, 0.0]])
    assert lo.rotate(x, c, s, False).tolist() == [[[-3.0, 2.0, 1.0, 4.0, 9.0]]]
    assert lo.rotate(x, c, s, True).tolist() == [[[-2.0, 1.0, 3.0, 4.0, 9.0]]]
    g = np.random.default_rng(0)
    x, angle = g.normal(size=(5, 2, 12)), g.normal(size=(5, 4))
    for inter in (False, True):
        a, b = (slice(0, 8, 2), slice(1, 8, 2)) if inter else (slice(0, 4), slice(4, 8))
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * angle)[:, None]
        y = lo.rotate(x, np.cos(angle), np.sin(angle), inter)
        assert np.allclose(y[..., a], z.real, atol=1e-6) and np.allclose(y[..., b], z.imag, atol=1e-6)
        assert np.array_equal(y[..., 8:], x[..., 8:].astype(np.float32))


def test_constants_match_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(sg.__file__)), "include", "sgmv.h")).read()
    defs = dict(re.findall(r"#define SGMV_([A-Z_0-9]+) (\d+)", text))
    for name in ("MAX_NORM_WIDTH", "BASE_MAX_SIZE", "BASE_MAX_SPLITS"):
        assert int(defs[name]) == getattr(sg, name)
    for name in ("BASE_I4", "BASE_E2M1"):
        assert re.search(r"SGMV_%s = %d\b" % (name, getattr(sg, name)), text)


# ---- sizes ----------------------------------------------------------------------------
def _init(N=40, K=300, group=128, format=sg.BASE_I4, dtype=sg.SGMV_BF16, zero=0):
    b, sizes = ly._Base(), [ctypes.c_size_t() for _ in range(3)]
    st = sg.library().sgmv_base_init(N, K, group, format, dtype, zero, ctypes.byref(b), *map(ctypes.byref, sizes))
    return st, b, [s.value for s in sizes]


def test_base_sizes():
    # 3 tiles of 16 n, 3 blocks of 128 k (1 KB each)
    assert _init()[0] == OK and _init()[2] == [9 * 1024, 3 * 3 * 16 * 2, 0]
    assert _init(zero=1, dtype=sg.SGMV_F32)[2] == [9 * 1024, 3 * 3 * 16 * 4, 3 * 3 * 16]
    assert _init(group=32, zero=1)[2] == [9 * 1024, 3 * 3 * 16 * 4 * 2, 3 * 3 * 16 * 4]
    assert _init(group=64)[2] == [9 * 1024, 3 * 3 * 16 * 2 * 2, 0]
    assert _init(group=256)[2] == [9 * 1024, 3 * 2 * 16 * 2, 0]
    assert _init(group=512)[2] == [9 * 1024, 3 * 1 * 16 * 2, 0]
    assert _init(group=32, format=sg.BASE_E2M1)[2] == [9 * 1024, 3 * 3 * 16 * 4, 0]
    assert _init(N=1, K=1)[2] == [1024, 32, 0]


BAD_BASES = [(dict(N=0), E), (dict(K=0), E), (dict(group=0), E), (dict(format=2), E), (dict(format=-1), E),
             (dict(dtype=2), E), (dict(zero=2), E), (dict(group=16), UNS), (dict(group=96), UNS), (dict(group=192), UNS),
             (dict(N=4194305), UNS), (dict(K=4194305), UNS), (dict(format=1), E), (dict(format=1, group=64), E),
             (dict(format=1, group=32, zero=1), E)]


@pytest.mark.parametrize("kw,status", BAD_BASES)
def test_base_init_refuses(kw, status):
    assert _init(**kw)[0] == status
    lib, b, s = sg.library(), ly._Base(), ctypes.c_size_t()
    r = ctypes.byref
    for args in ((None, r(s), r(s), r(s)), (r(b), None, r(s), r(s)), (r(b), r(s), None, r(s)), (r(b), r(s), r(s), None)):
        assert lib.sgmv_base_init(16, 128, 128, 0, 1, 0, *args) == E


def _base(**kw):
    d = dict(codes=0x10000, scale=0x20000, zero=0x30000, N=40, K=300, group=64, format=sg.BASE_I4, dtype=sg.SGMV_BF16,
             has_zero=1)
    d.update(kw)
    return ly._Base(**d)


def test_base_calls_refuse():
    lib, need = sg.library(), ctypes.c_size_t()

    def pack(b=None, codes=0x1000, ldc=150, scale=0x2000, zero=0x3000):
        return lib.sgmv_base_pack(codes, ldc, scale, zero, ctypes.byref(b or _base()), None)

    def product(b=None, x=0x1000, ldx=300, T=3, y=0x9000, ldy=40, n_split=0, ws=None, size=0):
        return lib.sgmv_base_product(x, ldx, T, ctypes.byref(b or _base()), y, ldy, n_split, ws, size, None)

    for kw in (dict(codes=None), dict(ldc=149), dict(scale=None), dict(zero=None), dict(b=_base(has_zero=0, zero=0))):
        assert pack(**kw) == E, kw
    bad = [(dict(codes=0), E), (dict(scale=0), E), (dict(zero=0), E), (dict(has_zero=0), E), (dict(codes=0x10008), E),
           (dict(scale=0x20004), E), (dict(zero=0x30008), E), (dict(N=0), E), (dict(K=-1), E), (dict(format=7), E),
           (dict(dtype=9), E), (dict(group=48), UNS), (dict(format=1), E)]
    for kw, status in bad:
        b = _base(**kw)
        assert pack(b) == status and product(b) == status, kw
        assert lib.sgmv_base_product_workspace(3, ctypes.byref(b), 0, ctypes.byref(need)) == status
    assert lib.sgmv_base_pack(0x1000, 150, 0x2000, 0x3000, None, None) == E
    assert lib.sgmv_base_product(0x1000, 300, 3, None, 0x9000, 40, 0, None, 0, None) == E
    assert lib.sgmv_base_product_workspace(3, None, 0, ctypes.byref(need)) == E
    assert lib.sgmv_base_product_workspace(3, ctypes.byref(_base()), 0, None) == E
    for kw in (dict(x=None), dict(y=None), dict(y=0x1000), dict(ldx=299), dict(ldy=39), dict(T=-1), dict(n_split=-1), dict(n_split=17)):
        assert product(**kw) == E, kw
    assert product(T=0, x=None, y=None) == OK
    assert lib.sgmv_base_product_workspace(0, ctypes.byref(_base()), 0, ctypes.byref(need)) == OK and need.value == 0


def test_base_workspace():
    """Rows in blocks of 64 x 128 (16 KB, for I4 with the sums of their groups behind them), and the ranges' sums."""
    lib, need = sg.library(), ctypes.c_size_t()

    def size(T, n_split=0, **kw):
        assert lib.sgmv_base_product_workspace(T, ctypes.byref(_base(**kw)), n_split, ctypes.byref(need)) == OK
        return need.value

    assert size(64) == 0 and size(64, 1) == 3 * (16384 + 64 * 2 * 4)
    assert size(65, 3) == 2 * 3 * (16384 + 64 * 2 * 4) + 3 * 2 * 64 * 256 * 4
    assert size(65, 2, N=257) == 2 * 3 * (16384 + 64 * 2 * 4) + 2 * 2 * 2 * 64 * 256 * 4
    assert size(65, 16) == size(65, 3)  # three blocks of K
    assert size(64, 1, format=sg.BASE_E2M1, group=32, has_zero=0, zero=0) == 3 * 16384
    assert size(64, 1, dtype=sg.SGMV_F32) == 3 * 3 * (16384 + 64 * 2 * 4)  # in three parts each
    big = dict(N=8192, K=8192, group=128)
    assert size(32, **big) == 0 and size(128, **big) == 0 and size(1024, **big) == 16 * 64 * (16384 + 64 * 4)
    assert size(256, **big) == 4 * 64 * (16384 + 64 * 4) + 4 * 128 * 64 * 256 * 4
    call = lambda ws, n: lib.sgmv_base_product(0x1000, 300, 65, ctypes.byref(_base()), 0x9000, 40, 3, ws, n, None)
    n = size(65, 3)
    assert call(None, n) == E and call(0x10008, n) == E and call(0x10000, n - 1) == sg.SGMV_ECAPACITY


def test_launches_past_the_limit_are_refused():
    b = _base(N=4194304, K=4194304, group=128)
    assert sg.library().sgmv_base_product(0x1000, 1 << 23, 2 ** 31 - 1, ctypes.byref(b), 0x9000, 1 << 23, 0, 0x10,
                                          1 << 62, None) == UNS


def _norm(**kw):
    d = dict(x=0x1000, residual=0x2000, weight=0x3000, residual_out=0x4000, out=0x5000, codes=0x6000, scale=0x7000, T=3,
             heads=2, width=64, dtype=sg.SGMV_BF16, format=sg.KV_E4M3, eps=1e-6)
    d.update({f"ld{a}_token": 128 for a in "xrsoc"})
    d.update({f"ld{a}_head": 64 for a in "xrsoc"})
    d.update(kw)
    return ly._Norm(**d)


def test_norm_refuses():
    lib = sg.library()
    call = lambda **kw: lib.sgmv_rms_norm(ctypes.byref(_norm(**kw)), None)
    bad = [dict(x=0), dict(weight=0), dict(T=-1), dict(heads=0), dict(width=0), dict(dtype=2), dict(eps=0.0),
           dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(format=sg.KV_BF16), dict(scale=0),
           dict(codes=0), dict(residual=0), dict(out=0, codes=0, scale=0), dict(out=0x4000)]
    bad += [{f"ld{a}_token": 127} for a in "xrsoc"] + [{f"ld{a}_head": 63} for a in "xrsoc"]
    for kw in bad:
        assert call(**kw) == E, kw
    assert lib.sgmv_rms_norm(None, None) == E
    assert call(width=32769) == UNS
    wide = {f"ld{a}_token": 1 << 40 for a in "xrsoc"} | {f"ld{a}_head": 32768 for a in "xrsoc"}
    assert call(T=2 ** 31 - 1, heads=65535, width=32768, **wide) == UNS
    assert call(T=0, x=0) == OK


def _cache(**kw):
    d = dict(k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000, pages=4, page_size=16, heads=2, head_dim=64,
             format=sg.KV_I8)
    d.update(kw)
    return sv._KvCache(**d)


def _batch(**kw):
    d = dict(q_start=0x50000, kv_len=0x60000, page_table=0x70000, ldp=4, table_pages=4, B=2, T=3, max_q=2, max_kv=64)
    d.update(kw)
    return sv._KvBatch(**d)


def _append(turn=None, cache=None, batch=None, k=0x80000, kt=128, kh=64, v=0x90000, vt=128, vh=64, dtype=sg.SGMV_BF16,
            **kw):
    d = dict(cos_sin=0x1000, ld=64, positions=64, rotary=64, interleaved=0, heads=4, q=0xa0000, q_out=0xb0000,
             ldq_token=256, ldq_head=64, ldo_token=256, ldo_head=64)
    d.update(kw)
    return sg.library().sgmv_kv_append(ctypes.byref(turn or ly._Rotation(**d)), k, kt, kh, v, vt, vh, dtype,
                                       ctypes.byref(batch or _batch()), ctypes.byref(cache or _cache()), None)


def test_append_refuses():
    for kw in (dict(k=None), dict(v=None), dict(kt=127), dict(vt=127), dict(kh=63), dict(vh=0), dict(dtype=2),
               dict(cos_sin=0), dict(cos_sin=0x1002), dict(ld=63), dict(positions=0), dict(rotary=0), dict(rotary=80),
               dict(rotary=-16), dict(interleaved=2), dict(interleaved=-1), dict(heads=-1), dict(q=0), dict(q_out=0),
               dict(q_out=0xa0000, ldo_token=512), dict(q_out=0xa0000, ldo_head=60 + 8, ldo_token=512),
               dict(ldq_token=255), dict(ldq_head=63), dict(ldo_token=255), dict(ldo_head=1),
               dict(cache=_cache(k=0)), dict(cache=_cache(format=9)), dict(batch=_batch(T=-1)), dict(batch=_batch(ldp=1))):
        assert _append(**kw) == E, kw
    native = dict(k_scale=0, v_scale=0)
    assert _append(cache=_cache(format=sg.KV_F32, **native)) == E  # bf16 rows, fp32 cache
    assert _append(cache=_cache(format=sg.KV_BF16, **native), dtype=sg.SGMV_F32) == E
    for kw in (dict(rotary=40), dict(rotary=8), dict(heads=1025, ldq_token=1 << 20, ldo_token=1 << 20)):
        assert _append(**kw) == UNS, kw
    many = dict(batch=_batch(T=2 ** 31 - 1, max_q=2 ** 31 - 1), heads=1024, ldq_token=1 << 20, ldo_token=1 << 20)
    assert _append(**many) == UNS
    assert sg.library().sgmv_kv_append(None, 0x80000, 128, 64, 0x90000, 128, 64, 1, ctypes.byref(_batch()),
                                       ctypes.byref(_cache()), None) == E
    for b in (_batch(B=0, T=0), _batch(T=0)):
        assert _append(batch=b, k=None, v=None, q=0, q_out=0, cos_sin=0) == OK


# ---- refusals of the binding -----------------------------------------------------------
def test_norm_binding_refuses():
    x, w = torch.zeros(3, 2, 64), torch.zeros(64)
    call = lambda **kw: sg.sgmv_rms_norm(**{**dict(x=x, weight=w), **kw})
    for kw in (dict(x=x.half()), dict(weight=w.bfloat16()), dict(weight=w[:32]), dict(weight=torch.zeros(128)[::2]),
               dict(residual=x.bfloat16()), dict(out=x.bfloat16()), dict(residual=x, residual_out=x.bfloat16()),
               dict(quantise=torch.float16), dict(quantise=torch.int8, codes=x.to(torch.float8_e4m3fn)),
               dict(quantise=torch.int8, scale=torch.zeros(3)), dict(quantise=torch.int8, scale=torch.zeros(3, 2).double())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(x=x[0, 0]), dict(x=x[None]), dict(x=torch.zeros(3, 64, 2).transpose(1, 2)), dict(residual=x[:2]),
               dict(residual_out=x), dict(residual=x, residual_out=x[:, :1]), dict(out=x[..., :32]), dict(codes=x),
               dict(scale=w), dict(want_out=False), dict(quantise=torch.int8, codes=torch.zeros(3, 2, 32, dtype=torch.int8))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError, match="GPU"):
        call()


def test_base_binding_refuses():
    codes, scale, zero = torch.zeros(5, 100, dtype=torch.uint8), torch.zeros(5, 2), torch.zeros(5, 2, dtype=torch.uint8)
    call = lambda **kw: sg.sgmv_base_pack(**{**dict(codes=codes, scale=scale, zero=zero), **kw})
    for kw in (dict(codes=codes.int()), dict(codes=codes[0]), dict(codes=codes.T), dict(scale=scale.half()),
               dict(zero=zero.int()), dict(dtype=torch.bfloat16), dict(format=sg.BASE_E2M1)):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(K=198), dict(K=201), dict(scale=scale[:4]), dict(zero=zero[:, :1]), dict(scale=torch.zeros(5, 4)[:, ::2]),
               dict(K=2 ** 40)):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(group=100), dict(group=0), dict(format=5)):
        with pytest.raises(sg.SgmvError):
            call(**kw)
    with pytest.raises(ValueError, match="GPU"):
        call()
    w = sg.BaseWeight(codes, scale, None, _base(N=5, K=200), torch.float32)
    x = torch.zeros(3, 200)
    for kw in (dict(x=x[:, :199]), dict(x=x[0]), dict(x=torch.zeros(200, 3).T), dict(x=x, y=torch.zeros(3, 4)),
               dict(x=x, y=torch.zeros(5, 3).T), dict(x=x, y=torch.zeros(3, 5).bfloat16())):
        with pytest.raises(ValueError):
            sg.sgmv_base_product(base=w, **kw)
    with pytest.raises(TypeError):
        sg.sgmv_base_product(x.bfloat16(), w)
    with pytest.raises(ValueError):
        sg.sgmv_base_product(x, w, n_split=2 ** 40)
    with pytest.raises(ValueError, match="GPU"):
        sg.sgmv_base_product(x, w)


def test_append_binding_refuses():
    c = sg.sgmv_kv_init(4, 16, 2, 64, torch.int8, "cpu")
    b = sg.sgmv_kv_batch(I32(0, 1, 3), I32(5, 6), torch.zeros(2, 4, dtype=torch.int32), 3, 2, 6)
    k, q, table = torch.zeros(3, 2, 64), torch.zeros(3, 4, 64), torch.zeros(64, 64)
    call = lambda **kw: sg.sgmv_kv_append(**{**dict(q=q, k=k, v=k, batch=b, cache=c, cos_sin=table), **kw})
    for kw in (dict(v=k.bfloat16()), dict(k=k.half(), v=k.half()), dict(q=q.bfloat16()), dict(q_out=q.bfloat16()),
               dict(cos_sin=table.double()), dict(cos_sin=table[0]), dict(cos_sin=torch.zeros(64, 128)[:, ::2])):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(k=k[:2]), dict(v=k[:, :1]), dict(q=q[..., :32]), dict(q_out=q[:, :3]), dict(q=None, q_out=q)):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError, match="GPU"):
        call()
