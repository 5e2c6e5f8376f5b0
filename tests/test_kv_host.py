"""CPU tests of the paged cache, its attention and the draft check: the oracle's pins, sizes,
and the refusals of the C-ABI and of the binding. Nothing is launched."""
import ctypes
import math

import numpy as np
import pytest
import torch

import segmented_gather_gemv_amd as sg
from oracle import kv_oracle as ko
from segmented_gather_gemv_amd import _serving as sv


# ---- the oracle's pins ----------------------------------------------------------------
def test_e4m3_values_are_the_formats():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).double().numpy()
    got = ko.e4m3_value(np.arange(256))
    assert np.array_equal(np.isnan(ref), np.isnan(got))
    assert np.array_equal(ref[~np.isnan(ref)], got[~np.isnan(ref)])


def test_e4m3_rounding_is_to_nearest_even():
    # between 1.0 and 1.125 (codes 56 and 57), 0 and the smallest, and the largest
    y = np.array([1.0625, np.nextafter(1.0625, 2), np.nextafter(1.0625, 0), 1.1875, 2.0 ** -10,
                  3 * 2.0 ** -10, 448.0, -448.0])
    assert ko.e4m3_code(y).tolist() == [56, 57, 56, 58, 0, 2, 126, 254]
    x = torch.randn(4096, generator=torch.Generator().manual_seed(1)) * 100
    x = x.clamp(-448, 448)
    assert np.array_equal(ko.e4m3_code(x.double().numpy()),
                          x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_quantise_by_hand():
    code, scale = ko.quantise(np.array([[1.0, -2.0, 0.5, 0.0]]), "i8")
    assert code.tolist() == [[64, -127, 32, 0]] and scale[0] == 2 / 127  # 63.5 and 31.75
    code, scale = ko.quantise(np.array([[0.0, 0.0], [np.inf, 1.0], [np.nan, 3.0]]), "e4m3")
    assert code.tolist() == [[0, 0]] * 3 and scale[0] == 0 and np.isnan(scale[1:]).all()


def test_layout_is_a_permutation_and_the_documented_one():
    for D, elem in ((64, 1), (80, 2), (16, 4)):
        c = ko.Cache(32, D, elem)
        for f in (c.k_index, c.v_index):
            assert sorted(np.concatenate([f(t) for t in range(32)])) == list(range(32 * D))
    assert [ko.place(r) for r in range(16)] == [0, 1, 2, 3, 8, 9, 10, 11, 4, 5, 6, 7, 12, 13, 14, 15]


def test_attention_row_by_hand():
    q, k, v = np.array([1.0]), np.array([[0.0], [math.log(3.0)]]), np.array([[4.0], [8.0]])
    out, lse, _, _ = ko.attention_row(q, k, v, 1.0)
    assert abs(out[0] - 7.0) < 1e-12 and abs(lse - math.log(4.0)) < 1e-12
    out, lse, _, _ = ko.attention_row(q, k[:0], v[:0], 1.0)
    assert out[0] == 0 and lse == -np.inf


def test_verify_by_hand():
    t = np.array([[0.5, 0.5, 0.0], [0.0, 0.25, 0.75]])
    d = np.array([[0.25, 0.25, 0.5]])
    assert ko.verify(t, d, [1], [0.9], 0.2) == ([1, 1], 1)         # 0.225 < 0.5; then p_2
    assert ko.verify(t, d, [1], [0.9], 0.25) == ([1, 2], 1)        # 0.25 is not > 0.25
    assert ko.verify(t, d, [2], [0.0], 0.5) == ([1], 0)            # 0 < 0 fails; rest (1/4, 1/4, 0)
    assert ko.verify(t, None, [0], [0.5], 0.99) == ([1], 0)        # certain draft, rest (0, 1/2, 0)
    assert ko.verify(t * 0, None, [0], [0.5], 0.5) == ([-1], 0)


# ---- sizes ----------------------------------------------------------------------------
def test_cache_sizes_and_wrap():
    for dtype, elem in ((torch.float32, 4), (torch.bfloat16, 2), (torch.float8_e4m3fn, 1),
                        (torch.int8, 1)):
        c = sg.sgmv_kv_init(5, 32, 3, 80, dtype, "cpu")
        assert c.k.numel() == c.v.numel() == 5 * 32 * 3 * 80 and c.k.element_size() == elem
        assert (c.k_scale is not None) == (elem == 1)
        if elem == 1:
            assert tuple(c.k_scale.shape) == (5, 3, 32)
        w = sg.sgmv_kv_wrap(c.k, c.v, c.k_scale, c.v_scale)
        assert w.desc.k == c.k.data_ptr() and w.page_size == 32 and w.heads == 3


def test_constants_match_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(sg.__file__)), "include", "sgmv.h")).read()
    defs = dict(re.findall(r"#define SGMV_([A-Z_0-9]+) (\d+)", text))
    for name in ("KV_GROUP", "KV_MAX_PAGE", "KV_MAX_HEAD_DIM", "KV_MAX_HEADS", "KV_MAX_B",
                 "KV_MAX_SPLITS"):
        assert int(defs[name]) == getattr(sg, name), name
    for name in ("KV_F32", "KV_BF16", "KV_E4M3", "KV_I8"):
        assert re.search(r"SGMV_%s = %d\b" % (name, getattr(sg, name)), text), name


# ---- refusals of the C-ABI -------------------------------------------------------------
def _cache(**kw):
    d = dict(k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000, pages=4, page_size=16,
             heads=2, head_dim=64, format=sg.KV_I8)
    d.update(kw)
    return sv._KvCache(**d)


def _batch(**kw):
    d = dict(q_start=0x50000, kv_len=0x60000, page_table=0x70000, ldp=4, table_pages=4, B=2, T=3,
             max_q=2, max_kv=64)
    d.update(kw)
    return sv._KvBatch(**d)


def _attn(**kw):
    d = dict(q=0x80000, out=0x90000, lse=0, ldq_token=256, ldq_head=64, ldo_token=256, ldo_head=64,
             heads=4, dtype=sg.SGMV_BF16, scale=0.125, window=0, n_split=1)
    d.update(kw)
    return sv._Attention(**d)


BAD_SHAPES = [(dict(pages=0), sg.SGMV_EINVAL), (dict(page_size=0), sg.SGMV_EINVAL),
              (dict(heads=0), sg.SGMV_EINVAL), (dict(head_dim=0), sg.SGMV_EINVAL),
              (dict(format=4), sg.SGMV_EINVAL), (dict(format=-1), sg.SGMV_EINVAL),
              (dict(page_size=8), sg.SGMV_EUNSUPPORTED), (dict(page_size=48), sg.SGMV_EUNSUPPORTED),
              (dict(page_size=8192), sg.SGMV_EUNSUPPORTED), (dict(head_dim=24), sg.SGMV_EUNSUPPORTED),
              (dict(head_dim=272), sg.SGMV_EUNSUPPORTED), (dict(heads=1025), sg.SGMV_EUNSUPPORTED)]
BAD_CACHES = BAD_SHAPES + [(dict(k=0), sg.SGMV_EINVAL), (dict(v=0), sg.SGMV_EINVAL),
                           (dict(k_scale=0), sg.SGMV_EINVAL), (dict(v_scale=0), sg.SGMV_EINVAL),
                           (dict(k=0x10008), sg.SGMV_EINVAL), (dict(v_scale=0x40004), sg.SGMV_EINVAL)]
BAD_BATCHES = [(dict(B=-1), sg.SGMV_EINVAL), (dict(T=-1), sg.SGMV_EINVAL),
               (dict(max_q=-1), sg.SGMV_EINVAL), (dict(max_kv=-1), sg.SGMV_EINVAL),
               (dict(table_pages=-1), sg.SGMV_EINVAL), (dict(ldp=3), sg.SGMV_EINVAL),
               (dict(q_start=0), sg.SGMV_EINVAL), (dict(kv_len=0), sg.SGMV_EINVAL),
               (dict(page_table=0), sg.SGMV_EINVAL), (dict(B=65537), sg.SGMV_EUNSUPPORTED)]


def _calls(cache, batch):
    """Every call that takes a cache and a batch, with otherwise good arguments."""
    lib = sg.library()
    c, b, need = ctypes.byref(cache), ctypes.byref(batch), ctypes.c_size_t()
    a = _attn()
    return [lib.sgmv_kv_write(0x80000, 128, 64, 0x90000, 128, 64, sg.SGMV_BF16, b, c, None),
            lib.sgmv_kv_read(b, c, 0x1000, 3, 0x80000, 128, 64, 0x90000, 128, 64, sg.SGMV_BF16, None),
            lib.sgmv_kv_attention_workspace(ctypes.byref(a), b, c, ctypes.byref(need)),
            lib.sgmv_kv_attention(ctypes.byref(a), b, c, None, 0, None)]


@pytest.mark.parametrize("kw,status", BAD_SHAPES)
def test_init_refuses(kw, status):
    d = dict(pages=4, page_size=16, heads=2, head_dim=64, format=sg.KV_I8)
    d.update(kw)
    c, x, y = sv._KvCache(), ctypes.c_size_t(), ctypes.c_size_t()
    lib = sg.library()
    assert lib.sgmv_kv_init(*d.values(), ctypes.byref(c), ctypes.byref(x), ctypes.byref(y)) == status
    assert lib.sgmv_kv_init(4, 16, 2, 64, 3, None, ctypes.byref(x), ctypes.byref(y)) == sg.SGMV_EINVAL
    assert lib.sgmv_kv_init(4, 16, 2, 64, 3, ctypes.byref(c), None, ctypes.byref(y)) == sg.SGMV_EINVAL


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused(kw, status):
    assert _calls(_cache(**kw), _batch()) == [status] * 4


@pytest.mark.parametrize("kw,status", BAD_BATCHES)
def test_bad_batches_are_refused(kw, status):
    assert _calls(_cache(), _batch(**kw)) == [status] * 4


def test_null_structs_are_refused():
    lib, need = sg.library(), ctypes.c_size_t()
    a, b, c = _attn(), _batch(), _cache()
    for x, y, z in ((None, b, c), (a, None, c), (a, b, None)):
        args = [None if t is None else ctypes.byref(t) for t in (x, y, z)]
        assert lib.sgmv_kv_attention(*args, None, 0, None) == sg.SGMV_EINVAL
        assert lib.sgmv_kv_attention_workspace(*args, ctypes.byref(need)) == sg.SGMV_EINVAL
    assert lib.sgmv_kv_attention_workspace(ctypes.byref(a), ctypes.byref(b), ctypes.byref(c),
                                           None) == sg.SGMV_EINVAL


def test_row_types_and_strides_are_checked():
    lib, b = sg.library(), ctypes.byref(_batch())
    E = sg.SGMV_EINVAL

    def write(cache=None, k=0x80000, kt=128, kh=64, v=0x90000, vt=128, vh=64, dtype=sg.SGMV_BF16):
        return lib.sgmv_kv_write(k, kt, kh, v, vt, vh, dtype, b, ctypes.byref(cache or _cache()), None)

    for kw in (dict(k=None), dict(v=None), dict(kt=127), dict(vt=127), dict(kh=63), dict(vh=0),
               dict(dtype=2), dict(dtype=-1)):
        assert write(**kw) == E, kw
    native = dict(k_scale=0, v_scale=0)
    assert write(_cache(format=sg.KV_F32, **native)) == E        # bf16 rows, fp32 cache
    assert write(_cache(format=sg.KV_BF16, **native), dtype=sg.SGMV_F32) == E

    def read(out_start=0x1000, rows=3, k=0x80000, kt=128, dtype=sg.SGMV_BF16):
        return lib.sgmv_kv_read(b, ctypes.byref(_cache()), out_start, rows, k, kt, 64, 0x90000, 128,
                                64, dtype, None)

    for kw in (dict(out_start=None), dict(rows=-1), dict(k=None), dict(kt=1), dict(dtype=7)):
        assert read(**kw) == E, kw
    for kw in (dict(q=0), dict(out=0), dict(ldq_head=63), dict(ldo_token=255), dict(heads=3),
               dict(heads=0), dict(dtype=2), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(window=-1),
               dict(n_split=-1), dict(n_split=65)):
        a = _attn(**kw)
        assert lib.sgmv_kv_attention(ctypes.byref(a), b, ctypes.byref(_cache()), None, 0, None) == E, kw
    a = _attn(heads=2048)
    assert lib.sgmv_kv_attention(ctypes.byref(a), b, ctypes.byref(_cache()), None, 0,
                                 None) == sg.SGMV_EUNSUPPORTED


def test_workspace_is_checked():
    lib, b, c = sg.library(), _batch(max_kv=4096), _cache()
    a = _attn(n_split=4)
    need = ctypes.c_size_t()
    args = [ctypes.byref(x) for x in (a, b, c)]
    assert lib.sgmv_kv_attention_workspace(*args, ctypes.byref(need)) == sg.SGMV_OK
    assert need.value == 4 * 3 * 4 * (64 + 2) * 4
    assert lib.sgmv_kv_attention(*args, None, 0, None) == sg.SGMV_EINVAL
    assert lib.sgmv_kv_attention(*args, 0xa0008, need.value, None) == sg.SGMV_EINVAL
    assert lib.sgmv_kv_attention(*args, 0xa0000, need.value - 1, None) == sg.SGMV_ECAPACITY


def test_empty_calls_do_nothing():
    lib, c = sg.library(), ctypes.byref(_cache())
    for b in (_batch(B=0, T=0), _batch(T=0)):
        b = ctypes.byref(b)
        assert lib.sgmv_kv_write(None, 0, 0, None, 0, 0, sg.SGMV_BF16, b, c, None) == sg.SGMV_OK
        assert lib.sgmv_kv_read(b, c, None, 0, None, 0, 0, None, 0, 0, sg.SGMV_BF16, None) == sg.SGMV_OK
        a, need = _attn(q=0, out=0), ctypes.c_size_t(7)
        assert lib.sgmv_kv_attention(ctypes.byref(a), b, c, None, 0, None) == sg.SGMV_OK
        assert lib.sgmv_kv_attention_workspace(ctypes.byref(a), b, c, ctypes.byref(need)) == sg.SGMV_OK
        assert need.value == 0
    assert lib.sgmv_verify_drafts(None, 0, None, 0, 10, 0, None, None, 0, 0, 0, None, None, None, 0,
                                  None, None, 0, None) == sg.SGMV_OK


def test_verify_refuses():
    def call(target=0x1000, ldt=10, draft=0x2000, ldd=10, vocab=10, dtype=0, ids=0x3000, start=0x4000,
             B=2, N=3, most=2, au=0x5000, su=0x6000, tokens=0x7000, ldo=3, accepted=0x8000,
             ws=0x9000, size=32):
        return sg.library().sgmv_verify_drafts(target, ldt, draft, ldd, vocab, dtype, ids, start, B, N,
                                               most, au, su, tokens, ldo, accepted, ws, size, None)

    for kw in (dict(target=None), dict(ldt=9), dict(ldd=9), dict(vocab=0), dict(dtype=2), dict(ids=None),
               dict(start=None), dict(B=-1), dict(N=-1), dict(most=-1), dict(au=None), dict(su=None),
               dict(tokens=None), dict(ldo=2), dict(accepted=None), dict(ws=None), dict(ws=0x9008)):
        assert call(**kw) == sg.SGMV_EINVAL, kw
    assert sg.library().sgmv_verify_drafts_workspace(2, 10) == 32
    assert call(size=31) == sg.SGMV_ECAPACITY
    assert call(B=65536, size=1 << 30) == sg.SGMV_EUNSUPPORTED
    assert call(vocab=(1 << 30) + 1, ldt=1 << 31, ldd=1 << 31, size=1 << 40) == sg.SGMV_EUNSUPPORTED


# ---- refusals of the binding -----------------------------------------------------------
def test_binding_refuses():
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    c = sg.sgmv_kv_init(4, 16, 2, 64, torch.int8, "cpu")
    b = sg.sgmv_kv_batch(i32(0, 1, 3), i32(5, 6), torch.zeros(2, 4, dtype=torch.int32), 3, 2, 6)
    k = torch.zeros(3, 2, 64)
    with pytest.raises(TypeError):
        sg.sgmv_kv_init(4, 16, 2, 64, torch.float16, "cpu")
    with pytest.raises(sg.SgmvError):
        sg.sgmv_kv_init(4, 20, 2, 64, torch.int8, "cpu")
    for bad in ((c.k, c.v, None, None), (c.k, c.v, c.k_scale[:2], c.v_scale),
                (c.k[:2], c.v, c.k_scale, c.v_scale), (c.v, c.v, c.k_scale, c.v_scale)):
        with pytest.raises(ValueError):
            sg.sgmv_kv_wrap(*bad)
    with pytest.raises(TypeError):
        sg.sgmv_kv_batch(torch.zeros(3), i32(5, 6), torch.zeros(2, 4, dtype=torch.int32), 3, 2, 6)
    with pytest.raises(ValueError):
        sg.sgmv_kv_batch(i32(0, 3), i32(5, 6), torch.zeros(2, 4, dtype=torch.int32), 3, 2, 6)
    for bad in (k[:2], k[:, :1], k[..., :32], torch.zeros(3, 2, 128)[..., ::2]):
        with pytest.raises(ValueError):
            sg.sgmv_kv_write(bad, k, b, c)
        with pytest.raises(ValueError):
            sg.sgmv_kv_write(k, bad, b, c)
    with pytest.raises(TypeError):
        sg.sgmv_kv_write(k, k.bfloat16(), b, c)
    with pytest.raises(TypeError):
        sg.sgmv_kv_write(k.half(), k.half(), b, c)
    with pytest.raises(TypeError):
        sg.sgmv_kv_read(b, c, torch.zeros(3), 3)
    with pytest.raises(TypeError):
        sg.sgmv_kv_read(b, c, i32(0, 1, 3), 3, torch.bfloat16, k=k)
    q = torch.zeros(3, 4, 64)
    with pytest.raises(TypeError):
        sg.sgmv_kv_attention(q, b, c, out=q.bfloat16())
    with pytest.raises(TypeError):
        sg.sgmv_kv_attention(q, b, c, lse=torch.zeros(3, 3))
    with pytest.raises(sg.SgmvError):
        sg.sgmv_kv_attention(torch.zeros(3, 3, 64), b, c)
    f = torch.zeros(3)
    t = torch.zeros(5, 10)
    good = dict(target=t, draft=t[:3], draft_ids=i32(0, 0, 0), draft_start=i32(0, 1, 3), accept_u=f,
                sample_u=f[:2], max_drafts=2)
    for kw in (dict(target=t[:4]), dict(draft=t[:2]), dict(draft=t[:3, :5])):
        with pytest.raises(ValueError):
            sg.sgmv_verify_drafts(**{**good, **kw})
    for kw in (dict(draft=t[:3].bfloat16()), dict(draft_start=i32(0, 1)), dict(accept_u=f.double()),
               dict(draft_ids=torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(TypeError):
            sg.sgmv_verify_drafts(**{**good, **kw})


def test_binding_launches_nothing_on_host_tensors():
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    c = sg.sgmv_kv_init(4, 16, 2, 64, torch.int8, "cpu")
    b = sg.sgmv_kv_batch(i32(0, 1, 3), i32(5, 6), torch.zeros(2, 4, dtype=torch.int32), 3, 2, 6)
    k = torch.zeros(3, 2, 64)
    for call in (lambda: sg.sgmv_kv_write(k, k, b, c), lambda: sg.sgmv_kv_read(b, c, i32(0, 1, 3), 3),
                 lambda: sg.sgmv_kv_attention(k, b, c),
                 lambda: sg.sgmv_verify_drafts(torch.zeros(2, 5), None, i32(1), i32(0, 1), k[0, 0, :1],
                                               k[0, 0, :1], 1)):
        with pytest.raises(ValueError, match="GPU"):
            call()
