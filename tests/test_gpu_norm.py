"""GPU parity of the root-mean-square norm against the oracle.

Bars, element by element (u = 2^-24): h and g are one fp32 rounding each, equal to the oracle's; a row's sum of
squares adds at most 64 numbers one after another in a thread and then over at most 16 + 10 partial sums, each rounded
once, of terms rounded once: (64 + 26 + 1) u of it, half of that in the root, the root and its inverse and the last
product u or 2 u each: 50 u in all. Then the output's own rounding (bf16: half of its eps, 2^-8; fp32: u).
The residual is the exact sum rounded to fp32 and once more to bf16. Codes are equal, scales off by 50 u and 3 u.
"""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, E4M3, I8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.int8
NAMES = {E4M3: "e4m3", I8: "i8", None: None}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import segmented_gather_gemv_amd as m
    return m


def _f32(t):
    return None if t is None else t.detach().float().cpu().numpy()


def _close(got, ref, rel, tiny):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)])
    d, lim = abs(got - ref)[fine], (rel * abs(ref) + tiny)[fine]
    assert (d <= lim).all(), float((d - lim).max())


def _check(got, x, w, eps, residual, quantise):
    out, h, codes, scale = lo.rms_norm(_f32(x), _f32(w), eps, _f32(residual), NAMES[quantise])
    half = 2.0 ** -8 if x.dtype == BF16 else U
    if got.out is not None:
        assert got.out.dtype == x.dtype
        _close(got.out, out, half + 51 * U, 2.0 ** -133)  # the smallest bf16
    if residual is not None:
        want = torch.from_numpy(h).float().to(x.dtype)
        assert torch.equal(got.residual.cpu().view(torch.int16 if x.dtype == BF16 else torch.int32)[~torch.isnan(want)],
                           want.view(torch.int16 if x.dtype == BF16 else torch.int32)[~torch.isnan(want)])
    if quantise is not None:
        assert np.array_equal(got.codes.cpu().view(torch.uint8).numpy(), codes.view(np.uint8))
        _close(got.scale, scale, 53 * U, 2.0 ** -149)


SHAPES = [(1, 1, 1), (3, 1, 7), (5, 1, 8), (2, 1, 9), (33, 1, 64), (17, 3, 80), (6, 5, 128), (4, 1, 129), (9, 2, 255),
          (7, 1, 513), (3, 1, 1000), (600, 1, 520), (513, 1, 1032), (5, 1, 2048), (515, 1, 4104), (2, 1, 8200), (520, 1, 8193),
          (3, 1, 16384), (513, 1, 9000), (2, 1, 32768), (1, 1, 32761)]


@pytest.mark.parametrize("dtype,quantise", [(BF16, None), (BF16, E4M3), (BF16, I8), (F32, None), (F32, E4M3), (F32, I8)])
@pytest.mark.parametrize("T,heads,W", SHAPES)
def test_norm_against_oracle(sg, T, heads, W, dtype, quantise):
    g = torch.Generator().manual_seed(T * 7 + W)
    shape = (T, W) if heads == 1 else (T, heads, W)
    x = torch.randn(shape, generator=g).to(dtype)
    w = (1 + 0.3 * torch.randn(W, generator=g)).to(dtype)
    r = (4 * torch.randn(shape, generator=g)).to(dtype) if (T + W) % 2 or quantise is None else None
    got = sg.sgmv_rms_norm(x.to(DEV), w.to(DEV), 1e-5, residual=None if r is None else r.to(DEV), quantise=quantise)
    assert (got.residual is None) == (r is None) and (got.codes is None) == (quantise is None)
    _check(got, x, w, 1e-5, r, quantise)


@pytest.mark.parametrize("T,W,dtype,quantise", [(2100, 1099, BF16, E4M3), (700, 1501, BF16, I8), (1030, 16001, BF16, I8),
                                                (1030, 9000, BF16, None), (2100, 777, F32, I8), (1030, 8001, F32, E4M3)])
def test_norm_of_many_rows(sg, T, W, dtype, quantise):
    """Shapes that many rows take; every eighth row is the same."""
    g = torch.Generator().manual_seed(T + W)
    x, r = (torch.randn(8, W, generator=g).to(dtype) for _ in range(2))
    w = torch.randn(W, generator=g).to(dtype)
    many = lambda t: t.repeat(-(-T // 8), 1)[:T].to(DEV)
    got = sg.sgmv_rms_norm(many(x), w.to(DEV), residual=many(r), quantise=quantise)
    _check(sg.Normed(*(None if t is None else t[:8] for t in got)), x, w, 1e-6, r, quantise)
    for t in got:
        if t is not None:
            t = t.view(torch.uint8) if t.element_size() == 1 else t
            assert torch.equal(t, t[:8].repeat(-(-T // 8), *[1] * (t.dim() - 1))[:T])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("W", [48, 300, 2056])
def test_norm_of_zeros_extremes_and_rows_that_are_not_finite(sg, dtype, W):
    g = torch.Generator().manual_seed(W)
    x = torch.randn(12, W, generator=g)
    x[0] = 0
    x[1] *= 2.0 ** 100          # squares past fp32
    x[2] *= 2.0 ** -90          # squares below it
    x[3, 5] = float("inf")
    x[4, W - 1] = float("nan")
    x[5, 0] = float("-inf")
    x[6] = 3.3e38               # the largest, and their sum of squares
    x[7] *= 2.0 ** -70
    x[8, 1:] = 0
    x[9] *= 1e18
    x[10] = -0.0
    x = x.to(dtype)
    w = (1 + 0.1 * torch.rand(W, generator=g)).to(dtype)
    w[:8] = 1
    for eps in (1e-6, 1e-30):
        for quantise in (E4M3, I8):
            got = sg.sgmv_rms_norm(x.to(DEV), w.to(DEV), eps, quantise=quantise)
            # products past fp32 are infinite, here and there
            _check(got, x, w, eps, None, quantise)
    assert torch.isfinite(got.out[[0, 1, 2, 7, 8, 9, 10, 11]]).all()


def test_norm_head_by_head_in_place_of_a_fused_projection(sg):
    """Unaligned column slices of one wide row, normed in place; what is between them stays."""
    g = torch.Generator().manual_seed(3)
    wide = torch.randn(29, 5 + 4 * 96 + 3 * 80 + 2, generator=g).to(BF16)
    w = torch.randn(80, generator=g).to(BF16)
    dev = wide.to(DEV)
    view = lambda t: t[:, 5 + 4 * 96:5 + 4 * 96 + 240].unflatten(1, (3, 80))
    got = sg.sgmv_rms_norm(view(dev), w.to(DEV), 1e-6, out=view(dev))
    assert got.out.data_ptr() == view(dev).data_ptr()
    _check(got, view(wide), w, 1e-6, None, None)
    assert torch.equal(dev[:, :5 + 4 * 96].cpu(), wide[:, :5 + 4 * 96]) and torch.equal(dev[:, -2:].cpu(), wide[:, -2:])
    # the same rows by a head stride of 128, from an aligned place: 16-byte pieces
    wide = torch.randn(29, 3 * 128, generator=g).to(BF16)
    dev = wide.to(DEV)
    view = lambda t: t.unflatten(1, (3, 128))[:, :, :80]
    _check(sg.sgmv_rms_norm(view(dev), w.to(DEV), 1e-6, out=view(dev)), view(wide), w, 1e-6, None, None)
    assert torch.equal(dev.unflatten(1, (3, 128))[:, :, 80:].cpu(), wide.unflatten(1, (3, 128))[:, :, 80:])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("W", [100, 1024, 5000])
def test_norm_in_place_and_into_strided_rows(sg, dtype, W):
    g = torch.Generator().manual_seed(W)
    x, r = (torch.randn(11, W, generator=g).to(dtype) for _ in range(2))
    w = torch.randn(W, generator=g).to(dtype)
    want = sg.sgmv_rms_norm(x.to(DEV), w.to(DEV), 1e-5, residual=r.to(DEV), quantise=I8)
    _check(want, x, w, 1e-5, r, I8)
    xd, rd = x.to(DEV), r.to(DEV)
    got = sg.sgmv_rms_norm(xd, w.to(DEV), 1e-5, residual=rd, residual_out=rd, out=xd)
    assert torch.equal(rd, want.residual) and torch.equal(xd, want.out) and got.codes is None
    rd = r.to(DEV)
    xd = x.to(DEV)
    sg.sgmv_rms_norm(xd, w.to(DEV), 1e-5, residual=rd, residual_out=xd, out=rd)  # each over the other
    assert torch.equal(xd, want.residual) and torch.equal(rd, want.out)
    out = torch.full((11, W + 9), 7.0, dtype=dtype, device=DEV)
    codes = torch.full((11, W + 5), 77, dtype=I8, device=DEV)
    scale = torch.empty(11, device=DEV)
    got = sg.sgmv_rms_norm(x.to(DEV), w.to(DEV), 1e-5, residual=r.to(DEV), quantise=I8, out=out[:, 3:3 + W],
                           codes=codes[:, 1:1 + W], scale=scale)
    assert torch.equal(got.out, want.out) and torch.equal(got.codes, want.codes) and torch.equal(scale, want.scale)
    assert (out[:, :3] == 7).all() and (out[:, 3 + W:] == 7).all()
    assert (codes[:, :1] == 77).all() and (codes[:, 1 + W:] == 77).all()
    only = sg.sgmv_rms_norm(x.to(DEV), w.to(DEV), 1e-5, residual=r.to(DEV), quantise=I8, want_out=False)
    assert only.out is None and torch.equal(only.codes, want.codes) and torch.equal(only.scale, want.scale)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_of_rows_with_heads_outermost(sg, dtype):
    g = torch.Generator().manual_seed(3)
    x, r = (torch.randn(5, 33, 80, generator=g).to(dtype) for _ in range(2))
    w = torch.randn(80, generator=g).to(dtype)
    dx, dr = x.to(DEV).transpose(0, 1), r.to(DEV).transpose(0, 1)
    got = sg.sgmv_rms_norm(dx, w.to(DEV), residual=dr, quantise=I8)
    assert got.out.is_contiguous() and got.codes.is_contiguous()
    _check(got, x.transpose(0, 1), w, 1e-6, r.transpose(0, 1), I8)
    again = sg.sgmv_rms_norm(dx, w.to(DEV), residual=dr, out=dx, residual_out=dr)  # where they are
    assert torch.equal(again.out, got.out) and torch.equal(dx, got.out) and torch.equal(dr, got.residual)


def test_norm_of_no_rows(sg):
    w = torch.ones(64, device=DEV)
    got = sg.sgmv_rms_norm(torch.empty(0, 64, device=DEV), w, quantise=E4M3)
    assert got.out.shape == (0, 64) and got.codes.shape == (0, 64) and got.scale.shape == (0,)
    got = sg.sgmv_rms_norm(torch.empty(0, 3, 64, device=DEV), w)
    assert got.out.shape == (0, 3, 64)


def test_norm_captured_and_replayed_beside_another_stream(sg):
    g = torch.Generator().manual_seed(9)
    x, r = (torch.randn(40, 1536, generator=g).to(BF16).to(DEV) for _ in range(2))
    w = torch.randn(1536, generator=g).to(BF16).to(DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        first = sg.sgmv_rms_norm(x, w, residual=r, quantise=E4M3)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sg.sgmv_rms_norm(x, w, residual=r, quantise=E4M3)
    for seed in range(3):
        x.copy_(torch.randn(40, 1536, generator=g))
        graph.replay()
        want = sg.sgmv_rms_norm(x, w, residual=r, quantise=E4M3)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.isfinite(first.out).all()
