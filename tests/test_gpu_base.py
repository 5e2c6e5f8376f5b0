"""GPU parity of the base product of 4-bit weights against the oracle.

Bars, element by element (u = 2^-24): products of bf16 values and whole numbers below 16 are exact in fp32, so that y is
off by its sums' roundings: at most K + 16 terms one after another and the groups' scaling and joining (3 roundings each,
below K + 48 in all), each u of the sum of sizes A = sum s (c + z) |x| that the sums meet (E2M1: A = sum |w x|; of fp32
rows, each in three parts, 3 K + 48). Then y's own rounding (bf16: half of its eps, 2^-8; fp32: u).
"""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import segmented_gather_gemv_amd as m
    return m


class Weight:
    def __init__(self, sg, N, K, fmt, dtype, group, zero, seed=0):
        g = torch.Generator().manual_seed(seed + N + K)
        G = -(-K // group)
        self.N, self.K, self.group, self.fmt = N, K, group, fmt
        self.codes = torch.randint(0, 256, (N, (K + 1) // 2), generator=g, dtype=torch.uint8)
        if fmt == "e2m1":
            self.scale = torch.randint(110, 140, (N, G), generator=g, dtype=torch.uint8)
        else:
            self.scale = (torch.randn(N, G, generator=g) * torch.exp(torch.randn(N, G, generator=g))).to(dtype)
        self.zero = torch.randint(0, 16, (N, G), generator=g, dtype=torch.uint8) if zero else None
        dev = lambda t: None if t is None else t.to(DEV)
        self.packed = sg.sgmv_base_pack(dev(self.codes), dev(self.scale), dev(self.zero), K=K, group=group,
                                        format=sg.BASE_E2M1 if fmt == "e2m1" else sg.BASE_I4, dtype=dtype)
        self.value, self.size = lo.base_weight(
            self.codes.numpy(), K, self.scale.float().numpy() if fmt == "i4" else self.scale.numpy(),
            None if self.zero is None else self.zero.numpy(), group, fmt)

    def check(self, y, x):
        x64 = x.double().cpu().numpy()
        ref, A = x64 @ self.value.T, abs(x64) @ self.size.T
        f32 = x.dtype == F32
        d = abs(y.double().cpu().numpy() - ref)
        lim = (U if f32 else 2.0 ** -8) * abs(ref) + ((3 if f32 else 1) * self.K + 48) * U * A + 2.0 ** -133
        assert (d <= lim).all(), float((d - lim).max())


FORMS = [("i4", 128, False), ("i4", 128, True), ("i4", 64, True), ("i4", 64, False), ("i4", 32, False), ("i4", 32, True),
         ("i4", 256, True), ("i4", 1024, False), ("e2m1", 32, False)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt,group,zero", FORMS)
@pytest.mark.parametrize("N,K", [(1, 1), (16, 128), (17, 129), (40, 300), (100, 520), (96, 1500), (250, 2048)])
def test_product_against_oracle(sg, N, K, fmt, group, zero, dtype):
    w = Weight(sg, N, K, fmt, dtype, group, zero)
    g = torch.Generator().manual_seed(1)
    for T in (1, 2, 16, 17, 40):
        x = torch.randn(T, K, generator=g).to(dtype)
        w.check(sg.sgmv_base_product(x.to(DEV), w.packed), x)
        for n in (1, 3) if T in (1, 40) else ():  # in tiles, K in ranges
            w.check(sg.sgmv_base_product(x.to(DEV), w.packed, n_split=n), x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt,group,zero", FORMS)
@pytest.mark.parametrize("T", [64, 65, 128, 129, 200, 333])
def test_product_of_many_rows(sg, T, fmt, group, zero, dtype):
    N, K = (331, 700) if T % 2 else (384, 640)
    w = Weight(sg, N, K, fmt, dtype, group, zero)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(T)).to(dtype)
    for n in (0, 1, 2, 16):
        w.check(sg.sgmv_base_product(x.to(DEV), w.packed, n_split=n), x)


@pytest.mark.parametrize("T,N,K,fmt,group,zero", [(200, 5000, 10050, "e2m1", 32, False), (260, 8200, 4700, "i4", 128, True),
                                                  (2100, 2048, 2400, "i4", 64, False), (1500, 1790, 300, "i4", 32, True),
                                                  (1200, 1801, 1100, "i4f32", 64, True), (2400, 900, 333, "e2m1f32", 32, False),
                                                  (340, 1500, 10050, "i4f32", 128, False), (480, 700, 15403, "i4f32", 32, True)])
def test_product_as_the_library_chooses(sg, T, N, K, fmt, group, zero):
    """Sizes that go to the tiles by themselves, with and without ranges."""
    dtype, fmt = F32 if fmt.endswith("f32") else BF16, fmt.replace("f32", "")
    w = Weight(sg, N, K, fmt, dtype, group, zero)
    assert sg.sgmv_base_product_workspace(T, w.packed) > 0
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(T)).to(dtype)
    y = sg.sgmv_base_product(x.to(DEV), w.packed)
    w.check(y, x)
    need = sg.sgmv_base_product_workspace(T, w.packed)
    space = torch.full((need + 64,), 7, dtype=torch.uint8, device=DEV)
    assert torch.equal(sg.sgmv_base_product(x.to(DEV), w.packed, workspace=space[:need]), y)
    assert (space[need:] == 7).all()


@pytest.mark.parametrize("N", [256, 272, 500])
@pytest.mark.parametrize("T", [64, 67, 700])
def test_every_launch_shape_gives_the_same_sums(sg, T, N):
    """Whole numbers, so that sums are exact and every kernel's results are equal."""
    K = 900
    g = torch.Generator().manual_seed(N + T)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    for zero in (None, torch.randint(0, 16, (N, 15), generator=g, dtype=torch.uint8)):
        w = sg.sgmv_base_pack(codes.to(DEV), torch.ones(N, 15).to(BF16).to(DEV), None if zero is None else zero.to(DEV),
                              K=K, group=64)
        x = torch.randint(-3, 4, (T, K), generator=g).to(BF16).to(DEV)
        want = sg.sgmv_base_product(x, w)
        for n in (1, 2, 5, 8):
            assert torch.equal(sg.sgmv_base_product(x, w, n_split=n), want)
        for rows in (1, 4, 5, 16, 17, 32, 33):  # other instances of the kernel of few rows
            assert torch.equal(sg.sgmv_base_product(x[:rows], w), want[:rows])


@pytest.mark.parametrize("N,T", [(4096, 16), (8192, 3), (8208, 5), (16384, 9), (16400, 16), (8192, 40), (16384, 33)])
def test_wide_weights_of_few_rows(sg, N, T):
    """The instances that take several tiles of columns and rows."""
    w = Weight(sg, N, 200, "i4", BF16, 128, True)
    x = torch.randn(T, 200, generator=torch.Generator().manual_seed(T)).to(BF16)
    w.check(sg.sgmv_base_product(x.to(DEV), w.packed), x)
    w = Weight(sg, N, 200, "e2m1", BF16, 32, False)
    w.check(sg.sgmv_base_product(x.to(DEV), w.packed), x)


@pytest.mark.parametrize("T", [1, 5, 20, 100])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product_of_strided_unaligned_rows(sg, T, dtype):
    w = Weight(sg, 70, 264, "i4", dtype, 64, True)
    g = torch.Generator().manual_seed(T)
    for first in (0, 3, 8):
        x = torch.randn(T, 264 + 24, generator=g).to(dtype)[:, first:first + 264]
        y = torch.full((T, 90), 7.0, dtype=dtype, device=DEV)
        xd = torch.full((T, 300), float("nan"), dtype=dtype, device=DEV)[:, first:first + 264].copy_(x)
        assert sg.sgmv_base_product(xd, w.packed, y=y[:, 9:79]) is not None
        w.check(y[:, 9:79], x)
        assert (y[:, :9] == 7).all() and (y[:, 79:] == 7).all()
        assert torch.equal(sg.sgmv_base_product(xd, w.packed), y[:, 9:79])
        if dtype == BF16:
            y.fill_(7.0)
            sg.sgmv_base_product(xd, w.packed, y=y[:, 9:79], n_split=2)
            w.check(y[:, 9:79], x)
            assert (y[:, :9] == 7).all() and (y[:, 79:] == 7).all()


@pytest.mark.parametrize("fmt,zero", [("i4", True), ("e2m1", False)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [6, 90, 200])
def test_rows_that_are_not_finite_spoil_their_own_results_only(sg, fmt, zero, dtype, T):
    w = Weight(sg, 48, 384, fmt, dtype, 32, zero)
    clean = torch.randn(T, 384, generator=torch.Generator().manual_seed(2)).to(dtype)
    x = clean.clone()
    x[1, 7], x[3, 383], x[T - 2, 200] = float("nan"), float("inf"), float("-inf")
    bad = [1, 3, T - 2]
    good = [t for t in range(T) if t not in bad]
    for n in (0, 2) if dtype == BF16 else (0,):
        want = sg.sgmv_base_product(clean.to(DEV), w.packed, n_split=n)
        y = sg.sgmv_base_product(x.to(DEV), w.packed, n_split=n)
        assert torch.equal(y[good], want[good])
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[3]).any() and not torch.isfinite(y[T - 2]).any()


@pytest.mark.parametrize("T", [1, 30, 200])
def test_every_code_is_its_value(sg, T):
    """One code per row of the weight, against x of whole numbers: sums are exact."""
    for fmt, K in (("i4", 320), ("e2m1", 320)):
        codes = torch.arange(16, dtype=torch.uint8)[:, None].expand(16, K)
        packed = (codes[:, ::2] | codes[:, 1::2] << 4).contiguous()
        x = torch.randint(-4, 5, (T, K), generator=torch.Generator().manual_seed(T)).to(BF16)
        total = x.double().sum(1)
        if fmt == "i4":
            scale, value, form = torch.full((16, 10), 0.5).to(BF16), 0.5 * (torch.arange(16.).double() - 8), sg.BASE_I4
        else:
            scale, form = torch.full((16, 10), 126, dtype=torch.uint8), sg.BASE_E2M1
            value = 0.5 * torch.from_numpy(np.concatenate([lo.E2M1, -lo.E2M1]))
        w = sg.sgmv_base_pack(packed.to(DEV), scale.to(DEV), group=32, format=form)
        y = sg.sgmv_base_product(x.to(DEV), w)
        assert torch.equal(y.cpu(), (total[:, None] * value).to(BF16))


def test_scales_of_e2m1_over_their_range(sg):
    """Exponents at both ends, and 255, which is NaN and reaches its own n only."""
    K, exps = 64, [0, 1, 2, 60, 127, 200, 252, 255]
    scale = torch.tensor(exps, dtype=torch.uint8)[:, None].expand(8, 2).contiguous()
    scale[:, 1] = 127
    codes = torch.full((8, 32), 0x22, dtype=torch.uint8)  # 1.0
    x = torch.zeros(3, K)
    x[:, 0] = torch.tensor([1.0, -2.0, 0.5])
    x[:, 40] = torch.tensor([0.0, 0.0, 2.0 ** -20])
    for dtype in (BF16, F32):
        w = sg.sgmv_base_pack(codes.to(DEV), scale.to(DEV), group=32, format=sg.BASE_E2M1, dtype=dtype)
        y = sg.sgmv_base_product(x.to(dtype).to(DEV), w).double().cpu()
        assert torch.isnan(y[:, 7]).all()
        ref = x[:, :1].double() * 2.0 ** (torch.tensor(exps[:7]).double() - 127) + x[:, 40:41].double()
        # (products below 2^-126 may come out as 0: the matrix cores)
        assert ((y[:, :7] - ref).abs() <= (2.0 ** -8 if dtype == BF16 else 2.0 ** -23) * ref.abs() + 2.0 ** -126).all()


def test_base_then_delta(sg):
    """The base product with the delta added to it, as a layer has them."""
    import oracle
    import workloads
    w = workloads.custom(M=33, K=256, N=160, L=5, R=16, no_lora_frac=0.2, seed=4, name="base")
    base = Weight(sg, 160, 256, "i4", BF16, 64, True)
    pool = sg.sgmv_pool_pack(w.a.to(DEV), w.b.to(DEV), w.rank.tolist(), w.alpha.tolist())
    x = w.x.to(DEV)
    y = sg.sgmv_base_product(x, base.packed)
    base.check(y, w.x)
    y0 = y.float().cpu().numpy()
    sg.sgmv_lora_delta_ids(w.ids.to(DEV), x, pool, sg.sgmv_segments_alloc(33, 5, 0, DEV), y)
    ref = oracle.lora_delta(w.x.float().numpy(), y0, w.ids.numpy(), w.a.float().numpy(), w.b.float().numpy(),
                            w.rank.numpy(), w.alpha.numpy())
    assert np.linalg.norm(y.float().cpu().numpy() - ref) <= 5e-3 * np.linalg.norm(ref)


def test_no_rows_and_captured_calls(sg):
    w = Weight(sg, 256, 512, "i4", BF16, 128, True)
    assert sg.sgmv_base_product(torch.empty(0, 512, dtype=BF16, device=DEV), w.packed).shape == (0, 256)
    g = torch.Generator().manual_seed(5)
    for T, n in ((3, 0), (150, 0), (150, 3)):
        x = torch.randn(T, 512, generator=g).to(BF16).to(DEV)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            first = sg.sgmv_base_product(x, w.packed, n_split=n)
        side.synchronize()
        w.check(first, x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = sg.sgmv_base_product(x, w.packed, n_split=n)
        for _ in range(3):
            x.copy_(torch.randn(T, 512, generator=g))
            graph.replay()
            want = sg.sgmv_base_product(x, w.packed, n_split=n)
            torch.cuda.synchronize()
            assert torch.equal(y, want)
            w.check(y, x)
