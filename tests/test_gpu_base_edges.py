"""GPU tests of the base product at the edges of what it states: all 24 bits of fp32 rows, the smallest values and weights.

In the first, rows of x have one value that is not zero, a whole number with bits in the first, the second and the last eight of its 24, so
that each of the three bf16 parts that the kernels make of it counts. Codes and zero points are such that every sum
on the way is a whole multiple of the code's power of two below 2^24 of it, whatever the order of the parts (z a power of two
and codes 0, z and 2 z, or 0 and z / 2; z = 0 and codes powers of two), and scales are powers of two: results are equal to the
exact ones, which no bar of roundings can say (a row without its last part is off by 2^-16 of itself, the bars of long sums allow more).
"""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32 = torch.float32


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import segmented_gather_gemv_amd as m
    return m


def _parts(v):
    """The leading eight bits of fp32 values, the next of what is left, and the last."""
    out = []
    for _ in range(3):
        top = (v.view(np.uint32) & 0xffff0000).view(np.float32)
        out.append(top)
        v = v - top
    assert not v.any()
    return out


def _rows(T, K, g):
    """One number a row, over all of K."""
    v = 2 ** 23 + 2 ** 15 + 2 * torch.randint(0, 64, (T,), generator=g) + 1
    v = v + (torch.randint(0, 2 ** 7, (T,), generator=g) << 16) + (torch.randint(0, 2 ** 7, (T,), generator=g) << 8)
    v = v.float() * torch.where(torch.rand(T, generator=g) < 0.5, -1.0, 1.0)
    assert all((p != 0).all() for p in _parts(v.numpy()))
    at = (torch.arange(T) * K // T + torch.randint(0, max(1, K // T), (T,), generator=g)).clamp(max=K - 1)
    at[-1] = K - 1
    x = torch.zeros(T, K)
    x[torch.arange(T), at] = v
    return x


def _weight(sg, N, K, fmt, group, zero, g):
    G = -(-K // group)
    if fmt == "e2m1":
        code = torch.tensor([0, 1, 2, 4, 6, 9, 10, 12, 14])[torch.randint(0, 9, (N, K), generator=g)]  # 0, 0.5, 1, 2, 4
        scale = torch.randint(117, 137, (N, G), generator=g, dtype=torch.uint8)
        z = None
    else:
        z = torch.tensor([0, 1, 2, 4, 8])[torch.randint(0, 5, (N, G), generator=g)] if zero else None
        of = (torch.full((N, G), 8) if z is None else z).repeat_interleave(group, 1)[:, :K]
        pick = torch.randint(0, 3, (N, K), generator=g)
        code = torch.where(of == 0, 2 ** pick, torch.where(of == 8, 4 * pick, of * pick))
        scale = 2.0 ** torch.randint(-10, 10, (N, G), generator=g)
        z = None if z is None else z.to(torch.uint8)
    code = torch.cat([code, code.new_zeros(N, K % 2)], 1).to(torch.uint8)
    packed = code[:, ::2] | code[:, 1::2] << 4
    dev = lambda t: None if t is None else t.to(DEV)
    base = sg.sgmv_base_pack(dev(packed), dev(scale), dev(z), K=K, group=group, dtype=F32,
                             format=sg.BASE_E2M1 if fmt == "e2m1" else sg.BASE_I4)
    value, _ = lo.base_weight(packed.numpy(), K, scale.numpy(), None if z is None else z.numpy(), group, fmt)
    return base, value


FORMS = [("i4", 128, False), ("i4", 128, True), ("i4", 64, True), ("i4", 32, False), ("i4", 32, True), ("i4", 512, True),
         ("e2m1", 32, False)]


@pytest.mark.parametrize("fmt,group,zero", FORMS)
@pytest.mark.parametrize("T,N,K,splits", [(1, 40, 300, (0, 1)), (5, 33, 2048, (0, 1, 2, 16)), (16, 272, 1029, (0, 2)), (17, 1100, 700, (0, 1, 3)),
                                          (65, 300, 4000, (0, 1, 2, 16)), (340, 1500, 10050, (0, 1, 16)), (480, 700, 15403, (0, 1)),
                                          (1200, 1801, 1100, (0,))])
def test_every_bit_of_fp32_rows(sg, T, N, K, splits, fmt, group, zero):
    g = torch.Generator().manual_seed(T + N)
    base, value = _weight(sg, N, K, fmt, group, zero, g)
    x = _rows(T, K, g)
    want = torch.from_numpy(x.double().numpy() @ value.T)
    assert torch.equal(want.float().double(), want)
    for n in splits:
        assert torch.equal(sg.sgmv_base_product(x.to(DEV), base, n_split=n).cpu(), want.float()), n


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("T", [3, 70])
def test_values_below_what_the_parts_hold(sg, T, zero):
    """Bits below 2^-133 do not enter, in the products and in the zero points' share alike: with weights of 1 (codes
    9, zeros 8) a row is off by less than 2^-133 for its one value, and its result's own rounding."""
    K, N = 300, 40
    g = torch.Generator().manual_seed(T)
    codes = torch.full((N, K // 2), 0x99, dtype=torch.uint8, device=DEV)
    z = torch.full((N, 5), 8, dtype=torch.uint8, device=DEV) if zero else None
    base = sg.sgmv_base_pack(codes, torch.ones(N, 5, device=DEV), z, group=64)
    x = torch.zeros(T, K)
    v = torch.ldexp(1 + torch.rand(T, generator=g, dtype=torch.float64), -(13 * torch.arange(T) % 30) - 110).float()
    x[torch.arange(T), torch.randint(0, K, (T,), generator=g)] = v
    v = v.double()[:, None]
    for n in (0, 1, 2):
        y = sg.sgmv_base_product(x.to(DEV), base, n_split=n).cpu().double()
        # (9 x and 8 x are rounded before they are subtracted: 2^-24 of each)
        assert ((y - v).abs() <= 2.0 ** -133 + 18 * 2.0 ** -24 * v).all(), n


@pytest.mark.parametrize("dtype", [torch.bfloat16, F32])
@pytest.mark.parametrize("T", [1, 20, 70])
def test_every_weight_of_e2m1(sg, T, dtype):
    """All codes with all scales against single values that are powers of two: exact, weights and results below 2^-126
    among them; weights past fp32 are infinite (here met by zeros too: NaN), and so for scales of 255, NaN."""
    K, i = 32, torch.arange(16 * 256)
    code, scale = (i % 16).to(torch.uint8), (i // 16).to(torch.uint8)
    packed = (code | code << 4)[:, None].expand(len(i), K // 2).contiguous()
    base = sg.sgmv_base_pack(packed.to(DEV), scale[:, None].to(DEV), group=32, format=sg.BASE_E2M1, dtype=dtype)
    value = torch.from_numpy(np.concatenate([lo.E2M1, -lo.E2M1]))[code.long()] * torch.exp2(scale.double() - 127)
    lost = (value.abs() >= 2.0 ** 128) | (scale == 255)
    assert lost.sum() == 12 + 16
    for e in (0, -20, 20):
        x = torch.zeros(T, K)
        x[:, 3] = 2.0 ** e
        y = sg.sgmv_base_product(x.to(dtype).to(DEV), base).cpu()
        assert torch.isnan(y[:, lost]).all()
        assert torch.equal(y[:, ~lost], (value * 2.0 ** e).to(dtype)[None, ~lost].expand(T, -1))
