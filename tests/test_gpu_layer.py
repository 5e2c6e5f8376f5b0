"""The norm, the base product, the delta, the rotated append and the attention one after another, as a layer runs them.

Each call is held against its own oracle over what the call before it gave, so that every bar is that call's alone (they
are derived in the calls' own tests): norm test_gpu_norm.py, product test_gpu_base.py, queries and cache bytes equal,
test_gpu_append.py. The attention after them is compared with the one over a cache that sgmv_kv_write filled with keys
turned beforehand: equal caches and queries give equal outputs.
"""
import importlib.util
import os

import pytest
import torch

from test_gpu_append import _table, _turned
from test_gpu_base import Weight
from test_gpu_kv import BF16, DEV, E4M3, F32, I8, Step, _raw, _same
from test_gpu_norm import _check

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serving_steps.py")
L, R = 3, 16


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import segmented_gather_gemv_amd as m
    return m


class Layer:
    def __init__(self, sg, st, width, Hq, H, D, fmt, dtype, group=64, zero=False):
        self.sg, self.Hq, self.H, self.D, self.st, self.dtype = sg, Hq, H, D, st, dtype
        n = (Hq + 2 * H) * D
        self.qkv = Weight(sg, n, width, fmt, dtype, 32 if fmt == "e2m1" else group, zero)
        self.norm_in = (1 + 0.1 * st.randn(width)).to(dtype)
        self.norm_q = (1 + 0.1 * st.randn(D)).to(dtype)
        # (values of the product are of any size: the norm of the heads brings them to order)
        self.pool = sg.sgmv_pool_pack((st.randn(L, R, width) * width ** -0.5).to(dtype).to(DEV),
                                      (st.randn(L, n, R) * R ** -0.5).to(dtype).to(DEV), [R] * L, [float(R)] * L)
        self.ids = (torch.arange(st.T, dtype=torch.int32) % (L + 1) - 1).to(DEV)
        self.table = _table(max(st.kv_len) + 1, D // 2 * 2)
        self.dev = [t.to(DEV) for t in (self.norm_in, self.norm_q, self.table)]
        self.seg = sg.sgmv_segments_alloc(st.T, L, 0, torch.device(DEV))

    def run(self, x, residual):
        """The layer's calls. Returns what each gave."""
        sg, (w_in, w_q, table) = self.sg, self.dev
        normed = sg.sgmv_rms_norm(x, w_in, residual=residual)
        y = sg.sgmv_base_product(normed.out, self.qkv.packed)
        base = y.clone()
        sg.sgmv_lora_delta_ids(self.ids, normed.out, self.pool, self.seg, y)
        q, k, v = (t.unflatten(1, (-1, self.D)) for t in y.split([self.Hq * self.D, self.H * self.D, self.H * self.D], 1))
        before = y.clone()
        sg.sgmv_rms_norm(q, w_q, out=q)
        sg.sgmv_rms_norm(k, w_q, out=k)
        turned = sg.sgmv_kv_append(q, k, v, self.st.batch, self.st.cache, table)
        out, _ = sg.sgmv_kv_attention(turned, self.st.batch, self.st.cache)
        return normed, base, before, q, k, v, turned, out

    def check(self, x, residual, got, other):
        """other: a Step of the same batch whose cache takes rows turned beforehand."""
        normed, base, before, q, k, v, turned, out = got
        _check(normed, x, self.norm_in, 1e-6, residual, None)
        self.qkv.check(base, normed.out.cpu())
        q0, k0, _ = (t.unflatten(1, (-1, self.D)) for t in before.split(
            [self.Hq * self.D, self.H * self.D, self.H * self.D], 1))
        for a, b in ((q0, q), (k0, k)):
            _check(self.sg.Normed(b, None, None, None), a, self.norm_q, 1e-6, None, None)
        assert _same(turned, _turned(self.st, q.cpu(), self.table, False).to(self.dtype))
        rows = _turned(self.st, k.cpu(), self.table, False)
        held = self.dtype if other.fmt in (BF16, F32) else F32  # (codes are of turned rows before they are rounded)
        self.sg.sgmv_kv_write(rows.to(held).to(DEV), v.to(held).contiguous(), other.batch, other.cache)
        for a, b in ((self.st.cache.k, other.cache.k), (self.st.cache.v, other.cache.v)):
            assert _same(_raw(a), _raw(b).cpu())
        again, _ = self.sg.sgmv_kv_attention(turned, other.batch, other.cache)
        assert bool(torch.isfinite(out).all()) and torch.equal(out, again)


STEPS = {
    # name: new, kv_len, width, query heads, heads, D, cache, rows, weight, zero
    "decode_bf16_i4": ([1, 1, 1], [30, 5, 64], 512, 8, 2, 64, BF16, BF16, "i4", True),
    "chunk_bf16_e2m1": ([70, 1, 9], [70, 20, 40], 320, 4, 2, 64, BF16, BF16, "e2m1", False),
    "odd_f32_i4": ([5, 19], [50, 19], 301, 6, 2, 48, F32, F32, "i4", False),
    "ragged_i8_i4": ([33, 0, 2], [40, 7, 12], 256, 6, 3, 80, I8, BF16, "i4", False),
    "one_e4m3_e2m1": ([1], [1], 256, 4, 1, 128, E4M3, BF16, "e2m1", False),
}


def _make(sg, name):
    new, kv_len, width, Hq, H, D, cache, rows, fmt, zero = STEPS[name]
    st, other = (Step(sg, new, kv_len, 16, H, D, cache, seed=7, rows=rows) for _ in range(2))
    st.fill(sg)
    other.fill(sg)  # (the same)
    layer = Layer(sg, st, width, Hq, H, D, fmt, rows, zero=zero)
    return layer, other, [(st.randn(st.T, width).to(rows), st.randn(st.T, width).to(rows)) for _ in range(3)]


@pytest.mark.parametrize("name", sorted(STEPS))
def test_the_layers_calls_one_after_another(sg, name):
    layer, other, inputs = _make(sg, name)
    for x, r in inputs:
        layer.check(x, r, layer.run(x.to(DEV), r.to(DEV)), other)


@pytest.mark.parametrize("name", ["decode_bf16_i4", "chunk_bf16_e2m1"])
def test_the_layers_calls_captured_and_replayed(sg, name):
    layer, other, inputs = _make(sg, name)
    x, r = (t.to(DEV) for t in inputs[0])
    layer.run(x, r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.run(x, r)
    for a, b in inputs:
        x.copy_(a)
        r.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        layer.check(a, b, got, other)


def test_two_steps_at_once_on_two_streams(sg):
    """Layers of their own on streams of their own."""
    both = [_make(sg, n) for n in ("decode_bf16_i4", "chunk_bf16_e2m1")]
    streams = [torch.cuda.Stream() for _ in both]
    dev = [[(x.to(DEV), r.to(DEV)) for x, r in inputs] for _, _, inputs in both]
    for (layer, _, _), d in zip(both, dev):
        layer.run(*d[0])
    torch.cuda.synchronize()
    for i in range(3):
        got = []
        for (layer, _, _), d, s in zip(both, dev, streams):
            with torch.cuda.stream(s):
                got.append(layer.run(*d[i]))
        torch.cuda.synchronize()
        for (layer, other, inputs), g in zip(both, got):
            layer.check(*inputs[i], g, other)


def _far(rows, width, dtype):
    """Rows 2^27 elements apart: the last ones lie past 2^32 elements."""
    step = 1 << 27
    return torch.empty((rows - 1) * step + width, dtype=dtype, device=DEV).as_strided((rows, width), (step, 1))


def test_rows_past_32_bits(sg):
    T, K, N = 36, 300, 272
    g = torch.Generator().manual_seed(5)
    w = Weight(sg, N, K, "i4", BF16, 64, True)
    x, y = _far(T, K, BF16), _far(T, N, BF16)
    x.copy_(torch.randn(T, K, generator=g).to(BF16))
    for n in (0, 1, 2):
        y.fill_(7.0)
        sg.sgmv_base_product(x, w.packed, y, n_split=n)
        w.check(y.contiguous(), x.cpu())
    weight = torch.randn(K, generator=g).to(BF16)
    keep, W = x.cpu(), N - 7
    got = sg.sgmv_rms_norm(x[:, :W], weight[:W].to(DEV), residual=x[:, 8:8 + W], out=y[:, 3:3 + W], quantise=I8)
    _check(got._replace(out=got.out.contiguous()), keep[:, :W], weight[:W], 1e-6, keep[:, 8:8 + W], I8)


@pytest.mark.parametrize("new", [[1, 2, 1], [40, 3, 17]])
@pytest.mark.parametrize("fmt", [BF16, I8])
def test_append_into_pages_past_32_bits(sg, fmt, new):
    H, D, ps, pages = 8, 256, 64, 20000 if fmt == BF16 else 36000
    lens = [n + 50 for n in new]
    cache = sg.sgmv_kv_init(pages, ps, H, D, fmt, DEV)
    small = Step(sg, new, lens, ps, H, D, fmt, seed=9)
    start = small.batch.q_start
    far = torch.from_numpy(small.table).to(DEV)
    far = torch.where(far >= 0, far + (pages - small.pages), far)
    batch = sg.sgmv_kv_batch(start, small.batch.kv_len, far, small.T, max(new), max(lens))
    g = torch.Generator().manual_seed(6)
    k, v, q = (torch.randn(small.T, h, D, generator=g).to(BF16).to(DEV) for h in (H, H, 16))
    table = _table(max(lens), 192).to(DEV)
    for c in (cache, small.cache):
        for t in (c.k, c.v):
            _raw(t)[-small.pages:].zero_()
        for t in (c.k_scale, c.v_scale) if fmt == I8 else ():
            t[-small.pages:].fill_(1.0)
    a = sg.sgmv_kv_append(q, k, v, batch, cache, table)
    b = sg.sgmv_kv_append(q, k, v, small.batch, small.cache, table)
    assert torch.equal(a, b)
    for far_part, part in ((cache.k, small.cache.k), (cache.v, small.cache.v)):
        assert torch.equal(_raw(far_part)[-small.pages:], _raw(part))
    out = [sg.sgmv_kv_attention(a, x, c)[0] for x, c in ((batch, cache), (small.batch, small.cache))]
    assert torch.equal(*out)


@pytest.mark.parametrize("N", [1, 16, 20, 48])
def test_narrow_weights_of_many_rows(sg, N):
    for dtype in (BF16, F32):
        w = Weight(sg, N, 200, "i4", dtype, 128, True)
        x = torch.randn(9000, 200, generator=torch.Generator().manual_seed(N)).to(dtype)
        w.check(sg.sgmv_base_product(x.to(DEV), w.packed), x)


@pytest.mark.parametrize("base,fmt", [("i4", "bf16"), ("i4", "i8"), ("e2m1", "e4m3")])
def test_serving_steps_of_a_whole_layer(sg, base, fmt, capsys):
    spec = importlib.util.spec_from_file_location("serving_steps", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main(["--cache", fmt, "--base", base, "--steps", "6"]) == 0
    assert "sequence 2" in capsys.readouterr().out
