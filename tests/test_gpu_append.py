"""GPU parity of the rotated append against the oracle, and against writing rows that were rotated before.

Bars: every product and sum of the rotation is rounded to fp32 as the oracle rounds it, so that everything is equal, bit
for bit: queries (fp32 values rounded once), and the cache's bytes and scales (tests/test_gpu_kv.py).
"""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from test_gpu_kv import BF16, DEV, E4M3, F32, I8, NAMES, Step, _check_scales, _expected_cache, _i32, _raw, _same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import segmented_gather_gemv_amd as m
    return m


def _table(positions, rotary, seed=0):
    angle = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, rotary, 2) / rotary) + seed
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float()


def _positions(st):
    """Of each row of the step (negative: it does not exist)."""
    return np.concatenate([np.arange(L - n, L) for n, L in zip(st.new, st.kv_len)] or [np.zeros(0, int)])


def _turned(st, x, table, interleaved):
    """fp32 rows; those at negative positions as they were."""
    pos = _positions(st)
    c, s = np.split(table.numpy()[np.clip(pos, 0, None)], 2, 1)
    y = torch.from_numpy(lo.rotate(x.float().numpy(), c, s, interleaved))
    return torch.where(torch.from_numpy(pos >= 0)[:, None, None], y, x.float())


APPENDS = {
    # name: new, kv_len, page size, heads, query heads, D, rotary, format, row type
    "one_token": ([1], [1], 16, 1, 1, 16, 16, BF16, BF16),
    "decode_bf16": ([1, 1, 1], [17, 64, 5], 16, 2, 8, 128, 128, BF16, BF16),
    "decode_e4m3": ([1, 1, 1], [17, 64, 5], 16, 3, 9, 64, 64, E4M3, BF16),
    "decode_i8_part": ([1, 2, 1], [17, 64, 5], 32, 2, 14, 128, 96, I8, BF16),
    "ragged_i8_80": ([5, 0, 40, 1], [21, 7, 40, 33], 32, 2, 4, 80, 80, I8, BF16),
    "ragged_e4m3_f32": ([19, 3], [30, 70], 16, 2, 2, 96, 48, E4M3, F32),
    "wide_i8_f32": ([33], [50], 64, 2, 6, 256, 256, I8, F32),
    "wide_bf16": ([33, 2], [50, 300], 128, 1, 40, 256, 64, BF16, BF16),
    "f32_48": ([7, 18], [7, 33], 16, 2, 5, 48, 32, F32, F32),
    "f32_decode": ([1, 1], [7, 33], 16, 2, 7, 80, 16, F32, F32),
    "chunk_bf16_112": ([70, 9], [70, 300], 16, 2, 4, 112, 112, BF16, BF16),
    "more_new_than_tokens": ([6, 4], [2, 0], 16, 2, 4, 64, 32, E4M3, BF16),
    "more_new_than_tokens_chunk": ([60, 40], [20, 0], 16, 2, 4, 64, 64, I8, BF16),
    "many_sequences": ([1, 0, 2] * 50, [9, 4, 40] * 50, 16, 1, 3, 32, 32, I8, BF16),
    "chunk_16_i8": ([9, 33], [20, 33], 16, 2, 3, 16, 16, I8, BF16),
    "chunk_32_e4m3": ([30, 5, 1], [64, 5, 9], 32, 3, 3, 32, 16, E4M3, F32),
    "four_new_i8": ([4, 3, 1, 4] * 9, [4, 40, 17, 19] * 9, 16, 8, 8, 128, 96, I8, BF16),
    "two_new_bf16": ([2, 1] * 20, [40, 3] * 20, 16, 7, 14, 48, 32, BF16, BF16),
    "many_rows_f32_256": ([1] * 90, [19, 64, 5] * 30, 16, 3, 3, 256, 240, F32, F32),
    "many_tokens": ([700, 500], [700, 800], 64, 1, 32, 128, 128, E4M3, BF16),
    "no_queries": ([1, 20], [9, 40], 16, 2, 0, 64, 64, BF16, BF16),
}


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("name", sorted(APPENDS))
def test_append_against_oracle(sg, name, interleaved):
    new, kv_len, ps, H, Hq, D, rotary, fmt, rows = APPENDS[name]
    st = Step(sg, new, kv_len, ps, H, D, fmt, seed=3, rows=rows)
    k = (st.randn(st.T, H, D) * torch.exp(2 * st.randn(st.T, H, 1))).to(rows)
    v = (st.randn(st.T, H, D) * torch.exp(2 * st.randn(st.T, H, 1))).to(rows)
    q = st.randn(st.T, Hq, D).to(rows) if Hq else None
    table = _table(max(kv_len) + 1, rotary)
    turned = _turned(st, k, table, interleaved)
    if fmt in (BF16, F32):
        turned = turned.to(fmt)
    bufs, scales = _expected_cache(st, turned, v)
    poison = None if q is None else torch.full_like(q, 7.0).to(DEV)
    got = sg.sgmv_kv_append(None if q is None else q.to(DEV), k.to(DEV), v.to(DEV), st.batch, st.cache,
                            table.to(DEV), interleaved, q_out=poison)
    assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])
    if fmt in NAMES:
        _check_scales(st.cache.k_scale, scales[0])
        _check_scales(st.cache.v_scale, scales[1])
    if q is None:
        assert got is None
        return
    # rows at negative positions are not written
    here = torch.from_numpy(_positions(st) >= 0)
    want = torch.where(here[:, None, None], _turned(st, q, table, interleaved).to(rows), torch.full_like(q, 7.0))
    assert got.data_ptr() == poison.data_ptr() and _same(got, want)


@pytest.mark.parametrize("fmt,rows", [(BF16, BF16), (E4M3, BF16), (F32, F32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("new", [2, 30])
def test_append_in_place_of_a_fused_projection(sg, fmt, rows, interleaved, new):
    """q turned in place in unaligned (and then aligned) column slices of one wide row, k and v read from there;
    a table with rows of its own stride."""
    H, Hq, D, rotary = 2, 6, 80, 48
    for first, ld in ((7, rotary + 3), (8, rotary + 4)):
        st = Step(sg, [new, 1, new + 3], [new + 20, 8, new + 3], 16, H, D, fmt, seed=5, rows=rows)
        wide = st.randn(st.T, first + (Hq + 2 * H) * D + 8).to(rows)
        cut = lambda t: [x.unflatten(1, (-1, D)) for x in t[:, first:first + (Hq + 2 * H) * D].split(
            [Hq * D, H * D, H * D], 1)]
        table = torch.full((60, ld), float("nan"))
        table[:, :rotary] = _table(60, rotary)
        q, k, v = cut(wide)
        turned = _turned(st, k, table[:, :rotary], interleaved)
        bufs, _ = _expected_cache(st, turned.to(fmt) if fmt in (BF16, F32) else turned, v)
        dev = wide.to(DEV)
        qd, kd, vd = cut(dev)
        got = sg.sgmv_kv_append(qd, kd, vd, st.batch, st.cache, table.to(DEV)[:, :rotary], interleaved, q_out=qd)
        assert got.data_ptr() == qd.data_ptr()
        assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])
        q[:] = _turned(st, q, table[:, :rotary], interleaved).to(rows)
        assert _same(dev, wide)


def test_missing_pages_keep_queries_and_rows_past_the_table_are_nan(sg):
    st = Step(sg, [40, 40], [48, 48], 16, 2, 64, E4M3, holes=[(0, 1, -1), (1, 2, 1 << 30)])
    q, k, v = (st.randn(80, n, 64).to(BF16) for n in (4, 2, 2))
    table = _table(45, 64)
    full = _table(48, 64)
    full[45:] = float("nan")
    bufs, scales = _expected_cache(st, _turned(st, k, full, False), v)
    got = sg.sgmv_kv_append(q.to(DEV), k.to(DEV), v.to(DEV), st.batch, st.cache, table.to(DEV))
    assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])
    _check_scales(st.cache.k_scale, scales[0])
    want = _turned(st, q, full, False)
    nan = torch.isnan(want)
    assert nan.any() and torch.equal(torch.isnan(got.cpu()), nan) and _same(got[~nan.to(DEV)], want.to(BF16)[~nan])


@pytest.mark.parametrize("new", [1, 20])
def test_rows_of_no_sequence_stay_as_they_were(sg, new):
    """A step padded to more rows than its sequences have, the first ones among them."""
    st = Step(sg, [new, new], [30, 40], 16, 2, 64, BF16)
    T = 2 * new + 9
    start = _i32([4, 4 + new, 4 + 2 * new])
    batch = sg.sgmv_kv_batch(start, st.batch.kv_len, st.batch.page_table, T, new, 40)
    q, k, v = (st.randn(T, n, 64).to(BF16) for n in (4, 2, 2))
    table = _table(40, 64)
    inside = slice(4, 4 + 2 * new)
    bufs, _ = _expected_cache(st, _turned(st, k[inside], table, False).to(BF16), v[inside])
    for t in (q, k, v):
        t[:4], t[4 + 2 * new:] = float("nan"), float("inf")
    out = torch.full((T, 4, 64), 7.0, dtype=BF16, device=DEV)
    sg.sgmv_kv_append(q.to(DEV), k.to(DEV), v.to(DEV), batch, st.cache, table.to(DEV), q_out=out)
    assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])
    assert (out[:4] == 7).all() and (out[4 + 2 * new:] == 7).all()
    assert _same(out[inside], _turned(st, q[inside], table, False).to(BF16))


@pytest.mark.parametrize("fmt", [BF16, I8])
def test_append_of_turns_by_nothing_is_a_write(sg, fmt):
    """With cosines 1 and sines 0 the cache holds what sgmv_kv_write leaves."""
    for new in ([1, 2, 1], [40, 1, 17]):
        st = Step(sg, new, [50, 64, 33], 16, 2, 128, fmt, seed=8)
        k, v = (st.randn(st.T, 2, 128).to(BF16).to(DEV) for _ in range(2))
        table = torch.cat([torch.ones(64, 64), torch.zeros(64, 64)], 1).to(DEV)
        sg.sgmv_kv_write(k, v, st.batch, st.cache)
        want = [t.clone() for t in (_raw(st.cache.k), _raw(st.cache.v))]
        for t in (st.cache.k, st.cache.v):
            _raw(t).zero_()
        sg.sgmv_kv_append(None, k, v, st.batch, st.cache, table)
        again = Step(sg, new, [50, 64, 33], 16, 2, 128, fmt, seed=8)
        sg.sgmv_kv_append(None, k, v, again.batch, again.cache, table)
        assert _same(_raw(again.cache.k), want[0].cpu()) and _same(_raw(again.cache.v), want[1].cpu())


def test_append_captured_and_replayed_with_fewer_tokens(sg):
    """A step of up to two rows of each sequence, captured, on a side stream too; then other rows, lengths and starts."""
    st = Step(sg, [2, 2, 2], [20, 30, 40], 16, 2, 64, E4M3)
    T = 6
    q, k, v = (st.randn(T, n, 64).to(BF16).to(DEV) for n in (4, 2, 2))
    table, out = _table(64, 64).to(DEV), torch.empty(T, 4, 64, dtype=BF16, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        sg.sgmv_kv_append(q, k, v, st.batch, st.cache, table, q_out=out)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sg.sgmv_kv_append(q, k, v, st.batch, st.cache, table, q_out=out)
    for starts, lens in (([0, 2, 4, 6], [22, 31, 42]), ([0, 1, 1, 3], [23, 31, 44]), ([0, 0, 2, 4], [23, 33, 46])):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=st.g))
        st.batch.q_start.copy_(_i32(starts))
        st.batch.kv_len.copy_(_i32(lens))
        out.fill_(7.0)
        graph.replay()
        got = [t.clone() for t in (_raw(st.cache.k), _raw(st.cache.v), st.cache.k_scale, out)]
        out.fill_(7.0)
        sg.sgmv_kv_append(q, k, v, st.batch, st.cache, table, q_out=out)
        torch.cuda.synchronize()
        for a, b in zip(got, (_raw(st.cache.k), _raw(st.cache.v), st.cache.k_scale, out)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert (out[starts[-1]:] == 7).all() and not (out[:starts[-1]] == 7).all()


def test_append_and_attend(sg):
    """What the attention sees after an append is what it sees after turning and writing rows apart."""
    for fmt in (BF16, E4M3):
        st, ref = (Step(sg, [3, 1, 25], [60, 9, 25], 16, 2, 128, fmt, seed=4) for _ in range(2))
        for s in (st, ref):
            s.g.manual_seed(1)
            s.fill(sg)
        q, k, v = (st.randn(st.T, n, 128).to(BF16) for n in (8, 2, 2))
        table = _table(60, 128)
        got = sg.sgmv_kv_append(q.to(DEV), k.to(DEV), v.to(DEV), st.batch, st.cache, table.to(DEV))
        rows = torch.float32 if fmt == E4M3 else BF16
        sg.sgmv_kv_write(_turned(st, k, table, False).to(rows).to(DEV), v.to(rows).to(DEV), ref.batch, ref.cache)
        want = _turned(st, q, table, False).to(BF16).to(DEV)
        for a, b in zip(sg.sgmv_kv_attention(got, st.batch, st.cache), sg.sgmv_kv_attention(want, ref.batch, ref.cache)):
            assert torch.equal(a, b)
