"""GPU parity of the paged cache, its attention and the draft check against the fp64 oracle.

Bars, element by element:
  * written codes, scales and every byte around them: equal. Scales are one fp32 division of the
    row's exact amax (equal to torch's); codes are the oracle's rounding of the exact quotient.
  * read back: code * scale in fp32, rounded once to bf16: equal to torch's product and rounding.
  * attention, with A = sum p |v| / sum p and S = the largest scale |q| . |k| of the row: a score is
    a sum of D exact (bf16) or once rounded (fp32) products, so it is off by at most
    (D + 4) 2^-24 S, and its exponential by 2^-22 more (argument in base 2 and exp2, |s| < 2^5 for
    these inputs adds |s| 2^-23); the sums over n tokens by n 2^-24. e = that, twice (numerator
    and denominator). bf16 rows round each probability (2^-8 A; 2 * 2^-24 for the scales) and
    the output (2^-8 |ref|), fp32 rows only the output (2^-24 |ref|).
    |out - ref| <= r |ref| + (r_p + e) A,  |lse - ref| <= e + 2^-22 (|ref| + 6).
  * tokens and counts of the draft check: equal.
Unwritten cache memory, missing pages and places outside the rows are poisoned with NaN.
"""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as ko

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = {torch.float8_e4m3fn: "e4m3", torch.int8: "i8"}
F32, BF16, E4M3, I8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.int8


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import segmented_gather_gemv_amd as m
    return m


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _raw(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t


class Step:
    """Sequences with n new tokens each, kv_len tokens in all, pages in shuffled order."""

    def __init__(self, sg, new, kv_len, ps, H, D, fmt, seed=0, spare=2, holes=(), rows=BF16,
                 max_q=None):
        g = self.g = torch.Generator().manual_seed(seed)
        self.new, self.kv_len, self.ps, self.H, self.D, self.fmt = new, kv_len, ps, H, D, fmt
        need = [-(-v // ps) for v in kv_len]
        self.pages = sum(need) + spare
        ids = torch.randperm(self.pages, generator=g).tolist()
        cols = max(max(need), 1) + 1
        self.table = np.full((len(new), cols), -1, np.int32)
        for b, n in enumerate(need):
            for i in range(n):
                self.table[b, i] = ids.pop()
        for b, i, v in holes:
            self.table[b, i] = v
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(int)
        self.T = int(self.start[-1])
        self.cache = sg.sgmv_kv_init(self.pages, ps, H, D, fmt, DEV)
        poison = {F32: float("nan"), BF16: float("nan")}.get(fmt)
        for t in (self.cache.k, self.cache.v):  # e4m3 0x7f is NaN
            t.fill_(poison) if poison is not None else _raw(t).fill_(0x7f)
        if fmt in NAMES:
            self.cache.k_scale.fill_(float("nan"))
            self.cache.v_scale.fill_(float("nan"))
        self.batch = sg.sgmv_kv_batch(_i32(self.start.tolist()), _i32(kv_len),
                                      torch.from_numpy(self.table).to(DEV), self.T,
                                      max(new) if max_q is None else max_q, max(kv_len))
        self.rows = rows

    def page_ok(self, b):
        return [0 <= p < self.pages for p in self.table[b]]

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g)

    def fill(self, sg, std=1.0):
        """Write every existing token of every sequence through the write call; returns the values
        the cache then stands for, fp64 [tokens][H][D] per sequence (NaN where there is no page)."""
        keep = [max(0, v) for v in self.kv_len]
        T = sum(keep)
        k, v = (self.randn(T, self.H, self.D) * std).to(self.rows), self.randn(T, self.H, self.D).to(self.rows)
        start = np.concatenate([[0], np.cumsum(keep)]).astype(int)
        b = sg.sgmv_kv_batch(_i32(start.tolist()), _i32(self.kv_len), self.batch.page_table, T, max(keep),
                             max(keep))
        sg.sgmv_kv_write(k.to(DEV), v.to(DEV), b, self.cache)
        out = []
        for x in (k, v):
            y = x.double().numpy()
            if self.fmt in NAMES:
                code, scale = ko.quantise(y, NAMES[self.fmt])
                val = ko.e4m3_value(code) if self.fmt == E4M3 else code.astype(np.float64)
                # the scale as stored
                y = val * np.float32(abs(y).max(-1).astype(np.float32) / np.float32(ko.TOP[NAMES[self.fmt]])
                                     ).astype(np.float64)[..., None]
            out.append([y[start[i]:start[i + 1]] for i in range(len(keep))])
        return out


def _expected_cache(st, k, v):
    """The cache's bytes and scales after writing rows k, v [T, H, D], from its present ones."""
    name = NAMES.get(st.fmt)
    lay = ko.Cache(st.ps, st.D, st.cache.k.element_size())
    per = st.ps * st.D
    bufs = [_raw(t).cpu().reshape(st.pages, st.H, per) for t in (st.cache.k, st.cache.v)]
    bufs = [b.clone() for b in bufs]
    scales = [None if t is None else t.cpu().clone() for t in (st.cache.k_scale, st.cache.v_scale)]
    for which, x in enumerate((k, v)):
        if name:
            code, sc = ko.quantise(x.double().numpy(), name)
            code = torch.from_numpy(code.view(np.uint8))
            amax = x.float().abs().amax(-1)
            s32 = amax / np.float32(ko.TOP[name])
            s32[~torch.from_numpy(np.isfinite(sc))] = float("nan")
        for b in range(len(st.new)):
            for i in range(st.new[b]):
                pos = st.kv_len[b] - st.new[b] + i
                if pos < 0 or not st.page_ok(b)[pos // st.ps]:
                    continue
                page, off, row = st.table[b, pos // st.ps], pos % st.ps, st.start[b] + i
                idx = torch.from_numpy((lay.k_index if which == 0 else lay.v_index)(off))
                for h in range(st.H):
                    bufs[which][page, h, idx] = code[row, h] if name else x[row, h]
                    if name:
                        scales[which][page, h, off] = s32[row, h]
    return bufs, scales


def _same(a, b):
    a, b = a.cpu().reshape(-1), b.reshape(-1)
    if a.dtype in (F32, BF16):
        a, b = a.view(torch.int32 if a.dtype == F32 else torch.int16), b.view(torch.int32 if b.dtype == F32 else torch.int16)
    return torch.equal(a, b)


def _check_scales(got, ref):
    got = got.cpu()
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], ref[~nan])


WRITES = {
    # name: new, kv_len, page size, heads, D, format, row type
    "one_token_bf16": ([1], [1], 16, 1, 16, BF16, BF16),
    "decode_e4m3": ([1, 1, 1], [17, 64, 5], 16, 3, 64, E4M3, BF16),
    "ragged_i8": ([5, 0, 40, 1], [21, 7, 40, 33], 32, 2, 80, I8, BF16),
    "ragged_e4m3_f32": ([19, 3], [30, 70], 16, 2, 96, E4M3, F32),
    "wide_i8_f32": ([33], [50], 64, 2, 256, I8, F32),
    "wide_bf16": ([33, 2], [50, 300], 128, 2, 256, BF16, BF16),
    "f32": ([7, 18], [7, 33], 16, 2, 48, F32, F32),
    "more_new_than_tokens": ([6, 4], [2, 0], 16, 2, 64, E4M3, BF16),
    "many_sequences": ([1, 0, 2] * 50, [9, 4, 40] * 50, 16, 1, 32, I8, BF16),
}


@pytest.mark.parametrize("name", sorted(WRITES))
def test_write_leaves_exactly_the_rows_codes(sg, name):
    new, kv_len, ps, H, D, fmt, rows = WRITES[name]
    st = Step(sg, new, kv_len, ps, H, D, fmt, seed=3, rows=rows)
    k = (st.randn(st.T, H, D) * torch.exp(3 * st.randn(st.T, H, 1))).to(rows)
    v = (st.randn(st.T, H, D) * torch.exp(3 * st.randn(st.T, H, 1))).to(rows)
    bufs, scales = _expected_cache(st, k, v)
    sg.sgmv_kv_write(k.to(DEV), v.to(DEV), st.batch, st.cache)
    assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])
    if fmt in NAMES:
        _check_scales(st.cache.k_scale, scales[0])
        _check_scales(st.cache.v_scale, scales[1])
    # and back: the new tokens, code * scale rounded once
    ko_, vo = sg.sgmv_kv_read(st.batch, st.cache, st.batch.q_start, st.T, rows)
    for got, buf, sc, index in ((ko_, bufs[0], scales[0], "k_index"), (vo, bufs[1], scales[1], "v_index")):
        lay = ko.Cache(ps, D, st.cache.k.element_size())
        for b in range(len(new)):
            for i in range(new[b]):
                pos = kv_len[b] - new[b] + i
                if pos < 0:
                    continue
                page, off = st.table[b, pos // ps], pos % ps
                x = buf[page][:, torch.from_numpy(getattr(lay, index)(off))].contiguous()
                x = x.view(fmt).float() if fmt in NAMES else x.float()
                if sc is not None:
                    x = x * sc[page, :, off][:, None]
                assert _same(got[st.start[b] + i], x.to(rows)), (b, i)


@pytest.mark.parametrize("fmt", [E4M3, I8])
@pytest.mark.parametrize("rows", [BF16, F32])
def test_write_of_zeros_extremes_and_nonfinite_rows(sg, fmt, rows):
    st = Step(sg, [9], [9], 16, 1, 64, fmt, rows=rows)
    k = st.randn(9, 1, 64)
    k[0] = 0
    k[1] *= 2.0 ** 120
    k[1, 0, 3] = 3.38e38
    k[2] *= 2.0 ** -100
    k[3, 0, 7] = float("inf")
    k[4, 0, 63] = float("nan")
    k[5, 0, 0] = float("-inf")
    k[6] = -0.0
    k[7] = 1.0
    k[8, 0, 1:] = 0  # one value alone
    k = k.to(rows)
    bufs, scales = _expected_cache(st, k, k)
    # a row of zeros has codes 0 whatever the zeros' signs
    sg.sgmv_kv_write(k.to(DEV), k.to(DEV), st.batch, st.cache)
    assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])
    _check_scales(st.cache.k_scale, scales[0])
    back, _ = sg.sgmv_kv_read(st.batch, st.cache, st.batch.q_start, 9, rows)
    back = back.cpu().float()
    assert torch.isnan(back[3:6]).all() and torch.isfinite(back[[0, 1, 2, 6, 7, 8]]).all()


def test_write_reads_slices_of_a_fused_projection(sg):
    """k and v as unaligned column slices of one wide row."""
    st = Step(sg, [3, 20], [40, 20], 16, 2, 48, E4M3)
    wide = st.randn(23, 7 + 2 * 96 + 5).to(BF16).to(DEV)
    k, v = wide[:, 7:103].unflatten(1, (2, 48)), wide[:, 103:199].unflatten(1, (2, 48))
    bufs, _ = _expected_cache(st, k.cpu(), v.cpu())
    sg.sgmv_kv_write(k, v, st.batch, st.cache)
    assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])


def test_missing_pages_are_not_written_and_read_as_zeros(sg):
    st = Step(sg, [40, 40], [48, 48], 16, 2, 64, E4M3, holes=[(0, 1, -1), (1, 2, 1 << 30), (1, 0, 999)])
    k, v = st.randn(80, 2, 64).to(BF16), st.randn(80, 2, 64).to(BF16)
    bufs, _ = _expected_cache(st, k, v)
    sg.sgmv_kv_write(k.to(DEV), v.to(DEV), st.batch, st.cache)
    assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])
    ko_, vo = sg.sgmv_kv_read(st.batch, st.cache, st.batch.q_start, 80)
    zero = [b * 40 + i for b in range(2) for i in range(40) if not st.page_ok(b)[(8 + i) // 16]]
    assert len(zero) == 16 + 16 + 8
    assert (ko_[zero] == 0).all() and (vo[zero] == 0).all()
    rest = [i for i in range(80) if i not in zero]
    assert not torch.isnan(ko_[rest]).any()


def test_read_whole_sequences_into_strided_rows(sg):
    st = Step(sg, [1, 1, 1], [33, 1, 70], 32, 2, 80, I8)
    kv = st.fill(sg)
    out = [0, 33, 34, 104]
    buf = torch.full((104, 2, 200), 7.0, dtype=BF16, device=DEV)
    k, v = buf[:, :, 3:83], buf[:, :, 100:180]
    sg.sgmv_kv_read(st.batch, st.cache, _i32(out), 104, BF16, k=k, v=v)
    for got, ref in ((k, kv[0]), (v, kv[1])):
        ref = torch.from_numpy(np.concatenate(ref))
        # code * scale in fp32 (2^-24) and bf16 (2^-8)
        assert ((got.cpu().double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -23) * ref.abs()).all()
    assert (buf[:, :, :3] == 7).all() and (buf[:, :, 83:100] == 7).all() and (buf[:, :, 180:] == 7).all()
    # the last tokens only, and more than there are: rows before the first token are zeros
    k2 = torch.full((60, 2, 80), 7.0, dtype=BF16, device=DEV)
    v2 = k2.clone()
    sg.sgmv_kv_read(st.batch, st.cache, _i32([0, 10, 15, 60]), 60, BF16, k=k2, v=v2)
    assert torch.equal(k2[:10], k[23:33]) and torch.equal(k2[14], k[33]) and torch.equal(v2[15:], v[59:])
    assert (k2[10:14] == 0).all() and (v2[10:14] == 0).all()


# ---- attention --------------------------------------------------------------------------
def _check_attention(st, q, kv, out, lse, scale, window=0, rows=None):
    Hq, G, T = q.shape[1], q.shape[1] // st.H, st.T
    q64 = q.double().cpu().numpy()
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    bf16 = q.dtype == BF16
    r = 2.0 ** -8 if bf16 else 2.0 ** -24
    rp = 2.0 ** -8 + 2.0 ** -23 if bf16 else 2.0 ** -23
    for b in range(len(st.new)):
        ok = st.page_ok(b)
        for i in range(st.new[b]):
            if rows is not None and (b, i) not in rows:
                continue
            t = ko.visible(st.kv_len[b], st.new[b], i, window, ok, st.ps)
            row = st.start[b] + i
            for h in range(Hq):
                ref, l, A, S = ko.attention_row(q64[row, h], kv[0][b][t, h // G], kv[1][b][t, h // G], scale)
                e = 2 * ((st.D + 4) * 2.0 ** -24 * S + 2.0 ** -22 + S * 2.0 ** -23 + len(t) * 2.0 ** -24)
                d = abs(out[row, h] - ref)
                lim = r * abs(ref) + (rp + e) * A
                assert (d <= lim).all(), (b, i, h, float((d - lim).max()), len(t))
                if len(t) == 0:
                    assert lse[row, h] == -np.inf
                else:
                    assert abs(lse[row, h] - l) <= e + 2.0 ** -22 * (abs(l) + 6), (b, i, h, lse[row, h], l)


ATTENTION = {
    # name: new, kv_len, page size, heads, kv heads, D, format, rows, window
    "one_token_of_one": ([1], [1], 16, 1, 1, 16, BF16, BF16, 0),
    "decode": ([1, 1, 1], [1, 100, 333], 16, 8, 2, 128, BF16, BF16, 0),
    "decode_mha": ([1, 1], [31, 200], 32, 3, 3, 64, BF16, BF16, 0),
    "decode_mqa_40_heads": ([1, 2], [65, 97], 16, 40, 1, 64, BF16, BF16, 0),
    "decode_e4m3": ([1, 1], [500, 16], 64, 8, 2, 128, E4M3, BF16, 0),
    "decode_i8_256": ([1, 1], [129, 16], 128, 4, 2, 256, I8, BF16, 0),
    "drafts_i8": ([4, 2, 5], [64, 300, 5], 16, 14, 2, 128, I8, BF16, 0),
    "drafts_80": ([3, 6], [70, 300], 16, 4, 2, 80, E4M3, BF16, 0),
    "odd_dims_48": ([3, 1], [70, 30], 16, 4, 2, 48, I8, BF16, 0),
    "odd_dims_208": ([9, 1], [70, 30], 32, 4, 2, 208, BF16, BF16, 0),
    "zero_length_and_empty": ([0, 1, 0, 3, 0], [5, 9, 0, 3, 40], 16, 4, 2, 64, BF16, BF16, 0),
    "rows_before_the_first_token": ([5, 3, 2], [2, 0, 30], 16, 4, 2, 64, BF16, BF16, 0),
    "chunk": ([70, 33], [70, 300], 16, 4, 2, 128, BF16, BF16, 0),
    "chunk_g7": ([45, 100], [200, 130], 32, 7, 1, 128, BF16, BF16, 0),
    "chunk_e4m3_64": ([130], [400], 64, 4, 2, 64, E4M3, BF16, 0),
    "chunk_i8": ([90, 1, 64], [100, 50, 64], 128, 4, 1, 128, I8, BF16, 0),
    "chunk_past_empty_rows": ([100], [60], 16, 4, 1, 128, BF16, BF16, 0),
    "window_1": ([40, 1], [90, 40], 16, 4, 2, 64, BF16, BF16, 1),
    "window_17": ([60, 3], [200, 150], 16, 4, 2, 128, BF16, BF16, 17),
    "window_e4m3": ([150, 2], [300, 270], 32, 4, 1, 128, E4M3, BF16, 100),
    "mixed": ([120, 1, 1, 40, 1], [200, 300, 5, 40, 77], 16, 8, 2, 128, BF16, BF16, 0),
    "f32": ([5, 1, 30], [77, 140, 30], 16, 6, 2, 80, F32, F32, 0),
    "f32_i8_256": ([2, 1], [77, 40], 16, 2, 1, 256, I8, F32, 0),
    "f32_e4m3_window": ([20, 1], [77, 140], 16, 4, 2, 64, E4M3, F32, 33),
}


@pytest.mark.parametrize("n_split", [0, 3])
@pytest.mark.parametrize("name", sorted(ATTENTION))
def test_attention_against_oracle(sg, name, n_split):
    new, kv_len, ps, Hq, H, D, fmt, rows, window = ATTENTION[name]
    st = Step(sg, new, kv_len, ps, H, D, fmt, seed=11, rows=rows)
    kv = st.fill(sg)
    q = st.randn(st.T, Hq, D).to(rows)
    out, lse = sg.sgmv_kv_attention(q.to(DEV), st.batch, st.cache, window=window, n_split=n_split)
    _check_attention(st, q, kv, out, lse, D ** -0.5, window)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("new", [1, 90])
def test_attention_skips_missing_pages(sg, fmt, new):
    """Evicted pages (-1), ids out of range, and a sequence with no page at all."""
    st = Step(sg, [new, new, new], [170, 100, 96], 16, 2, 128, fmt,
              holes=[(0, 0, -1), (0, 4, -7), (0, 5, 1 << 20), (0, 10, -1)] + [(1, i, -1) for i in range(7)])
    kv = st.fill(sg)
    q = st.randn(st.T, 8, 128).to(BF16)
    for n_split in (0, 2):
        out, lse = sg.sgmv_kv_attention(q.to(DEV), st.batch, st.cache, n_split=n_split)
        _check_attention(st, q, kv, out, lse, 128 ** -0.5)


@pytest.mark.parametrize("fmt,rows", [(BF16, BF16), (F32, F32), (E4M3, BF16), (I8, BF16)])
@pytest.mark.parametrize("G", [2, 8])
def test_nonfinite_values_reach_only_rows_that_see_them(sg, fmt, rows, G):
    """A token with NaN, one with +inf in V, one with -inf: earlier rows of the same tiles are as if
    they were not there, later ones are not finite where the formula is not."""
    st = Step(sg, [70], [100], 16, 1, 64, fmt, rows=rows)
    st.fill(sg)
    k, v = st.randn(70, 1, 64).to(rows), st.randn(70, 1, 64).to(rows)
    k[40, 0, 3] = float("nan")
    v[25, 0, 5] = float("inf")
    v[30, 0, 6] = float("-inf")
    v[35, 0, 6] = float("inf")
    v[50, 0, 7] = float("nan")
    q = st.randn(70, G, 64).to(rows).to(DEV)
    clean_k, clean_v = k.clone(), v.clone()
    for i in (25, 30, 35, 40, 50):
        clean_k[i], clean_v[i] = 0.5, 0.5
    sg.sgmv_kv_write(clean_k.to(DEV), clean_v.to(DEV), st.batch, st.cache)
    ref, ref_lse = sg.sgmv_kv_attention(q, st.batch, st.cache)
    sg.sgmv_kv_write(k.to(DEV), v.to(DEV), st.batch, st.cache)
    out, lse = sg.sgmv_kv_attention(q, st.batch, st.cache)
    assert torch.isfinite(ref).all()
    assert torch.equal(out[:25], ref[:25]) and torch.equal(lse[:25], ref_lse[:25])
    assert torch.isnan(out[40:]).all() and torch.isnan(lse[40:]).all()  # a NaN score spoils the row
    assert torch.isfinite(lse[:40]).all()
    if fmt in NAMES:  # the whole row reads as NaN
        assert torch.isnan(out[25:]).all()
    else:
        assert (out[25:40, :, 5] == float("inf")).all()
        assert (out[30:35, :, 6] == float("-inf")).all() and torch.isnan(out[35:40, :, 6]).all()
        other = [d for d in range(64) if d not in (5, 6, 7)]
        assert torch.isfinite(out[:40][:, :, other]).all()


def test_attention_of_strided_rows_on_another_stream(sg):
    """q as an unaligned slice of a wider row, out and lse given, everything on a side stream."""
    st = Step(sg, [40, 1], [60, 200], 16, 2, 64, BF16)
    kv = st.fill(sg)
    wide = st.randn(41, 300).to(BF16)
    outs = []
    for first in (0, 3):
        q = wide[:, first:first + 256].unflatten(1, (4, 64))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            qd = wide.to(DEV)[:, first:first + 256].unflatten(1, (4, 64))
            buf = torch.full((41, 4, 70), 7.0, dtype=BF16, device=DEV)
            lse = torch.empty(41, 4, device=DEV)
            out, l2 = sg.sgmv_kv_attention(qd, st.batch, st.cache, out=buf[:, :, first:first + 64], lse=lse,
                                           scale=0.2, n_split=2)
        s.synchronize()
        assert l2 is lse and (buf[:, :, first + 64:] == 7).all()
        _check_attention(st, q, kv, out, lse, 0.2)
        outs.append(out)


def test_attention_is_the_same_every_time(sg):
    st = Step(sg, [300, 1, 1], [500, 900, 30], 32, 2, 128, E4M3)
    st.fill(sg)
    q = st.randn(st.T, 8, 128).to(BF16).to(DEV)
    for n_split in (0, 5):
        first = sg.sgmv_kv_attention(q, st.batch, st.cache, n_split=n_split)
        for _ in range(5):
            again = sg.sgmv_kv_attention(q, st.batch, st.cache, n_split=n_split)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_large_scores_and_growing_maxima(sg):
    """Scores that grow along the sequence, over hundreds of powers of two: the running maximum
    is carried, not the first one."""
    st = Step(sg, [2, 80], [400, 80], 16, 1, 64, F32, rows=F32)
    k = torch.zeros(480, 1, 64)
    pos = torch.cat([torch.arange(400), torch.arange(80)]).float()
    k[:, 0, 0] = pos
    v = st.randn(480, 1, 64)
    b = sg.sgmv_kv_batch(_i32([0, 400, 480]), _i32([400, 80]), st.batch.page_table, 480, 400, 400)
    sg.sgmv_kv_write(k.to(DEV), v.to(DEV), b, st.cache)
    q = torch.zeros(82, 2, 64)
    q[:, 0, 0], q[:, 1, 0] = 8.0, -8.0
    out, lse = sg.sgmv_kv_attention(q.to(DEV), st.batch, st.cache, scale=1.0)
    for i in range(82):
        n = 399 + i if i < 2 else i - 1
        vv = v[:400] if i < 2 else v[400:]
        w = torch.exp(-8.0 * torch.arange(n).double())
        w /= w.sum()
        up, down = (w[:, None] * vv[:n, 0].flip(0).double()).sum(0), (w[:, None] * vv[:n, 0].double()).sum(0)
        assert (out[i, 0].cpu().double() - up).abs().max() < 1e-5
        assert (out[i, 1].cpu().double() - down).abs().max() < 1e-5
        # scores are exact; lse is one fp32 number of that size
        assert abs(float(lse[i, 0]) - 8.0 * (n - 1)) <= 2.0 ** -21 * (8.0 * n + 1) + 4e-4
        assert abs(float(lse[i, 1])) <= 4e-4


def test_offsets_past_32_bits(sg):
    """A cache of 2^32 bytes and more of K: its last pages."""
    H, D, ps = 8, 128, 256
    pages = (1 << 32) // (H * D * ps) + 40
    cache = sg.sgmv_kv_init(pages, ps, H, D, I8, DEV)
    g = torch.Generator().manual_seed(5)
    for new in (1, 90):
        table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=DEV)
        low = torch.tensor([[3, 2]], dtype=torch.int32, device=DEV)
        k, v = (torch.randn(300, H, D, generator=g).to(BF16).to(DEV) for _ in range(2))
        q = torch.randn(new, 16, D, generator=g).to(BF16).to(DEV)
        got = []
        for t in (table, low):
            whole = sg.sgmv_kv_batch(_i32([0, 300]), _i32([300]), t, 300, 300, 300)
            sg.sgmv_kv_write(k, v, whole, cache)
            step = sg.sgmv_kv_batch(_i32([0, new]), _i32([300]), t, new, new, 300)
            got.append(sg.sgmv_kv_attention(q, step, cache) + sg.sgmv_kv_read(whole, cache, whole.q_start, 300))
        for a, b in zip(*got):
            assert torch.equal(a, b)
        assert (got[0][2].float() - k.float()).abs().max() < 0.05


def test_bad_lengths_stay_inside(sg):
    """Lengths past the table, negative lengths and starts past the rows are cut, not followed."""
    st = Step(sg, [2, 2], [30, 30], 16, 1, 64, BF16)
    st.fill(sg)
    k = st.randn(4, 1, 64).to(BF16).to(DEV)
    q = st.randn(4, 2, 64).to(BF16).to(DEV)
    table = st.batch.page_table
    for start, kv in (([0, 2, 4], [1 << 30, -5]), ([0, 900, 3], [30, 30]), ([-4, 2, 1 << 30], [30, 0]),
                      ([3, 1, 0], [30, 30])):
        b = sg.sgmv_kv_batch(_i32(start), _i32(kv), table, 4, 4, 48)
        sg.sgmv_kv_write(k, k, b, st.cache)
        sg.sgmv_kv_attention(q, b, st.cache)
        sg.sgmv_kv_read(b, st.cache, _i32(start), 4)
    torch.cuda.synchronize()


@pytest.mark.parametrize("new,fmt", [(1, BF16), (3, E4M3), (200, BF16)])
def test_step_in_a_graph(sg, new, fmt):
    """Write and attention captured once and replayed with other lengths, pages and values, against
    eager calls."""
    st = Step(sg, [new, new], [400, 400], 32, 2, 128, fmt, spare=20)
    st.fill(sg)
    k, v = (st.randn(st.T, 2, 128).to(BF16).to(DEV) for _ in range(2))
    q = st.randn(st.T, 8, 128).to(BF16).to(DEV)
    out = torch.empty(st.T, 8, 128, dtype=BF16, device=DEV)
    lse = torch.empty(st.T, 8, device=DEV)
    size = sg.sgmv_kv_attention_workspace(8, BF16, st.batch, st.cache, n_split=4)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)

    def step():
        sg.sgmv_kv_write(k, v, st.batch, st.cache)
        sg.sgmv_kv_attention(q, st.batch, st.cache, out=out, lse=lse, n_split=4, workspace=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.synchronize()
    for i in range(4):
        st.batch.kv_len.copy_(_i32([400 - 40 * i, 250 + 30 * i]))
        q.copy_(st.randn(st.T, 8, 128).to(BF16).to(DEV))
        k.copy_(st.randn(st.T, 2, 128).to(BF16).to(DEV))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        out.fill_(7)
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse), i


# ---- drafts -----------------------------------------------------------------------------
VERIFY = {
    # name: drafts of each sequence, vocabulary, type, certain drafts, sharpness
    "one": ([4], 32000, F32, False, 2.5),
    "ragged": ([0, 1, 5, 3, 0, 8], 5003, F32, False, 2.5),
    "bf16": ([3] * 20, 1500, BF16, False, 2.5),
    "certain": ([2, 0, 4] * 10, 777, F32, True, 6.0),
    "vocab_1": ([2, 0], 1, F32, False, 1.0),
    "vocab_3": ([2, 1, 7] * 20, 3, F32, False, 1.0),
    "long_flat": ([2] * 8, 131071, F32, False, 0.1),
    "many_drafts": ([130, 65, 64], 50, BF16, True, 8.0),
}


@pytest.mark.parametrize("name", sorted(VERIFY))
def test_verify_against_oracle(sg, name):
    n, V, dtype, certain, sharp = VERIFY[name]
    g = torch.Generator().manual_seed(9)
    N, B = sum(n), len(n)
    start = np.concatenate([[0], np.cumsum(n)]).astype(int)
    row = torch.tensor([start[b] + b + i for b in range(B) for i in range(n[b])], dtype=torch.long)
    logits = sharp * torch.randn(N + B, V, generator=g)
    target = torch.softmax(logits, 1)
    guess = torch.softmax(logits[row] + 0.5 * torch.randn(N, V, generator=g), 1)
    ids = torch.multinomial(target[row] if certain else guess, 1, generator=g)[:, 0].to(torch.int32)
    if N > 8:
        ids[3], ids[5] = -1, V  # not in the vocabulary
    au, su = torch.rand(N, generator=g), torch.rand(B, generator=g)
    if B > 2:
        su[0], su[1] = 0.0, 1 - 2.0 ** -24
    # rows of a wider matrix, poisoned outside
    target_w = torch.full((N + B, V + 5), float("nan"), dtype=dtype)
    target_w[:, :V] = target.to(dtype)
    draft = None if certain else guess.to(dtype)
    tokens, accepted = sg.sgmv_verify_drafts(target_w.to(DEV)[:, :V], None if certain else draft.to(DEV),
                                             ids.to(DEV), _i32(start.tolist()), au.to(DEV), su.to(DEV), max(n))
    tokens, accepted = tokens.cpu().tolist(), accepted.cpu().tolist()
    for b in range(B):
        lo, hi = start[b], start[b + 1]
        ref, taken = ko.verify(target_w[lo + b:hi + b + 1, :V].float().numpy(),
                               None if certain else draft[lo:hi].float().numpy(), ids[lo:hi].tolist(),
                               au[lo:hi].tolist(), float(su[b]))
        assert accepted[b] == taken, b
        assert tokens[b] == ref + [-1] * (max(n) - taken), b


@pytest.mark.parametrize("V", [7, 3001])
def test_verify_odd_rows(sg, V):
    """Rows of zeros, of entries that are not probabilities, a draft row equal to the target, and
    weights far from 1."""
    t = torch.zeros(8, V)
    d = torch.zeros(4, V)
    t[0, V - 1], d[0, 0] = 1.0, 1.0            # draft 0 certain not to be taken: drawn V - 1
    t[1] = float("nan")
    t[2] = 0.25
    d[1] = 0.25                                # taken unless u = 1
    t[3, 2], t[3, 4], t[3, 5] = float("inf"), -3.0, 1e-30
    t[4], d[2] = 1e-38, 3e-38                  # draft larger everywhere: the rest is all zero
    t[5] = 0
    t[6], t[7] = 0, 0                          # nothing to draw from
    ids = [0, 1, 3, 2]
    start = [0, 1, 2, 3, 4]
    au, su = [0.0, 0.5, 0.5, 0.5], [0.5, 0.999, 0.5, 0.3]
    tokens, accepted = sg.sgmv_verify_drafts(t.to(DEV), d.to(DEV), _i32(ids), _i32(start),
                                             torch.tensor(au, device=DEV), torch.tensor(su, device=DEV), 1)
    for b in range(4):
        ref, taken = ko.verify(t[2 * b:2 * b + 2].numpy(), d[b:b + 1].numpy(), ids[b:b + 1], au[b:b + 1], su[b])
        assert accepted[b].item() == taken
        assert tokens[b].cpu().tolist() == ref + [-1] * (1 - taken), b
    assert tokens[0].cpu().tolist() == [V - 1, -1] and tokens[1].cpu().tolist() == [1, 5]
    assert tokens[2].cpu().tolist()[1] == -1 and tokens[3].cpu().tolist() == [-1, -1]


def test_verify_in_a_graph_and_on_a_side_stream(sg):
    g = torch.Generator().manual_seed(2)
    t = torch.softmax(2 * torch.randn(9, 9001, generator=g), 1).to(DEV)
    d = torch.softmax(2 * torch.randn(6, 9001, generator=g), 1).to(DEV)
    ids, start = _i32([1, 2, 3, 4, 5, 6]), _i32([0, 2, 4, 6])
    au, su = torch.rand(6, generator=g).to(DEV), torch.rand(3, generator=g).to(DEV)
    tokens, accepted = sg.sgmv_verify_drafts(t, d, ids, start, au, su, 2)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            sg.sgmv_verify_drafts(t, d, ids, start, au, su, 2, tokens=tokens, accepted=accepted)
    for i in range(4):
        t.copy_(torch.softmax(2 * torch.randn(9, 9001, generator=g), 1).to(DEV))
        su.copy_(torch.rand(3, generator=g).to(DEV))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref = sg.sgmv_verify_drafts(t, d, ids, start, au, su, 2)
        assert torch.equal(ref[0], tokens) and torch.equal(ref[1], accepted)
