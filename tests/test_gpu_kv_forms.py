"""GPU parity of the attention's forms and of the cache's and draft check's paths that small cases do not
reach: tiles of every head dimension and type, workgroups of four and eight waves, sequences of few rows beside
tiles of many, values that are not finite in places that a product pads or masks.

The bars are those of test_gpu_kv (derived there). Where two calls have to give the same rows (a mixed
step and its sequences one by one), both are within them of the fp64 oracle.
"""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as ko
from test_gpu_kv import (BF16, DEV, E4M3, F32, I8, NAMES, Step, _check_attention, _check_scales,
                         _expected_cache, _i32, _raw, _same)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import segmented_gather_gemv_amd as m
    return m


def _run(sg, new, kv_len, ps, Hq, H, D, fmt, rows, window=0, holes=(), n_splits=(0, 3), check=None, seed=21):
    st = Step(sg, new, kv_len, ps, H, D, fmt, seed=seed, rows=rows, holes=holes)
    kv = st.fill(sg)
    q = st.randn(st.T, Hq, D).to(rows)
    for n_split in n_splits:
        out, lse = sg.sgmv_kv_attention(q.to(DEV), st.batch, st.cache, window=window, n_split=n_split)
        _check_attention(st, q, kv, out, lse, D ** -0.5, window, rows=check)


def _some(new, each=7):
    """About `each` rows of every sequence, the first and the last among them."""
    return {(b, i) for b, n in enumerate(new) for i in list(range(0, n, max(1, n // each))) + [n - 1] if n}


@pytest.mark.parametrize("fmt", [BF16, E4M3, I8])
@pytest.mark.parametrize("D", [64, 80, 96, 128, 192, 256])
def test_tiles_of_every_dimension(sg, D, fmt):
    """Chunks of many rows beside single tokens, several tiles of tokens, pages that end inside a tile."""
    new = [150, 1, 0, 37, 1]
    _run(sg, new, [333, 250, 9, 37, 64], 16, 6, 2, D, fmt, BF16, check=_some(new))


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("D", [80, 128, 256])
def test_tiles_with_a_window_and_missing_pages(sg, D, fmt):
    new = [120, 2]
    _run(sg, new, [400, 300], 32, 4, 1, D, fmt, BF16, window=90, check=_some(new),
         holes=[(0, 8, -1), (0, 11, 1 << 29), (1, 9, -1), (1, 4, -1)])


@pytest.mark.parametrize("fmt", [BF16, E4M3, I8])
@pytest.mark.parametrize("D", [16, 48, 64, 80, 96, 112, 128, 160, 192, 208, 256])
def test_few_rows_of_every_dimension(sg, D, fmt):
    """Up to 16 rows, and up to 32, per key/value head."""
    _run(sg, [1, 3, 1], [300, 90, 17], 16, 4, 1, D, fmt, BF16)
    _run(sg, [3, 5, 1], [150, 70, 6], 32, 5, 1, D, fmt, BF16)


@pytest.mark.parametrize("fmt", [F32, E4M3, I8])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 144, 192, 256])
def test_fp32_rows_of_every_dimension(sg, D, fmt):
    _run(sg, [1, 2], [200, 90], 16, 4, 2, D, fmt, F32)
    _run(sg, [11, 40], [60, 100], 32, 2, 1, D, fmt, F32, window=50)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("B,new", [(80, 1), (70, 6)])
def test_many_sequences(sg, fmt, B, new):
    """Enough sequences that a workgroup has four waves, of lengths from their new tokens on."""
    lens = [new + (37 * b) % 300 for b in range(B)]
    _run(sg, [new] * B, lens, 16, 32, 8, 64, fmt, BF16, n_splits=(0, 2),
         check={(b, i) for b in range(0, B, 9) for i in (0, new - 1)})


def test_long_sequences_are_split_and_joined(sg):
    """More parts than are joined side by side, of sequences that have fewer."""
    for fmt, D, n in ((E4M3, 128, 10000), (BF16, 64, 3000), (F32, 80, 1500)):
        _run(sg, [1, 1, 2], [n, 40, n // 3], 64, 4, 2, D, fmt, F32 if fmt == F32 else BF16,
             n_splits=(0, 7, 64))


def test_a_mixed_step_is_its_sequences(sg):
    """Sequences of few and of many rows in one call: each as it is alone, to the rounding of its parts."""
    new, kv_len = [70, 1, 8, 300, 1, 9, 2], [70, 513, 200, 420, 1, 64, 2000]
    st = Step(sg, new, kv_len, 32, 2, 128, BF16, seed=4)
    kv = st.fill(sg)
    q = st.randn(st.T, 8, 128).to(BF16)
    out, lse = sg.sgmv_kv_attention(q.to(DEV), st.batch, st.cache)
    _check_attention(st, q, kv, out, lse, 128 ** -0.5, rows=_some(new))
    for b in range(len(new)):
        lo, hi = st.start[b], st.start[b + 1]
        one = sg.sgmv_kv_batch(_i32([0, new[b]]), _i32([kv_len[b]]), st.batch.page_table[b:b + 1], new[b], new[b],
                               kv_len[b])
        o, l = sg.sgmv_kv_attention(q[lo:hi].to(DEV), one, st.cache)
        # both within the oracle's bars, with A at most the largest |v|, and S of any row
        k64, v64 = (torch.from_numpy(x[b]) for x in kv)
        S = max(float((q[lo:hi, h].double().abs() @ k64[:, h // 4].abs().T).max()) for h in range(8)) * 128 ** -0.5
        e = 2 * (132 * 2.0 ** -24 * S + 2.0 ** -22 + S * 2.0 ** -23 + kv_len[b] * 2.0 ** -24)
        ref = torch.maximum(o.double().abs(), out[lo:hi].double().abs()).cpu() * (1 + 2.0 ** -7)
        most = 2 * (2.0 ** -8 * ref + (2.0 ** -8 + 2.0 ** -23 + e) * float(v64.abs().max()))
        assert ((o.double() - out[lo:hi].double()).abs().cpu() <= most).all(), b
        assert float((l - lse[lo:hi]).abs().max()) <= 2 * (e + 2.0 ** -22 * (float(l.abs().max()) + 6)), b


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("fmt,rows", [(BF16, BF16), (F32, F32), (E4M3, BF16)])
def test_a_row_that_sees_only_nan_is_nan(sg, new, fmt, rows):
    """With a window of one token, and a token of NaN: nothing else is in its row's sums."""
    st = Step(sg, [new], [new + 200], 16, 1, 64, fmt, rows=rows)
    st.fill(sg)
    k, v = st.randn(new, 1, 64).to(rows), st.randn(new, 1, 64).to(rows)
    k[new - 1, 0, 9] = float("nan")
    sg.sgmv_kv_write(k.to(DEV), v.to(DEV), st.batch, st.cache)
    q = st.randn(new, 8, 64).to(rows).to(DEV)
    for n_split in (0, 4):
        out, lse = sg.sgmv_kv_attention(q, st.batch, st.cache, window=1, n_split=n_split)
        assert torch.isnan(out[new - 1]).all() and torch.isnan(lse[new - 1]).all()
        assert torch.isfinite(out[:new - 1]).all() and torch.isfinite(lse[:new - 1]).all()


@pytest.mark.parametrize("D", [48, 80, 112, 128, 208])
@pytest.mark.parametrize("fmt,rows", [(BF16, BF16), (F32, F32)])
def test_keys_of_minus_infinity_hide_their_token(sg, D, fmt, rows):
    """Scores of -inf (a key of -inf, a positive query) are tokens of no weight, also where the head
    dimension is padded with zeros of the query."""
    st = Step(sg, [1], [50], 16, 1, D, fmt, rows=rows)
    kv = st.fill(sg)
    k, v = st.randn(50, 1, D).to(rows), st.randn(50, 1, D).to(rows)
    k[20, 0, D - 1] = float("-inf")
    k[33, 0, 0] = float("-inf")
    whole = sg.sgmv_kv_batch(_i32([0, 50]), _i32([50]), st.batch.page_table, 50, 50, 50)
    sg.sgmv_kv_write(k.to(DEV), v.to(DEV), whole, st.cache)
    q = st.randn(1, 2, D).abs().to(rows) + 0.5
    out, lse = sg.sgmv_kv_attention(q.to(DEV), st.batch, st.cache)
    keep = [i for i in range(50) if i not in (20, 33)]
    st.new, st.kv_len = [1], [48]
    _check_attention(st, q, ([k.double().numpy()[keep]], [v.double().numpy()[keep]]), out, lse, D ** -0.5)


@pytest.mark.parametrize("D", [80, 128])
def test_nonfinite_values_in_tiles_with_wide_workgroups(sg, D):
    """inf and NaN in V at a token that part of a tile's rows see, other rows as without them."""
    st = Step(sg, [200], [330], 16, 1, D, BF16)
    st.fill(sg)
    k, v = st.randn(200, 1, D).to(BF16), st.randn(200, 1, D).to(BF16)
    odd = v.clone()
    odd[100, 0, D - 1], odd[100, 0, 0], odd[150, 0, 17] = float("inf"), float("-inf"), float("nan")
    for i in (100, 150):
        v[i] = 0.25
    q = st.randn(200, 4, D).to(BF16).to(DEV)
    got = []
    for x in (v, odd):
        sg.sgmv_kv_write(k.to(DEV), x.to(DEV), st.batch, st.cache)
        got.append(sg.sgmv_kv_attention(q, st.batch, st.cache))
    (ref, ref_lse), (out, lse) = got
    assert torch.equal(lse, ref_lse) and torch.equal(out[:100], ref[:100])
    assert (out[100:, :, D - 1] == float("inf")).all() and (out[100:, :, 0] == float("-inf")).all()
    assert torch.isnan(out[150:, :, 17]).all() and torch.isfinite(out[100:150, :, 17]).all()


# ---- cache ------------------------------------------------------------------------------
@pytest.mark.parametrize("new", [3, 40])
@pytest.mark.parametrize("D", [16, 80, 128, 256])
@pytest.mark.parametrize("fmt,rows", [(E4M3, BF16), (I8, F32), (BF16, BF16), (F32, F32)])
def test_writes_of_every_dimension(sg, new, D, fmt, rows):
    """By rows (few tokens of each sequence) and by groups of tokens: every byte, and the rows back."""
    news = [new, 0, max(1, new // 2), new]
    st = Step(sg, news, [new, 5, 90, 16 + new], 16, 3, D, fmt, seed=8, rows=rows)
    k, v = st.randn(st.T, 3, D).to(rows), st.randn(st.T, 3, D).to(rows)
    bufs, scales = _expected_cache(st, k, v)
    sg.sgmv_kv_write(k.to(DEV), v.to(DEV), st.batch, st.cache)
    assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])
    if fmt in NAMES:
        _check_scales(st.cache.k_scale, scales[0])
        _check_scales(st.cache.v_scale, scales[1])
    a = sg.sgmv_kv_read(st.batch, st.cache, st.batch.q_start, st.T, rows)
    if fmt not in NAMES:
        assert torch.equal(a[0].cpu(), k) and torch.equal(a[1].cpu(), v)
    # the other path of the read: more rows than tokens
    pad = [0]
    for n in news:
        pad.append(pad[-1] + (n + 60 if n else 0))
    b = sg.sgmv_kv_read(st.batch, st.cache, _i32(pad), pad[-1], rows)
    for i, n in enumerate(news):
        for x, y in zip(a, b):
            assert torch.equal(x[st.start[i]:st.start[i + 1]], y[pad[i + 1] - n:pad[i + 1]])


@pytest.mark.parametrize("fmt", [E4M3, I8])
def test_quotients_on_a_border_go_to_the_even_code(sg, fmt):
    """Rows whose quotients x F / amax are borders of the format, exactly: 0.65625 lies between the e4m3
    codes 50 and 51."""
    st = Step(sg, [12], [12], 16, 2, 32, fmt)
    k = torch.zeros(12, 2, 32)
    for i, (x, top) in enumerate([(0.01190185546875, 8.125), (0.031494140625, 21.5), (0.0177001953125, 8.75)]):
        k[i, :, 0], k[i, :, 1], k[i, :, 2] = top, x, -x
    for i in range(3, 12):  # amax 127 * 2^n: quotients of int8 are the values, halves among them
        k[i, :, 0] = 127.0 * 2.0 ** (i - 6)
        k[i, :, 1:] = (torch.arange(31) - 15.5) * 2.0 ** (i - 6)
    k = k.to(BF16)
    bufs, _ = _expected_cache(st, k, k)
    sg.sgmv_kv_write(k.to(DEV), k.to(DEV), st.batch, st.cache)
    assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])
    if fmt == E4M3:
        lay = ko.Cache(16, 32, 1)
        page = st.table[0, 0]
        got = [int(_raw(st.cache.k).cpu().reshape(st.pages, 2, -1)[page, 0, lay.k_index(i)[1]]) for i in range(3)]
        assert got == [50, 50, 54]


@pytest.mark.parametrize("by_rows", [True, False])
@pytest.mark.parametrize("fmt,rows", [(E4M3, BF16), (I8, BF16), (E4M3, F32), (I8, F32)])
def test_rows_of_every_magnitude(sg, fmt, rows, by_rows):
    """Maxima of every exponent of the type, subnormal ones too, beside rows of zeros and of NaN: one sequence's
    tokens (by groups), or each its own (by rows)."""
    exps = list(range(-149 if rows is F32 else -133, 128))
    T = len(exps)
    st = Step(sg, [1] * T if by_rows else [T], [5] * T if by_rows else [T + 3], 16, 2, 48, fmt, seed=14, rows=rows)
    k = st.randn(T, 2, 48)
    k = (k / k.abs().amax(-1, keepdim=True)).double() * 1.99
    k = k * torch.tensor([2.0 ** e for e in exps], dtype=torch.float64)[:, None, None]
    k = k.to(torch.float32).to(rows)
    assert torch.isfinite(k).all()
    k[::17, 0] = 0
    k[5::31, 1, 40] = float("nan")
    bufs, scales = _expected_cache(st, k, k)
    sg.sgmv_kv_write(k.to(DEV), k.to(DEV), st.batch, st.cache)
    assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])
    _check_scales(st.cache.k_scale, scales[0])
    _check_scales(st.cache.v_scale, scales[1])


@pytest.mark.parametrize("fmt", [E4M3, I8])
def test_every_quotient_of_two_bf16_significands(sg, fmt):
    """Rows with each significand as their maximum, and each other one below it in nine binades and a few far
    down: every border that a quotient can lie on or next to."""
    small = torch.tensor([(128 + m) * 2.0 ** -e for e in (8, 9, 10, 11, 12, 13, 14, 15, 16, 17, 18, 24)
                          for m in range(128)])
    per = 240
    rows = []
    for top in range(128, 256):
        x = small[small < top / 128.0] * torch.tensor([1.0, -1.0]).repeat(len(small))[:int((small < top / 128.0).sum())]
        for i in range(0, len(x), per - 1):
            row = torch.full((per,), top / 128.0)
            row[1:1 + len(x[i:i + per - 1])] = x[i:i + per - 1]
            rows.append(row)
    if len(rows) % 2:
        rows.append(rows[0])
    k = torch.stack(rows).reshape(-1, 2, per)
    assert torch.equal(k.to(BF16).float(), k)
    k = k.to(BF16)
    T = k.shape[0]
    st = Step(sg, [T], [T + 3], 64, 2, per, fmt, seed=2)
    bufs, _ = _expected_cache(st, k, k)
    sg.sgmv_kv_write(k.to(DEV), k.to(DEV), st.batch, st.cache)
    assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])


def test_rows_of_sequences_with_different_counts(sg):
    """Writes and reads by rows where a sequence's number is not its share of the tokens."""
    news = [0] * 30 + [8, 1] + [0] * 5 + [2] * 3 + [0, 7]
    lens = [max(n, (11 * i) % 50) for i, n in enumerate(news)]
    st = Step(sg, news, lens, 16, 2, 64, I8, seed=6)
    k, v = st.randn(st.T, 2, 64).to(BF16), st.randn(st.T, 2, 64).to(BF16)
    bufs, _ = _expected_cache(st, k, v)
    sg.sgmv_kv_write(k.to(DEV), v.to(DEV), st.batch, st.cache)
    assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])
    a = sg.sgmv_kv_read(st.batch, st.cache, st.batch.q_start, st.T)
    back = sum(ko.quantise(k.double().numpy(), "i8")[0].reshape(-1).astype(int) != 0)
    assert int((a[0] != 0).sum()) == back


# ---- drafts -----------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [1024, 1025, 4099, 70001])
def test_draws_at_the_borders_of_parts(sg, V, dtype):
    """One entry carries nearly all the weight, at the ends of the parts that a row is summed in, and the
    numbers that fall right before, into and behind it."""
    places = sorted({0, 15, 16, 1023, min(1024, V - 1), V // 2, V - 2, V - 1})
    us = [0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24]
    B = len(places) * len(us)
    t = torch.full((B, V), 2.0 ** -30)
    for b in range(B):
        t[b, places[b // len(us)]] = 0.5
    t = t.to(dtype)
    su = torch.tensor([us[b % len(us)] for b in range(B)])
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    tokens, accepted = sg.sgmv_verify_drafts(t.to(DEV), None, none, _i32([0] * (B + 1)),
                                             torch.empty(0, device=DEV), su.to(DEV), 0)
    assert (accepted == 0).all()
    for b in range(B):
        ref, _ = ko.verify(t[b:b + 1].float().numpy(), None, [], [], float(su[b]))
        assert tokens[b].cpu().tolist() == ref, (b, places[b // len(us)], us[b % len(us)])


@pytest.mark.parametrize("V", [16384, 16385, 20001, 32767, 32768, 32769])
def test_draws_of_rows_in_one_launch_and_in_two(sg, V):
    """Rows of as many parts as one workgroup does, one more and fewer: weights at their ends, and rejected
    drafts that leave nothing (the draft at least as likely everywhere; all weight on a certain draft), where
    the token comes from the target's own row."""
    places = sorted({0, 1023, 1024, 16383, min(16384, V - 1), V // 2 + 1, V - 2, V - 1})
    us = [0.0, 0.3, 0.5, 0.7, 1 - 2.0 ** -24]
    cases = [(p, u) for p in places for u in us]
    B = len(cases)
    t = torch.zeros(2 * B, V)
    d = torch.zeros(B, V)
    for b, (p, _) in enumerate(cases):
        t[2 * b, p], t[2 * b, (p + V // 3) % V] = 0.25, 0.125
        d[b, p], d[b, (p + V // 3) % V] = 0.5, 0.25
        if b % 3 == 0:  # something left, in one place
            t[2 * b, (p + V // 2) % V] = 0.0625
        t[2 * b + 1, p] = 1.0
    ids = [p for p, _ in cases]
    au = [0.25 if b % 7 == 6 else 0.75 for b in range(B)]
    su = [u for _, u in cases]
    for draft in (d, None):
        if draft is None:
            for b, (p, _) in enumerate(cases):
                if b % 3 == 1:
                    t[2 * b] = 0
                    t[2 * b, p] = 0.25
        tokens, accepted = sg.sgmv_verify_drafts(
            t.to(DEV), None if draft is None else draft.to(DEV), _i32(ids), _i32(list(range(B + 1))),
            torch.tensor(au, device=DEV), torch.tensor(su, device=DEV), 1)
        for b in range(B):
            ref, taken = ko.verify(t[2 * b:2 * b + 2].numpy(), None if draft is None else draft[b:b + 1].numpy(),
                                   ids[b:b + 1], au[b:b + 1], su[b])
            assert accepted[b].item() == taken, b
            assert tokens[b].cpu().tolist() == ref + [-1] * (1 - taken), (b, cases[b])
