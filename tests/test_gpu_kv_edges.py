"""GPU tests of the edges of the cache's, the attention's and the draft check's contracts: steps padded to a
fixed number of rows, lengths and starts that are cut, sequences of different counts, windows of any width, codes of NaN, draws that fall on the border of a part without a weight.

The bars are those of test_gpu_kv (derived there).
"""
import copy

import numpy as np
import pytest
import torch

from oracle import kv_oracle as ko
from test_gpu_kv import BF16, DEV, E4M3, F32, I8, Step, _check_attention, _expected_cache, _i32, _raw, _same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import segmented_gather_gemv_amd as m
    return m


# ---- steps of more rows than their sequences have ------------------------------------------
PADDED = {
    # name: new tokens, length, rows of the step's largest sequence, query heads, key/value heads, D
    "one_short": ([8], [300], 256, 8, 2, 128),
    "one_token": ([1], [90], 64, 4, 1, 64),
    "long_short_empty": ([64, 1, 0, 33], [200, 150, 40, 33], 64, 8, 2, 128),
    "all_empty_but_the_last": ([0, 0, 3], [5, 0, 70], 40, 4, 1, 96),
    "wide": ([2, 50], [60, 170], 50, 8, 2, 256),
    "no_tiles_of_this_dimension": ([2, 50], [60, 170], 50, 8, 2, 112),
}


def _padded(sg, st, max_q):
    """The step's batch with room for max_q rows of every sequence; q_start ends before them."""
    return sg.sgmv_kv_batch(st.batch.q_start, st.batch.kv_len, st.batch.page_table, len(st.new) * max_q, max_q,
                            max(st.kv_len))


def _pad(x, T):
    """Rows x on the GPU, followed by rows of NaN."""
    y = torch.full((T, *x.shape[1:]), float("nan"), dtype=x.dtype)
    y[:x.shape[0]] = x
    return y.to(DEV)


@pytest.mark.parametrize("fmt,rows", [(BF16, BF16), (E4M3, BF16), (I8, BF16), (F32, F32)])
@pytest.mark.parametrize("name", sorted(PADDED))
def test_padded_steps(sg, name, fmt, rows):
    """Sequences of any number of rows up to max_q, in a step of B max_q rows: each row of a sequence is
    there, and rows of none are not touched."""
    new, kv_len, max_q, Hq, H, D = PADDED[name]
    st = Step(sg, new, kv_len, 16, H, D, fmt, seed=17, rows=rows)
    kv = st.fill(sg)
    batch = _padded(sg, st, max_q)
    q = st.randn(st.T, Hq, D).to(rows)
    for n_split in (0, 3):
        out = torch.full((batch.T, Hq, D), float("nan"), dtype=rows, device=DEV)
        lse = torch.full((batch.T, Hq), float("nan"), device=DEV)
        out[st.T:], lse[st.T:] = 7, 7
        sg.sgmv_kv_attention(_pad(q, batch.T), batch, st.cache, out=out, lse=lse, n_split=n_split)
        _check_attention(st, q, kv, out, lse, D ** -0.5)
        assert (out[st.T:] == 7).all() and (lse[st.T:] == 7).all()
    k, v = st.randn(st.T, H, D).to(rows), st.randn(st.T, H, D).to(rows)
    bufs, _ = _expected_cache(st, k, v)
    sg.sgmv_kv_write(_pad(k, batch.T), _pad(v, batch.T), batch, st.cache)
    assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])
    back = [torch.full((batch.T, H, D), 7.0, dtype=rows, device=DEV) for _ in range(2)]
    sg.sgmv_kv_read(batch, st.cache, batch.q_start, batch.T, rows, k=back[0], v=back[1])
    for x in back:
        assert (x[st.T:] == 7).all() and (st.T == 0 or not (x[:st.T] == 7).all())


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_padded_step_in_a_graph(sg, fmt):
    """A step captured at its full size and replayed with fewer rows, against the oracle and eager calls."""
    max_q, Hq, H, D = 96, 8, 2, 128
    st = Step(sg, [max_q, max_q], [250, 180], 32, H, D, fmt, seed=5)
    kv = st.fill(sg)
    q = st.randn(st.T, Hq, D).to(BF16).to(DEV)
    out, lse = torch.empty(st.T, Hq, D, dtype=BF16, device=DEV), torch.empty(st.T, Hq, device=DEV)
    size = sg.sgmv_kv_attention_workspace(Hq, BF16, st.batch, st.cache, n_split=3)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)

    def step():
        sg.sgmv_kv_attention(q, st.batch, st.cache, out=out, lse=lse, n_split=3, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.synchronize()
    for new in ([max_q, max_q], [1, max_q], [0, 3], [5, 0], [max_q - 1, 8], [max_q, 1]):
        st.new, st.start = new, [0, new[0], sum(new)]
        st.T = sum(new)
        st.batch.q_start.copy_(_i32(st.start))
        q.copy_(st.randn(2 * max_q, Hq, D).to(BF16).to(DEV))
        got = []
        for run in (graph.replay, step):
            out.fill_(float("nan"))
            lse.fill_(float("nan"))
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            got.append((out[:st.T].clone(), lse[:st.T].clone()))
            assert torch.isnan(out[st.T:]).all() and torch.isnan(lse[st.T:]).all()
        same = torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        assert same, new
        some = {(b, i) for b, n in enumerate(new) for i in range(0, n, 9)} | {(b, n - 1) for b, n in enumerate(new) if n}
        _check_attention(st, q[:st.T].cpu(), kv, *got[0], D ** -0.5, rows=some)


# ---- what the calls touch -------------------------------------------------------------------
def _within(x, lo, hi, value):
    """Nothing but x[lo:hi] has changed from `value`."""
    assert bool((x[:lo] == value).all()) and bool((x[hi:] == value).all())


@pytest.mark.parametrize("fmt", [BF16, I8])
@pytest.mark.parametrize("start,kv_len", [([0, 2, 4], [1 << 30, -5]), ([0, 900, 3], [30, 30]), ([-4, 2, 1 << 30], [30, 0]),
                                          ([3, 1, 0], [30, 30]), ([0, 1, 4], [2 ** 31 - 1, 2]), ([1, 1, 3], [-2 ** 31, 31])])
def test_cut_lengths_and_starts_change_nothing_else(sg, start, kv_len, fmt):
    """q_start cut to [0, T], kv_len to what the table holds: the cache is as after a write of the rows and lengths
    so cut, and nothing around the outputs, the rows read and the workspace is written."""
    T, D = 4, 64
    st = Step(sg, [2, 2], [30, 30], 16, 1, D, fmt)
    st.fill(sg)
    k, v = st.randn(T, 1, D).to(BF16), st.randn(T, 1, D).to(BF16)
    q = st.randn(T, 2, D).to(BF16).to(DEV)
    cut = np.clip(np.array(start, np.int64), 0, T)
    as_cut = copy.copy(st)
    as_cut.start, as_cut.new = cut[:2], [max(int(cut[b + 1] - cut[b]), 0) for b in range(2)]
    as_cut.kv_len = [int(min(max(n, 0), st.table.shape[1] * 16)) for n in kv_len]
    bufs, _ = _expected_cache(as_cut, k, v)
    mine = sorted({int(cut[b]) + i for b in range(2) for i in range(as_cut.new[b])})
    others = [i for i in range(T) if i not in mine]
    for max_q in (4, 100):  # row by row, and by groups; few rows, and tiles
        b = sg.sgmv_kv_batch(_i32(start), _i32(kv_len), st.batch.page_table, T, max_q, 48)
        sg.sgmv_kv_write(k.to(DEV), v.to(DEV), b, st.cache)
        assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])
        for n_split in (1, 3):
            out = torch.full((T + 8, 2, D), 7.0, dtype=BF16, device=DEV)
            lse = torch.full((T + 8, 2), 7.0, device=DEV)
            size = sg.sgmv_kv_attention_workspace(2, BF16, b, st.cache, n_split=n_split)
            ws = torch.full((size + 512,), 0xab, dtype=torch.uint8, device=DEV)
            sg.sgmv_kv_attention(q, b, st.cache, out=out[4:4 + T], lse=lse[4:4 + T], n_split=n_split,
                                 workspace=ws[256:256 + size])
            _within(out, 4, 4 + T, 7)
            _within(lse, 4, 4 + T, 7)
            _within(ws, 256, 256 + size, 0xab)
            assert bool((out[4:4 + T][others] == 7).all()) and bool((lse[4:4 + T][others] == 7).all())
            assert not (out[4:4 + T][mine] == 7).any()
        for rows in (T, T + 40):  # both ways of reading, the second with room to spare
            back = [torch.full((rows + 8, 1, D), 7.0, dtype=BF16, device=DEV) for _ in range(2)]
            sg.sgmv_kv_read(b, st.cache, _i32([min(x, T) for x in start]), rows, k=back[0][4:4 + rows], v=back[1][4:4 + rows])
            for x in back:
                _within(x, 4, 4 + T, 7)
                assert bool((x[4:4 + T][others] == 7).all()) and not (x[4:4 + T][mine] == 7).any()


@pytest.mark.parametrize("fmt,rows", [(I8, BF16), (E4M3, F32), (BF16, BF16), (F32, F32)])
def test_every_row_of_sequences_with_different_counts(sg, fmt, rows):
    """Rows written and read where a sequence's number is not its share of the tokens, row by row and by groups of
    tokens: each is the code times the scale of its own token and head."""
    news = [0] * 30 + [8, 1] + [0] * 5 + [2] * 3 + [0, 7]
    lens = [max(n, (11 * i) % 50) for i, n in enumerate(news)]
    st = Step(sg, news, lens, 16, 2, 64, fmt, seed=6, rows=rows)
    k, v = st.randn(st.T, 2, 64).to(rows), st.randn(st.T, 2, 64).to(rows)
    bufs, scales = _expected_cache(st, k, v)
    sg.sgmv_kv_write(k.to(DEV), v.to(DEV), st.batch, st.cache)
    assert _same(_raw(st.cache.k), bufs[0]) and _same(_raw(st.cache.v), bufs[1])
    lay = ko.Cache(16, 64, st.cache.k.element_size())
    ref = [torch.empty(st.T, 2, 64, dtype=rows) for _ in range(2)]
    for which, index in ((0, lay.k_index), (1, lay.v_index)):
        for b, n in enumerate(news):
            for i in range(n):
                pos = lens[b] - n + i
                page, off = st.table[b, pos // 16], pos % 16
                x = bufs[which][page][:, torch.from_numpy(index(off))].contiguous()
                if fmt in (I8, E4M3):
                    x = x.view(fmt).float() * scales[which][page, :, off][:, None]
                ref[which][int(st.start[b]) + i] = x.to(rows)
    got = sg.sgmv_kv_read(st.batch, st.cache, st.batch.q_start, st.T, rows)
    pad = np.concatenate([[0], np.cumsum([n + 20 if n else 0 for n in news])])
    more = sg.sgmv_kv_read(st.batch, st.cache, _i32(pad.tolist()), int(pad[-1]), rows)
    for which in range(2):
        assert _same(got[which], ref[which])
        for b, n in enumerate(news):
            assert _same(more[which][int(pad[b + 1]) - n:int(pad[b + 1])].contiguous(), ref[which][int(st.start[b]):int(st.start[b + 1])].contiguous())


def test_more_rows_than_one_launch_by_rows_takes(sg):
    """65536 sequences' 8 tokens, 128 heads: 2^26 rows, of which a launch row by row would take 2^32 work items and
    more. (17 GB of device memory.)"""
    B, n, H, D = 65535, 8, 128, 16
    cache = sg.sgmv_kv_init(B, 16, H, D, BF16, DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    k = torch.randn(B * n, H, D, generator=g, device=DEV, dtype=BF16)
    v = torch.randn(B * n, H, D, generator=g, device=DEV, dtype=BF16)
    start = torch.arange(B + 1, dtype=torch.int32, device=DEV) * n
    table = torch.randperm(B, generator=g, device=DEV).to(torch.int32).view(B, 1)
    batch = sg.sgmv_kv_batch(start, torch.full((B,), n + 3, dtype=torch.int32, device=DEV), table, B * n, n, n + 3)
    sg.sgmv_kv_write(k, v, batch, cache)
    back = sg.sgmv_kv_read(batch, cache, start, B * n)
    assert torch.equal(back[0], k) and torch.equal(back[1], v)


# ---- windows ------------------------------------------------------------------------------
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 30])
@pytest.mark.parametrize("new,kv_len", [([5, 3, 2], [2, 0, 30]), ([100, 9], [60, 4])])
@pytest.mark.parametrize("fmt,rows", [(BF16, BF16), (E4M3, BF16), (F32, F32)])
def test_wide_windows_with_rows_before_the_first_token(sg, new, kv_len, window, fmt, rows):
    """A window wider than any sequence is none, also where a tile's first rows stand at negative positions: their
    position less the window is below -2^31."""
    st = Step(sg, new, kv_len, 16, 2, 128, fmt, seed=7, rows=rows)
    kv = st.fill(sg)
    q = st.randn(st.T, 8, 128).to(rows)
    for n_split in (0, 2):
        out, lse = sg.sgmv_kv_attention(q.to(DEV), st.batch, st.cache, window=window, n_split=n_split)
        _check_attention(st, q, kv, out, lse, 128 ** -0.5, window)


# ---- codes of NaN ---------------------------------------------------------------------------
NAN_CODES = {
    # name: new tokens, length, query heads, key/value heads, D, rows, window
    "decode": ([1, 1], [100, 70], 8, 2, 128, BF16, 0),
    "decode_window": ([1, 2], [400, 170], 4, 2, 80, BF16, 60),
    "drafts": ([3, 5], [150, 70], 8, 2, 128, BF16, 0),
    "drafts_odd_dim": ([6, 2], [90, 64], 4, 2, 48, BF16, 0),
    "drafts_256": ([6, 2], [90, 64], 4, 2, 256, BF16, 0),
    "chunk": ([90, 1], [150, 80], 8, 2, 128, BF16, 0),
    "chunk_window": ([90, 40], [300, 70], 8, 2, 80, BF16, 50),
    "chunk_64": ([200], [500], 4, 2, 64, BF16, 0),
    "chunk_256": ([70, 70], [150, 130], 4, 2, 256, BF16, 0),
    "chunk_112": ([70], [150], 4, 2, 112, BF16, 0),
    "fp32": ([40, 3], [100, 70], 4, 2, 128, F32, 0),
    "fp32_48": ([40, 3], [100, 70], 4, 2, 48, F32, 30),
}


@pytest.mark.parametrize("n_split", [0, 2])
@pytest.mark.parametrize("name", sorted(NAN_CODES))
def test_nan_codes_reach_the_rows_that_see_them(sg, name, n_split):
    """Codes of NaN (0x7f, 0xff) in a wrapped e4m3 cache: in V, their value of d is NaN in the rows that see the
    token; in K, the rows that see the token are NaN. All else is as without them."""
    new, kv_len, Hq, H, D, rows, window = NAN_CODES[name]
    st = Step(sg, new, kv_len, 16, H, D, E4M3, seed=9, rows=rows)
    st.fill(sg)
    c = st.cache
    cache = sg.sgmv_kv_wrap(c.k, c.v, c.k_scale, c.v_scale)
    q = st.randn(st.T, Hq, D).to(rows).to(DEV)
    lay, G = ko.Cache(16, D, 1), Hq // H
    run = lambda: sg.sgmv_kv_attention(q, st.batch, cache, window=window, n_split=n_split)
    clean, clean_lse = run()
    assert torch.isfinite(clean).all()

    def at(b, pos, h, d, which):
        """Where the code of (sequence, position, head, d) is held, in a flat view of K or V."""
        index = (lay.k_index if which == "k" else lay.v_index)(pos % 16)[d]
        return (int(st.table[b, pos // 16]) * H + h) * 16 * D + int(index)

    def spoil(which, places):
        flat = _raw(getattr(c, which)).view(-1)
        where = torch.tensor([at(*p, which) for p in places], device=DEV)
        kept = flat[where].clone()
        flat[where] = torch.tensor([0x7f, 0xff], dtype=torch.uint8, device=DEV)[torch.arange(len(places), device=DEV) % 2]
        got = run()
        flat[where] = kept
        return got

    for b in range(len(new)):
        first = kv_len[b] - new[b]
        lo = max(first - window + 1, 0) if window else 0
        for pos in sorted({lo, (lo + first) // 2, first, first + new[b] // 2, kv_len[b] - 1}):
            places = [(b, pos, 0, D - 1), (b, pos, H - 1, 3)]
            out, lse = spoil("v", places)
            bad = torch.zeros_like(clean, dtype=torch.bool)
            seen = torch.zeros(st.T, dtype=torch.bool, device=DEV)
            for i in range(new[b]):
                here = first + i
                seen[int(st.start[b]) + i] = pos <= here and not (window and pos <= here - window)
            for _, _, h, d in places:
                bad[seen, h * G:(h + 1) * G, d] = True
            assert torch.isnan(out[bad]).all(), (b, pos)
            assert bool((out[~bad] == clean[~bad]).all()) and torch.equal(lse, clean_lse), (b, pos)
            out, lse = spoil("k", places[:1])
            bad[:] = False
            bad[seen, :G] = True
            assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad[:, :, 0]]).all(), (b, pos)
            assert bool((out[~bad] == clean[~bad]).all()) and bool((lse[~bad[:, :, 0]] == clean_lse[~bad[:, :, 0]]).all())


@pytest.mark.parametrize("n_split", [0, 2])
@pytest.mark.parametrize("fmt", [E4M3, I8])
@pytest.mark.parametrize("new,rows,D", [(1, BF16, 128), (4, BF16, 64), (5, F32, 80), (5, BF16, 48), (90, BF16, 128)])
def test_nan_rows_of_no_weight_reach_the_rows_that_see_them(sg, new, rows, D, fmt, n_split):
    """A V row of NaN whose token's probability is below the smallest fp32 number: the rows that see it are NaN
    all the same, wherever in the sequence the token stands."""
    n = 150
    st = Step(sg, [new], [n], 16, 1, D, fmt, seed=12, rows=rows)
    k, v = st.randn(n, 1, D) * 0.1, st.randn(n, 1, D)
    whole = sg.sgmv_kv_batch(_i32([0, n]), _i32([n]), st.batch.page_table, n, n, n)
    q = (st.randn(new, 2, D).abs() + 0.5).to(rows)
    for pos in sorted({0, 63, 64, 70, 127, 128, n - new, n - new // 2 - 1, n - 1}):
        low = k.clone()
        low[pos] = -400.0  # scores below -200 sqrt(D), next to at most 0.1 * 128
        got = []
        for x in (0.0, float("nan")):
            spoilt = v.clone()
            spoilt[pos, 0, 5] = x
            sg.sgmv_kv_write(low.to(rows).to(DEV), spoilt.to(rows).to(DEV), whole, st.cache)
            got.append(sg.sgmv_kv_attention(q.to(DEV), st.batch, st.cache, n_split=n_split))
        (ref, ref_lse), (out, lse) = got
        seen = max(pos - (n - new), 0)  # the first row that sees it
        assert torch.isfinite(ref).all() and torch.equal(lse, ref_lse), pos
        assert torch.equal(out[:seen], ref[:seen]) and torch.isnan(out[seen:]).all(), pos


# ---- drafts -------------------------------------------------------------------------------
@pytest.mark.parametrize("V", [16 * 1024, 30 * 1024 + 5, 128 * 1024])
def test_draws_between_parts_without_weight(sg, V):
    """Parts of a row without a weight, where sums of the parts before them in different orders differ in their
    last bit and the number falls in between: 2^-53 + 2^-53 + 1 is 1 or 1 + 2^-52. The token has a weight, and the
    number falls on it to the rounding of such sums (V additions of at most 2^-53 of the total, on either side)."""
    per = 2048 if V > 64 * 1024 else 1024  # entries of a lane's parts
    rows = []
    for a in range(3, 12):
        for ones in ((2, a), (2,), (0, 5, a)):
            w = torch.zeros(V)
            w[0], w[per] = 2.0 ** -53, 2.0 ** -53
            for i in ones:
                w[i * per + a] = 1.0
            rows.append(w)
    us = [0.0, 2.0 ** -24, 0.25, 0.5, 0.75, 1 - 2.0 ** -24]
    t = torch.stack([w for w in rows for _ in us])
    su = torch.tensor(us * len(rows))
    none, B = torch.empty(0, dtype=torch.int32, device=DEV), t.shape[0]
    tokens, _ = sg.sgmv_verify_drafts(t.to(DEV), None, none, _i32([0] * (B + 1)), torch.empty(0, device=DEV),
                                      su.to(DEV), 0)
    tokens = tokens[:, 0].cpu().tolist()
    for b in range(B):
        w = t[b].double().numpy()
        at = np.flatnonzero(w)
        c = np.cumsum(w[at])
        tol = V * 2.0 ** -53 * c[-1]
        assert tokens[b] in at, (b, tokens[b])
        i = int(np.searchsorted(at, tokens[b]))
        x = float(su[b]) * c[-1]
        assert (c[i - 1] if i else 0.0) - tol <= x < c[i] + tol, (b, tokens[b])


def test_numbers_outside_the_unit_interval_draw_nothing(sg):
    t = torch.full((5, 3000), 1.0 / 3000, device=DEV)
    su = torch.tensor([-0.25, 1.0, float("nan"), float("inf"), 0.5], device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    tokens, accepted = sg.sgmv_verify_drafts(t, None, none, _i32([0] * 6), torch.empty(0, device=DEV), su, 0)
    assert tokens[:4, 0].tolist() == [-1] * 4 and tokens[4, 0].item() == 1500 and accepted.tolist() == [0] * 5
