"""fp64 CPU oracle for the paged key/value cache, its attention and the draft check.

TEST INFRASTRUCTURE ONLY, like ``sgmv_oracle``: it shares no code with the library. Inputs
come in as numpy arrays (bf16 values as their exact fp32 copies); every floating step runs
in fp64, token by token and row by row.

Definitions (include/sgmv.h states the same ones):
  * group g of 16 tokens of a (page, head) block: K[t][d] at ((g (D/c) + d/c) 16 + t%16) c + d%c
    with c = 16 bytes of elements; V[t][d] at (g D + d) 16 + place(t%16);
  * a row is quantised with amax = max |x|, scale = amax / F, code = x F / amax rounded to the
    format, ties to even; zeros give scale 0, a non-finite value scale NaN and codes 0;
  * token i of sequence b stands at kv_len - n + i and sees t <= pos (and > pos - window) on
    pages that exist; a row that sees nothing has output 0 and lse -inf;
  * drafts are taken while u q(d) < p(d); the next token is the lowest j whose running sum of
    max(p - q, 0) (or p) passes r times the total.
"""
from __future__ import annotations

import numpy as np

TOP = {"e4m3": 448.0, "i8": 127.0}


def e4m3_value(code):
    """Value of an e4m3 code: 1 sign, 4 exponent (bias 7), 3 mantissa bits, 0x7f NaN."""
    code = np.asarray(code, np.int64)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((code & 127) == 127, np.nan, v)
    return np.where(code & 128, -v, v)


_E4M3 = e4m3_value(np.arange(127))
_EDGES = (_E4M3[1:] + _E4M3[:-1]) / 2


def e4m3_code(y):
    """Code of the e4m3 value nearest to each y (|y| <= 448), ties to the even code; the sign of
    a zero is that of y."""
    y = np.asarray(y, np.float64)
    lo, hi = np.searchsorted(_EDGES, abs(y), "left"), np.searchsorted(_EDGES, abs(y), "right")
    at = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))
    return (at | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def quantise(x, fmt):
    """Codes (uint8 bytes for e4m3, int8) and scales of rows x [..., D]."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x).all(-1)
    amax = np.where(bad, 0.0, np.nanmax(np.where(np.isfinite(x), abs(x), 0), -1))
    top = TOP[fmt]
    y = np.where(np.isfinite(x), x, 0) * top / np.where(amax == 0, 1.0, amax)[..., None]
    y = np.where((amax == 0)[..., None], 0.0, y)
    code = e4m3_code(y) if fmt == "e4m3" else np.rint(y).astype(np.int8)
    return code, np.where(bad, np.nan, amax / top)


def place(r):
    """Place of token r (0..15) of a group in V."""
    return 8 * (r // 4 % 2) + 4 * (r // 8) + r % 4


class Cache:
    """A cache held token by token: {(page, head, offset): (k row, v row)}, and its layout."""

    def __init__(self, page_size, head_dim, elem):
        self.ps, self.D, self.c = page_size, head_dim, 16 // elem

    def k_index(self, t):
        """Flat index in a (page, head) block of K[t][0..D)."""
        d, g, r = np.arange(self.D), t // 16, t % 16
        return ((g * (self.D // self.c) + d // self.c) * 16 + r) * self.c + d % self.c

    def v_index(self, t):
        d, g = np.arange(self.D), t // 16
        return (g * self.D + d) * 16 + place(t % 16)


def visible(kv_len, n, i, window, page_ok, page_size):
    """Positions that new token i of a sequence of kv_len tokens, n of them new, sees."""
    pos = kv_len - n + i
    t = np.arange(0, max(pos + 1, 0))
    if window:
        t = t[t > pos - window]
    return t[[bool(page_ok[x // page_size]) for x in t]] if len(t) else t


def attention_row(q, k, v, scale):
    """(out, lse, bound terms) of one query over rows k, v [n, D]: also sum p |v| / sum p and the
    largest |q| . |k| scale, by which rounding errors are measured."""
    D = q.shape[0]
    if k.shape[0] == 0:
        return np.zeros(D), -np.inf, np.zeros(D), 0.0
    s = (k @ q) * scale
    m = s.max()
    p = np.exp(s - m)
    total = p.sum()
    return (p @ v / total, m + np.log(total), p @ abs(v) / total,
            float((abs(k) @ abs(q)).max() * scale))


def verify(target, draft, ids, u, r):
    """(tokens, accepted) of one sequence: target [n + 1, V], draft [n, V] or None."""
    clean = lambda x: np.where(np.isfinite(x) & (np.asarray(x) > 0), x, 0).astype(np.float64)
    V = target.shape[1]
    n = len(ids)
    taken = n
    for i in range(n):
        ok = 0 <= ids[i] < V
        if ok:
            q = 1.0 if draft is None else clean(draft[i])[ids[i]]
            ok = float(u[i]) * q < clean(target[i])[ids[i]]
        if not ok:
            taken = i
            break
    p = clean(target[taken])
    w = p.copy()
    if taken < n:
        if draft is None:
            if 0 <= ids[taken] < V:
                w[ids[taken]] = 0
        else:
            w = np.maximum(p - clean(draft[taken]), 0)
    if not w.sum() > 0:
        w = p
    c = np.cumsum(w)
    token = -1 if not c[-1] > 0 else int(np.searchsorted(c, float(r) * c[-1], "right"))
    return list(ids[:taken]) + [token], taken


__all__ = ["TOP", "e4m3_value", "e4m3_code", "quantise", "place", "Cache", "visible",
           "attention_row", "verify"]
