"""CPU oracle for the norm, the base product of 4-bit weights and the rotated append.

TEST INFRASTRUCTURE ONLY, like ``sgmv_oracle``: it shares no code with the library. Inputs come in as numpy
arrays (bf16 values as their exact fp32 copies); every floating step runs in fp64 but those whose fp32 rounding the
definitions name.

Definitions (include/sgmv.h states the same ones):
  * norm: h = fp32(x + residual), g = fp32(h weight), root = sqrt(mean h^2 + eps), out = g / root; codes of g as
    kv_oracle.quantise has them, their scale over the root;
  * base weight: scale (code - zero), or 2^(scale - 127) e2m1(code), `group` values of k to a scale;
  * rotation: (a, b) -> (a c - b s, b c + a s) of the first 2 * len(c) values, every product and sum rounded to fp32.
"""
from __future__ import annotations

import numpy as np

from .kv_oracle import quantise

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def rms_norm(x, weight, eps, residual=None, fmt=None):
    """(out, h, codes, scale) of rows x [..., W] (fp32 values), fp64."""
    with np.errstate(over="ignore", invalid="ignore"):
        h = np.asarray(x, np.float32)
        if residual is not None:
            h = h + np.asarray(residual, np.float32)
        g = h * np.asarray(weight, np.float32)
        root = np.sqrt((h.astype(np.float64) ** 2).mean(-1, keepdims=True) + eps)
        out = g.astype(np.float64) / root
        codes = scale = None
        if fmt is not None:
            codes, scale = quantise(g, fmt)
            scale = scale / root[..., 0]
    return out, h.astype(np.float64), codes, scale


def unpack(codes, K):
    """Codes [N, K] of rows of bytes, the even k in the low four bits."""
    codes = np.asarray(codes)
    return np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)[:, :K]


def base_weight(codes, K, scale, zero, group, fmt):
    """Values [N, K] of a packed weight, and their sizes as the sums meet them (|code| and zero apart)."""
    c = unpack(codes, K).astype(np.int64)
    at = np.arange(K) // group
    if fmt == "e2m1":
        v = np.where(c & 8, -1, 1) * E2M1[c & 7] * 2.0 ** (np.asarray(scale, np.float64)[:, at] - 127)
        return v, abs(v)
    z = np.full(scale.shape, 8) if zero is None else np.asarray(zero, np.int64)
    s = np.asarray(scale, np.float64)[:, at]
    return s * (c - z[:, at]), abs(s) * (c + z[:, at])


def rotate(x, c, s, interleaved):
    """Rows x [T, H, D] (fp32 values) turned by angles with cosines c and sines s [T, rotary / 2], fp32 step by step."""
    y = np.array(x, np.float32)
    half = c.shape[-1]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    c, s = (np.asarray(v, np.float32)[:, None, :] for v in (c, s))
    lo, hi = y[..., a].copy(), y[..., b].copy()
    y[..., a] = lo * c - hi * s
    y[..., b] = hi * c + lo * s
    return y


__all__ = ["rms_norm", "unpack", "base_weight", "rotate", "E2M1"]
