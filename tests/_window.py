"""The windowed attention's definition in fp64 over the oracle's dequantised
cache, with a bound on the GPU path's error, shared by the window tests.

The bound follows the GPU path's roundings. With A = scale * sum |q~_i y_i| ||k||
(the mass of a logit) and dy_i the error of the level that the path multiplies
with, a logit is off by at most d = 140 * 2^-24 A + scale * sum |q~_i dy_i| ||k||
(128 fp32 multiply-adds and the rotation's seven stages); a softmax weight is
then off by a factor of at most exp(2 d). P.V adds the relative error e_v of
V's levels, the fp32 sums over n tokens (n + 64) 2^-24, the weights' and the
exponential's 2^-20 in all, and (chunks) the fp16 halves' smallest step 2^-25
per token times the largest level. fp32 outputs of a decode step carry V's
levels in two fp16 parts, so e_v is 2^-22 there (the second part's rounding).
bf16 outputs of a chunk carry the weights as single fp16 values, each rounded
by at most 2^-11 of itself (or the half step 2^-25 counted above). Rotations keep the 2-norm, so each output
coordinate is off by at most the sum of these times the largest visible ||v||.
"""
from __future__ import annotations

import math

import numpy as np

from oracle import oracle as o


def level_errors(stream, frequency_weighted):
    """|fp16(kappa y) / kappa - y| per level for the scale that the library
    chooses: the least frequency-weighted absolute error (keys of a chunk) or
    the least relative one (values)."""
    y = stream.yf.astype(np.float64)
    f = np.asarray(stream.freq, np.float64)
    kappa = 1.0 + np.arange(65536) / 65536.0
    h = (kappa[:, None] * y).astype(np.float32).astype(np.float16).astype(np.float64) / kappa[:, None]
    err = np.abs(h - y)
    j = np.argmin((f * err).sum(1) if frequency_weighted else (err / np.abs(y)).max(1))
    return err[j]


def attention(tab, q, kcont, vcont, start, window, sinks, chunk, sm_scale=None, half_levels=True,
              half_weights=False):
    """q [B, n, Hq, 128]; flat containers [B, Hkv, T_cap, C]; query i of
    sequence b at position start[b] + i (a position outside the cache gives 0).
    Returns (out, bound) with bound [B, n, Hq, 1]."""
    q = np.asarray(q, np.float64)
    B, n, Hq, _ = q.shape
    Hkv, T_cap = kcont.shape[1], kcont.shape[2]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(128.0) if sm_scale is None else sm_scale
    dk = level_errors(tab.k, True) if chunk else np.zeros(len(tab.k.yf))
    ev = float((level_errors(tab.v, False) / np.abs(tab.v.yf.astype(np.float64))).max())
    if not half_levels:
        ev = 2.0 ** -22
    H = o.hadamard(128)
    out, bound = np.zeros((B, n, Hq, 128)), np.zeros((B, n, Hq, 1))
    for b in range(B):
        pos = int(start[b]) + np.arange(n)
        rows = np.nonzero((pos >= 0) & (pos < T_cap))[0]
        if not rows.size:
            continue
        t = np.arange(int(pos[rows].max()) + 1)
        seen = (t <= pos[rows, None]) & ((t > pos[rows, None] - window) | (t < sinks))
        used = np.nonzero(seen.any(0))[0]
        seen = seen[:, used]
        for h in range(Hkv):
            ks, kn, kst = o.decode_containers(tab.k, kcont[b, h, used])
            vs, vn, vst = o.decode_containers(tab.v, vcont[b, h, used])
            assert not kst.any() and not vst.any(), "corrupt container in oracle input"
            kh = o.dequantize(tab.k, ks, kn, tab.signs[h])
            vh = o.dequantize(tab.v, vs, vn, tab.signs[h])
            nk, nv = o.f16_to_f64(kn), o.f16_to_f64(vn)
            ya, yd = np.abs(tab.k.yf.astype(np.float64)[ks]), dk[ks]
            for g in range(G):
                qr = q[b, rows, h * G + g]
                a = np.where(seen, scale * (qr @ kh.T), -np.inf)
                qt = np.abs((qr * tab.signs[h]) @ H) / 128.0
                d = scale * nk * (140 * 2.0 ** -24 * (qt @ ya.T) + qt @ yd.T)
                d = np.where(seen, d, 0.0).max(1)
                p = np.exp(a - a.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                out[b, rows, h * G + g] = p @ vh
                big = np.where(seen, nv, 0.0).max(1)
                m = seen.sum(1)
                bound[b, rows, h * G + g, 0] = big * (np.expm1(2 * d) + ev + (m + 64) * 2.0 ** -24 + 2.0 ** -20)
                if half_weights:
                    bound[b, rows, h * G + g, 0] += 2.0 ** -11 * big
                if chunk:
                    bound[b, rows, h * G + g, 0] += 2.0 ** -25 * m * np.abs(tab.v.yf).max()
    return out, bound


def assert_within(got, ref, bound, half_out, what):
    """Each output within its bound, plus half a step of a bf16 output."""
    tol = bound + (2.0 ** -8 * (np.abs(ref) + bound) if half_out else 2.0 ** -24 * np.abs(ref))
    over = np.abs(got - ref) - tol
    assert np.all(np.isfinite(got)), what
    assert np.max(over, initial=-1.0) <= 0.0, "%s: %.3e over its bound at %s" % (
        what, over.max(), np.unravel_index(np.argmax(over), over.shape))
