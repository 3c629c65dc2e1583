"""The steps around the expert layers: norm, 8-bit linear, key/value cache and decode attention.
Test infrastructure only: plain loops and float64, from the definitions in include/w4a16.h.

The pages give no blocks between the expert layers, so these follow the usual definitions
(root-mean-square norm, symmetric quantisation with a scale per group, softmax attention) on this
library's formats: groups of 32, bf16 scales, layout L1 nibbles.
"""
from __future__ import annotations

import numpy as np

from . import bf16, q4

TOP = {"int8": 127, "int4": 7}


# ------------------------------------------------------------------------------------ norm
def rms_add(x_bits, residual_bits, weight_bits, eps):
    """-> (h bits, y float64): h = bf16(x + residual), y = h * w / sqrt(mean h^2 + eps)."""
    h = bf16.to_f64(x_bits)
    h_bits = np.asarray(x_bits, dtype=np.uint16)
    if residual_bits is not None:
        h_bits = bf16.from_f64(h + bf16.to_f64(residual_bits))
        h = bf16.to_f64(h_bits)
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    if weight_bits is not None:
        y = y * bf16.to_f64(weight_bits)
    return h_bits, y


# ---------------------------------------------------------------------------- 8-bit linear
def w4a8_linear(xq, xs, codes, scales):
    """y[m, n] = xs[m] * sum_k xq[m, k] W[n, k], float64 unrounded; W = s q."""
    return (np.asarray(xq, np.float64) * np.asarray(xs, np.float64)[:, None]) @ q4.dequant(codes, scales).T


def w4a8_magnitude(xq, xs, codes, scales):
    """sum over groups of |group sum| * |s| * |xs|: what float32 accumulation errors scale with."""
    M, K = xq.shape
    N = codes.shape[0]
    one = np.full((N, K // 32), 0x3F80, np.uint16)
    q = q4.dequant(codes, one).reshape(N, K // 32, 32)
    x = np.asarray(xq, np.float64).reshape(M, K // 32, 32)
    s = np.abs(bf16.to_f64(scales))
    out = np.zeros((M, N))
    for g in range(K // 32):
        out += np.abs(x[:, g] @ q[:, g].T) * s[:, g]
    return out * np.abs(np.asarray(xs, np.float64))[:, None]


# ----------------------------------------------------------------------------------- cache
def quantise_rows(x_bits, kind):
    """bf16 rows [R, D] -> (codes int [R, D], scale bits [R, D/32]); group by group."""
    x = bf16.to_f64(x_bits)
    R, D = x.shape
    top = TOP[kind]
    q = np.zeros((R, D), np.int64)
    s = np.zeros((R, D // 32), np.uint16)
    for r in range(R):
        for g in range(D // 32):
            v = x[r, 32 * g:32 * g + 32]
            if not np.isfinite(v).all():
                s[r, g] = bf16.QNAN_BITS
                continue
            sb = bf16.from_f64(np.array(np.abs(v).max() / top))
            s[r, g] = sb
            step = float(bf16.to_f64(sb))
            if step > 0:
                q[r, 32 * g:32 * g + 32] = np.clip(np.rint(v / step), -top, top)
    return q, s


def pack_l1(q):
    """codes -8..7 [R, D] -> uint32 words [R, D/8], nibble j of word w = q + 8 of element 8w + j."""
    R, D = q.shape
    w = np.zeros((R, D // 8), np.uint64)
    for j in range(8):
        w |= (q[:, j::8] + 8).astype(np.uint64) << np.uint64(4 * j)
    return w.astype(np.uint32)


def row_values(q, s):
    """codes [R, D], scale bits [R, D/32] -> float64 rows."""
    return q.astype(np.float64) * np.repeat(bf16.to_f64(s), 32, axis=1)


# ------------------------------------------------------------------------------- attention
def attend(q, k, v, scale, softcap=0.0, window=0):
    """One query row over one sequence's tokens: q [D], k, v [L, D] float64
    -> (out [D], lse, magnitude sum p |v|, largest sum |q k|, sum |v|)."""
    L = k.shape[0]
    if window:
        k, v = k[max(0, L - window):], v[max(0, L - window):]
    if k.shape[0] == 0:
        return np.zeros(q.shape[0]), -np.inf, np.zeros(q.shape[0]), 0.0, np.zeros(q.shape[0])
    z = (k @ q) * scale
    if softcap:
        z = softcap * np.tanh(z / softcap)
    top = z.max()
    e = np.exp(z - top)
    p = e / e.sum()
    return p @ v, top + np.log(e.sum()), p @ np.abs(v), float((np.abs(k) @ np.abs(q)).max()), np.abs(v).sum(axis=0)
