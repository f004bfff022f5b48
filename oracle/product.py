"""MXFP4 quantizer, products of packed 4-bit matrices and a mixture-of-experts
layer, in float64 numpy.  Test infrastructure only.

* MXFP4 quantizer: the ModelOpt MXFP4->NVFP4 guide §1 gives the format (E2M1
  elements, one E8M0 power of two per 32); the scale rule is that of the OCP
  Microscaling specification v1.0 §6.3: the exponent of the block max less 2
  (the exponent of E2M1's 6), held in the E8M0 range.  Readings: an all-zero
  block has code 0, a block with an infinity or NaN code 255 and zero nibbles.
* Products: y = x w^T of the formats' exact values ("Coder390 NVFP4
  校正（校准）方式" §3, the W4A16 and W4A4 tiers); no rounding here.
* Layer: sum over a token's experts of weight * W2 (silu(W1 x) * (W3 x)).
These are readings: no worked example on the pages confirms them.
"""
from __future__ import annotations

import math

import numpy as np

from .formats import E4M3_VALUES, bf16_bits_to_f64, e2m1_decode, e2m1_encode, pack_nibbles, unpack_nibbles


def mxfp4_quantize(x_bits):
    """(packed [rows, k/2], e8m0 [rows, k/32]) of bf16 patterns [rows, k]."""
    bits = np.asarray(x_bits, dtype=np.uint16)
    rows, k = bits.shape
    x = bf16_bits_to_f64(bits).reshape(rows, k // 32, 32)
    finite = np.isfinite(x).all(axis=2)
    xf = np.where(finite[..., None], x, 0.0)
    amax = np.abs(xf).max(axis=2)
    _, e = np.frexp(amax)                              # amax = m 2^e, 0.5 <= m < 1
    code = np.where(amax > 0, np.maximum(e - 1 - 2 + 127, 0), 0)
    nib = e2m1_encode(xf, np.exp2(code - 127.0)[..., None])
    nib = np.where(finite[..., None], nib, 0)
    code = np.where(finite, code, 255).astype(np.uint8)
    return pack_nibbles(nib.reshape(rows, k)), code


def nvfp4_values(packed, codes, s2=1.0):
    """Exact values e2m1 * e4m3(code) * scale_2 (scale_2 per leading index
    when an array)."""
    nib = unpack_nibbles(packed)
    v = e2m1_decode(nib).reshape(codes.shape + (16,)) * E4M3_VALUES[np.asarray(codes).astype(np.int64)][..., None]
    s2 = np.asarray(s2, dtype=np.float64)
    return v.reshape(nib.shape) * s2.reshape(s2.shape + (1,) * (nib.ndim - s2.ndim))


def matmul(x, w):
    """x w^T and the sum of the products' magnitudes (for error bounds)."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def moe_route(logits, top_k, normalize=True):
    """(ids, weights): largest logits first, lower expert first among equals;
    -inf and NaN never; +inf as the largest float32."""
    big = float(np.finfo(np.float32).max)
    ids = np.full((len(logits), top_k), -1, dtype=np.int32)
    wts = np.zeros((len(logits), top_k))
    for t, row in enumerate(np.asarray(logits, dtype=np.float64)):
        cand = sorted((-min(v, big), e) for e, v in enumerate(row) if v > -math.inf)
        if not cand:
            continue
        p = np.exp(np.array([-c[0] for c in cand]) + cand[0][0])
        n = min(top_k, len(cand))
        ids[t, :n] = [c[1] for c in cand[:n]]
        wts[t, :n] = p[:n] / (p[:n].sum() if normalize else p.sum())
    return ids, wts


def silu(a):
    return a / (1.0 + np.exp(-a))


def moe_forward(x, ids, weights, w13, w2):
    """y [tokens, hidden] and a magnitude bound of its sums; x float64, w13
    [experts, 2, inter, hidden] and w2 [experts, hidden, inter] exact values."""
    y, mag = np.zeros_like(x), np.zeros_like(x)
    for t in range(ids.shape[0]):
        for s in range(ids.shape[1]):
            e = int(ids[t, s])
            if 0 <= e < w13.shape[0]:
                h = silu(w13[e, 0] @ x[t]) * (w13[e, 1] @ x[t])
                y[t] += weights[t, s] * (w2[e] @ h)
                mag[t] += abs(weights[t, s]) * (np.abs(w2[e]) @ np.abs(h))
    return y, mag
