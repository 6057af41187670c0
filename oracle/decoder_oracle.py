"""Plain CPU oracle for what stands between a decoder's linears: the residual
addition with the RMS norm, rotary positions, the 8-bit key/value cache,
attention over it, and sampling.

TEST INFRASTRUCTURE ONLY, like qlin_oracle: nothing in the product path imports
it, and it shares no code with the CUDA library.

Sums and functions are float64.  Where the definition itself rounds (the
rotation's float32 operations, the cache's scales and codes), the same float32
operations are done one by one with numpy, so that codes can be compared bit
for bit.
"""

from __future__ import annotations

import math

import numpy as np

BLOCK = 64


def add_rms_norm(x, weight, residual, eps):
    """(y, h) in float64, unrounded."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    rms = np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return h / rms * np.asarray(weight, np.float64), h


def rope_frequencies(rot_dim, base, factor=1.0, short=0.0, long=0.0):
    """The angle of one position, for every pair."""
    out = []
    for i in range(rot_dim // 2):
        f = base ** (-2.0 * i / rot_dim)
        wave = 2.0 * math.pi / f
        if factor > 1.0 and wave > short:
            keep = 0.0
            if short > 0.0 and wave < long:
                keep = (1.0 / wave - 1.0 / long) / (1.0 / short - 1.0 / long)
            f = keep * f + (1.0 - keep) * f / factor
        out.append(f)
    return np.array(out)


def rotate(x, cos_sin, interleaved):
    """x [T, heads, D] float32, cos_sin [T, pairs, 2] float32: the rotated x in
    float32, one rounding to float32 for each operation."""
    x = np.array(x, np.float32)
    half = cos_sin.shape[1]
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = x[..., first].copy(), x[..., second].copy()
    c, s = cos_sin[:, None, :, 0], cos_sin[:, None, :, 1]
    x[..., first] = a * c - b * s
    x[..., second] = b * c + a * s
    return x


def quantise_block(block):
    """(codes uint8, scale) of one block of float32 values."""
    scale = np.float32(np.abs(block).max()) / np.float32(127)
    if scale == 0:
        return np.full(block.shape, 128, np.uint8), scale
    return (np.rint(block / scale) + 128).astype(np.uint8), scale


def attention(q, keys, values, position, scale):
    """One row: q [D] over keys, values [n, D] up to `position`, all float64.
    Returns (out, sum_j p_j |v_j|, sum of exp(score - max), the largest
    sum_d |q_d k_d| * scale)."""
    n = position + 1
    if n <= 0:
        return np.zeros(q.shape), np.zeros(q.shape), 0.0, 0.0
    score = keys[:n] @ q * scale
    e = np.exp(score - score.max())
    p = e / e.sum()
    size = (np.abs(keys[:n]) @ np.abs(q)).max() * scale
    return p @ values[:n], p @ np.abs(values[:n]), e.sum(), size


def sample_distribution(logits, temperature, top_k, top_p, min_p):
    """The kept tokens' probabilities in index order, float64 [V] (0: not kept);
    None for a row without a token."""
    x = np.array(logits, np.float64)
    x[np.isnan(x)] = -np.inf
    top = x.max()
    if top == -np.inf:
        return None
    order = np.argsort(-x, kind="stable")
    if temperature <= 0:
        p = np.zeros(x.size)
        p[order[0]] = 1.0
        return p
    with np.errstate(invalid="ignore"):
        e = np.where(x == top, 1.0, np.exp((x - top) / temperature))
    kept = order[:top_k] if top_k > 0 else order
    if top_p < 1:
        share = e[kept] / e[kept].sum()
        keep = np.cumsum(share) - share < top_p
        keep[0] = True
        kept = kept[keep]
    ok = e[kept] >= min_p
    ok[0] = True
    kept = kept[ok]
    p = np.zeros(x.size)
    p[kept] = e[kept] / e[kept].sum()
    return p
