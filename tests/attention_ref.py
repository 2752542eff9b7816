"""Attention, norms with rotation and eviction in 64 bits, plainly, with how far
the sums and roundings of a call may be off."""
import numpy as np

from block_ref import HALF_ULP, SUM_ULP, TINY, e4m3_values

# bf16 terms beside a query's values and the softmax weights: 1 for bf16 queries, 2 for
# fp16, 3 for fp32. n terms leave 2^-8n of the value (each rounding half a step, 2^-8).
TERMS = {"bf16": 1, "f16": 2, "f32": 3}


def rotate(x, gain, positions, freqs, eps=1e-6):
    """Result (n, heads, w) and the sum of the magnitudes that each value of it is made of."""
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = x * r * gain
    return turn(y, positions, freqs)


def turn(y, positions, freqs, back=False):
    half = len(freqs)
    a = positions.astype(np.float64)[:, None] * freqs
    c, s = np.cos(a)[:, None], np.sin(a)[:, None] * (-1 if back else 1)
    out, size = y.copy(), np.abs(y)
    lo, hi = y[..., :half], y[..., half:2 * half]
    out[..., :half] = lo * c - hi * s
    out[..., half:2 * half] = hi * c + lo * s
    both = np.abs(lo) + np.abs(hi)
    size[..., :half] = size[..., half:2 * half] = both
    return out, size


def rotate_tol(y, size, out):
    """w + 40 steps: w for the sum of squares, the rest for the reciprocal root, the
    products and the angle (a rounding of at most pi to 24 bits, sine and cosine each
    within two units)."""
    return (y.shape[-1] + 40) * 2.0 ** -24 * size + HALF_ULP[out] * 1.01 * np.abs(y) + TINY[out]


def rotate_grad(x, gain, positions, freqs, dy, eps=1e-6):
    """dx, dgain and the magnitudes they are made of."""
    w = x.shape[-1]
    u, size = turn(dy, positions, freqs, back=True)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    inner = (u * gain * x).mean(-1, keepdims=True)
    inner_size = (size * np.abs(gain * x)).mean(-1, keepdims=True)
    dx = r * gain * u - x * r ** 3 * inner
    dx_size = r * np.abs(gain) * size + np.abs(x) * r ** 3 * inner_size
    dg = (u * x * r).sum((0, 1))
    dg_size = (size * np.abs(x) * r).sum((0, 1))
    steps = 2 * w + 80
    return dx, steps * 2.0 ** -24 * dx_size, dg, (steps + x.shape[0] * x.shape[1]) * 2.0 ** -24 * dg_size


def softmax(s):
    if s.shape[-1] == 0:
        return s
    with np.errstate(invalid="ignore"):
        m = s.max(-1, keepdims=True)
        e = np.where(np.isneginf(m), 0.0, np.exp(s - np.where(np.isneginf(m), 0.0, m)))
        total = e.sum(-1, keepdims=True)
    return np.divide(e, total, out=np.zeros_like(e), where=total != 0)


def store_values(codes, scales, block, fmt):
    """Values of stored rows: codes (rows x d uint8) and E8M0 bytes."""
    v = e4m3_values()[codes] if fmt == "f8" else codes.view(np.int8).astype(np.float64)
    f = np.exp2(scales.astype(np.float64) - 127)
    f[scales == 255] = np.nan
    return v * f[:, np.arange(codes.shape[1]) // block]


def decode(q, k, v, scale, dtype):
    """One sequence: q hq x w, k and v places x hk x w. Result, what it may be off by,
    the weights of the places summed over the heads and what they may be off by."""
    hq, w = q.shape
    out, tol = np.zeros((hq, w)), np.zeros((hq, w))
    weight, wtol = np.zeros(len(k)), np.zeros(len(k))
    if len(k) == 0:
        return out, tol, weight, wtol
    group = hq // k.shape[1]
    for h in range(hq):
        kh, vh = k[:, h // group], v[:, h // group]
        p = softmax(kh @ q[h] * scale)
        # a score is a sum of w products for each term; its error is that of its weight,
        # relatively, and the largest one is that of their sum
        d = abs(scale) * (np.abs(kh) @ np.abs(q[h])) * ((TERMS[dtype] * w + 8) * SUM_ULP)
        rel = 2.1 * d.max() + (len(k) + 16) * SUM_ULP
        rounded = 2.0 ** (-8 * TERMS[dtype])
        out[h] = p @ vh
        tol[h] = (rel + rounded * 1.01) * (p @ np.abs(vh)) + HALF_ULP[dtype] * 1.01 * np.abs(out[h]) \
            + TINY[dtype]
        weight += p
        wtol += p * rel
    return out, tol, weight, wtol + hq * SUM_ULP * weight


def evict(weights, length, keep, recent):
    """Places that stay, in order."""
    if length <= keep:
        return list(range(length))
    w = np.where(np.isnan(weights), -np.inf, weights)
    old = sorted(range(length - recent), key=lambda p: (-w[p], p))[:keep - recent]
    return sorted(old) + list(range(length - recent, length))
