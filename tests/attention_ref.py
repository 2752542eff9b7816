"""Attention, norms with rotation and eviction in 64 bits, plainly, with how far
the sums and roundings of a call may be off."""
import numpy as np

from block_ref import HALF_ULP, SUM_ULP, TINY, e4m3_values

# bf16 terms that a query's values are made of: 1 for bf16 queries, 2 for fp16, 3 for fp32; the
# softmax weights have as many, or two for bf16 ones, for which the tolerance allows one. n
# terms leave 2^-8n of the value (each rounding half a step, 2^-8).
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


def seen(lq, lk, causal):
    return np.arange(lk) <= np.arange(lq)[:, None] + lk - lq if causal else np.ones((lq, lk), bool)


def attend(q, k, v, scale, causal, dtype):
    """One head of one sequence (rows x w each): result, what it may be off by, and what it
    may be off by before its rounding."""
    w, lk = q.shape[1], len(k)
    mask = seen(len(q), lk, causal)
    p = softmax(np.where(mask, q @ k.T * scale, -np.inf))
    rel = p_error(q, k, scale, mask, w)
    out = p @ v
    inner = (p * (rel + HALF_ULP[dtype] * 1.01)) @ np.abs(v)
    return out, inner + HALF_ULP[dtype] * 1.01 * np.abs(out) + TINY[dtype], inner


def p_error(q, k, scale, mask, w):
    """Relative error of the softmax weights of each row: that of its scores (w products and
    additions) twice, once by the sum, and that of the sum of its weights."""
    if not mask.shape[1]:
        return np.zeros((len(q), 1))
    d = np.where(mask, np.abs(scale) * (np.abs(q) @ np.abs(k).T), 0.0).max(1, keepdims=True) * ((w + 8) * SUM_ULP)
    return 2.1 * d + (mask.shape[1] + 24) * SUM_ULP


def attend_grad(q, k, v, do, scale, causal, dtype, top=None):
    """One head of one sequence: (dq, dk, dv) and what each may be off by. top: the largest
    |dO| and |V| of the call, for fp16's weights' gradients: 2^-38 of 2 w top for what the
    step at zero takes from them (they are kept times a power of two of their row)."""
    w = q.shape[1]
    mask = seen(len(q), len(k), causal)
    p = softmax(np.where(mask, q @ k.T * scale, -np.inf))
    rel = p_error(q, k, scale, mask, w)
    out = p @ v
    dp, d = do @ v.T, (do * out).sum(1, keepdims=True)
    ds = p * (dp - d)
    dq, dk, dv = scale * ds @ k, scale * ds.T @ q, p.T @ do
    half = HALF_ULP[dtype] * 1.01
    # O stands in D as it was before its rounding to 16 bits, with 16 bits more or less
    o_off = (p * (rel + half)) @ np.abs(v) + half * half * np.abs(out) + TINY[dtype]
    d_off = (np.abs(do) * o_off).sum(1, keepdims=True) + (w + 8) * SUM_ULP * (np.abs(do) * np.abs(out)).sum(1, keepdims=True)
    dp_off = (w + 8) * SUM_ULP * (np.abs(do) @ np.abs(v).T)
    steps = max(len(q), len(k)) + 16
    off = p * (dp_off + d_off) + np.abs(ds) * (rel + half + steps * SUM_ULP) + 4 * SUM_ULP * p * (np.abs(dp) + np.abs(d))
    pv_off = p * (rel + half + steps * SUM_ULP)
    if dtype == "f16":
        off = off + mask * 2.0 ** -24 * 2 * w * (top or 0.0) / 2.0 ** 14
        pv_off = pv_off + mask * 2.0 ** -24 * 2.0 ** -14
    tols = (abs(scale) * off @ np.abs(k), abs(scale) * off.T @ np.abs(q), pv_off.T @ np.abs(do))
    return (dq, dk, dv), tols


def grad_slopes(q, k, v, do, grads, scale, causal, dtype):
    """One sequence (rows x heads x w each), for dq, dk and dv of `grads` in turn along the
    definition's own gradient (a part that is missing or too much shows there): the change of
    sum(o do) that they say, the one that differences of the definition give (to
    some 1e-9 of it), and what the first may be off by."""
    hq, group, inputs = q.shape[1], q.shape[1] // k.shape[1], [q, k, v]

    def loss(x):
        return sum((attend(x[0][:, h], x[1][:, h // group], x[2][:, h // group], scale, causal, dtype)[0] * do[:, h]).sum()
                   for h in range(hq))

    exact, tols = ([np.zeros(x.shape) for x in inputs] for _ in range(2))
    for h in range(hq):
        kv = h // group
        top = np.abs(do[:, h]).max() * np.abs(v[:, kv]).max()
        values, off = attend_grad(q[:, h], k[:, kv], v[:, kv], do[:, h], scale, causal, dtype, top)
        for i, at in enumerate((h, kv, kv)):
            exact[i][:, at] += values[i]
            tols[i][:, at] += off[i]
    for i, (g, e, t) in enumerate(zip(grads, exact, tols)):
        way = e / np.linalg.norm(e)
        ends = [loss([x + sign * 1e-4 * way if j == i else x for j, x in enumerate(inputs)]) for sign in (1, -1)]
        t = t + (HALF_ULP[dtype] * 1.01 + group * SUM_ULP) * np.abs(e) + TINY[dtype]
        yield (g * way).sum(), (ends[0] - ends[1]) / 2e-4, (np.abs(way) * t).sum()
