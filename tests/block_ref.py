"""Block codes in 64 bits, plainly: the scale rule, rounding to the E4M3 and
int8 grids, and the products and reads of the values that codes stand for."""
import numpy as np

TOP = {"f8": 448.0, "i8": 127.0}
SUM_ULP = 2.0 ** -23   # error of one fp32 addition, rounded or cut, relative to its operands
# The FP8 matrix unit, which results of 16 bits come from, adds products in groups of eight aligned
# to the largest, keeping 13 bits below its exponent: each of the other seven loses less than
# 2^-13 of it, under 2^-10 of the group's largest product together.
FP8_UNIT = 2.0 ** -10
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


def e4m3_values():
    """Value of every E4M3 byte."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if (c & 0x7F) == 0x7F else (-x if c & 0x80 else x)
    return v


def exponent(a, top):
    """Smallest e in [-127, 127] with a <= top 2^e; 0 where a is 0."""
    a = np.asarray(a, np.float64)
    e = np.full(a.shape, -127)
    for _ in range(254):
        e = np.where(a > top * np.exp2(e.astype(np.float64)), e + 1, e)
    return np.where(a > 0, e, 0)


def grid(y, fmt):
    """Nearest code value of y, ties to even, saturating; NaN kept (int8: 0)."""
    if fmt == "i8":
        return np.nan_to_num(np.clip(np.rint(y), -127, 127), nan=0.0)
    size = np.clip(np.abs(y), 2.0 ** -6, 448.0)
    with np.errstate(invalid="ignore"):
        step = np.exp2(np.floor(np.log2(size)) - 3)
    with np.errstate(invalid="ignore", over="ignore"):
        return np.clip(np.rint(y / step) * step, -448.0, 448.0)


def finite_max(x, axis):
    return np.max(np.where(np.isfinite(x), np.abs(x), 0.0), axis=axis, initial=0.0)


def encode(x, fmt="f8", block=128):
    """(code values, exponents) of the rows of x, blocks along the row."""
    x = np.asarray(x, np.float64)
    n, d = x.shape
    nb = -(-d // block)
    codes, e = np.empty((n, d)), np.empty((n, nb), int)
    for b in range(nb):
        part = x[:, b * block:(b + 1) * block]
        e[:, b] = exponent(finite_max(part, 1), TOP[fmt])
        codes[:, b * block:(b + 1) * block] = grid(part * np.exp2(-e[:, b].astype(float))[:, None],
                                                   fmt)
    return codes, e


def encode_tiles(x, block=128):
    x = np.asarray(x, np.float64)
    n, d = x.shape
    codes, e = np.empty((n, d)), np.empty((-(-n // block), -(-d // block)), int)
    for i in range(e.shape[0]):
        for j in range(e.shape[1]):
            at = np.s_[i * block:(i + 1) * block, j * block:(j + 1) * block]
            e[i, j] = exponent(finite_max(x[at], None), 448.0)
            codes[at] = grid(x[at] * 2.0 ** -float(e[i, j]), "f8")
    return codes, e


def values(codes, e, block=128):
    """What codes stand for; e per row and block, or per tile."""
    n, d = codes.shape
    rows = np.arange(n) if e.shape[0] == n else np.arange(n) // block
    return codes * np.exp2(e.astype(np.float64))[rows][:, np.arange(d) // block]


def product(a, b, out):
    """a b^T in 64 bits and how far the sums and one rounding to `out` may be
    off. Each of the k products is exact, and is part of at most k fp32
    additions; results of 16 bits are summed by the FP8 unit."""
    y, size = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = (a.shape[1] + 1) * SUM_ULP * size + HALF_ULP[out] * np.abs(y) + TINY[out]
    if out != "f32":
        tol = tol + FP8_UNIT * size
    return y, tol * (1 + 2.0 ** -8)   # the rounding acts on the summed value, not on y
