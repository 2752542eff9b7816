"""Block codes on the GPU at the edges of their number formats, for every kernel
of the product: scale bytes of NaN beside any other scale."""
import numpy as np
import pytest

import block_ref as ref
from test_gpu_block import NUMBERS, T, f64, mm  # noqa: F401

pytestmark = pytest.mark.gpu


def on_gpu(byte, ebyte, pitch=0):
    """Codes with rows `pitch` bytes past a multiple of 16 apart, and scales."""
    import torch
    n, k = byte.shape
    room = torch.full((n, -(-k // 16) * 16 + pitch), 0x7F, dtype=torch.uint8, device="cuda")
    codes = room[:, :k]
    codes.copy_(torch.from_numpy(byte))
    return codes.view(torch.float8_e4m3fn), torch.from_numpy(ebyte.astype(np.uint8)).cuda()


def finite_codes(rng, n, k):
    byte = rng.integers(0, 256, (n, k)).astype(np.uint8)
    byte[(byte & 0x7F) == 0x7F] = 0x40
    return byte


# Sizes of every kernel: rows, rows of k-steps shared by waves, 64 x 64, its split of k, 128 x 128
# (whole lines of fp32 and not), 256 x 256 with 16-bit results, rows past whole rounds of tiles,
# rows that do not start at multiples of 16 bytes.
KERNELS = [(1, 140, 384, 0), (16, 140, 2100, 0), (40, 140, 384, 0), (40, 140, 4096, 0),
           (300, 200, 4000, 0), (1500, 1480, 384, 0), (1500, 1490, 1100, 0), (4000, 4090, 300, 0),
           (4099, 4096, 384, 0), (40, 140, 384, 1), (300, 140, 500, 3)]


@pytest.mark.parametrize("m,n,k,pitch", KERNELS)
@pytest.mark.parametrize("other", [0, 60, 127, 194])
def test_nan_scale_beside_any_other(mm, m, n, k, pitch, other):
    """A scale byte of 255 makes every output it enters NaN, whatever the other
    side's scale of that block, and where the block's codes are zeros too."""
    rng = np.random.default_rng(m + other)
    ba, bb = finite_codes(rng, m, k), finite_codes(rng, n, k)
    kb = -(-k // 128)
    ea, eb = rng.integers(115, 140, (m, kb)), rng.integers(115, 140, (n, kb))
    eb[:, 1] = ea[:, 2] = other
    va = ref.values(ref.e4m3_values()[ba], ea - 127)
    vb = ref.values(ref.e4m3_values()[bb], eb - 127)
    rows, cols = {m // 2, m - 1}, {3, 7}
    for r in rows:
        ea[r, 1] = 255                       # beside b's `other`
    for c in cols:
        eb[c, 2] = 255                       # beside a's
    ba[m - 1, 128:256] = 0
    bb[7, 256:384] = 0
    bad = np.zeros((m, n), bool)
    bad[list(rows)] = True
    bad[:, list(cols)] = True
    a, sa = on_gpu(ba, ea, pitch)
    b, sb = on_gpu(bb, eb, pitch)
    for out in NUMBERS:
        y, tol = ref.product(va, vb, out)
        got = f64(mm.block_matmul(a, sa, b, sb, out_dtype=T(out)))
        assert np.array_equal(np.isnan(got), bad), (out, int((np.isnan(got) != bad).sum()))
        ok = ~bad & ((np.abs(y) + tol < 65504) if out == "f16" else True)
        assert np.all(np.abs(got - y)[ok] <= tol[ok]), out
