"""Block codes on the GPU at the edges of their number formats, for every kernel
of the product: scale bytes of NaN beside any other scale, scales at both ends
of their range, and exact integers at sizes of each kernel."""
import numpy as np
import pytest

import block_ref as ref
from test_gpu_block import NUMBERS, T, code_matrix, f64, mm, numbers  # noqa: F401

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


@pytest.mark.parametrize("m,n,k,pitch", KERNELS)
def test_nan_codes(mm, m, n, k, pitch):
    """NaN codes of either sign, in the first and the last place of a row."""
    rng = np.random.default_rng(m)
    ba, bb = finite_codes(rng, m, k), finite_codes(rng, n, k)
    ba[m - 1, k - 1] = 0xFF
    bb[3, 0], bb[5, k - 1] = 0x7F, 0xFF
    bad = np.zeros((m, n), bool)
    bad[m - 1] = bad[:, 3] = bad[:, 5] = True
    kb = -(-k // 128)
    a, sa = on_gpu(ba, np.full((m, kb), 120), pitch)
    b, sb = on_gpu(bb, np.full((n, kb), 125), pitch)
    for out in NUMBERS:
        got = f64(mm.block_matmul(a, sa, b, sb, out_dtype=T(out)))
        assert np.array_equal(np.isnan(got), bad), out


def exact(mm, rng, m, n, k, pitch, ea, eb):
    """Integer codes of -8 .. 8: with scales that leave sums below 2^24, exact in
    either matrix unit, so the result is the rounded sum. This pins each value
    and each scale to its place."""
    import torch
    va, vb = (rng.integers(-8, 9, (rows, k)).astype(float) for rows in (m, n))
    code = lambda v: torch.from_numpy(v).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()  # noqa: E731
    a, sa = on_gpu(code(va), ea + 127, pitch)
    b, sb = on_gpu(code(vb), eb + 127, pitch)
    y = torch.from_numpy(ref.values(va, ea) @ ref.values(vb, eb).T)
    for out in NUMBERS:
        got = mm.block_matmul(a, sa, b, sb, out_dtype=T(out)).cpu()
        assert torch.equal(got, y.to(T(out))), (out, int((got != y.to(T(out))).sum()))


@pytest.mark.parametrize("m,n,k,pitch", KERNELS + [(4100, 4100, 520, 0), (4096, 4099, 768, 0)])
@pytest.mark.parametrize("tiles", [False, True])
def test_matmul_of_small_integers_is_exact_in_every_kernel(mm, m, n, k, pitch, tiles):
    rng = np.random.default_rng(m + n + k)
    kb = -(-k // 128)
    exact(mm, rng, m, n, k, pitch, rng.integers(0, 2, (m, kb)),
          rng.integers(0, 2, (-(-n // 128) if tiles else n, kb)))


@pytest.mark.parametrize("m,n,k,pitch", KERNELS)
def test_scales_at_both_ends_cancel(mm, m, n, k, pitch):
    """Scales from 2^-127 to 2^127 whose products are 1 and 2: beyond what the
    bf16 unit's operands hold (2^+-50), in splits of k and in redone tiles too."""
    rng = np.random.default_rng(m + n + k)
    kb = -(-k // 128)
    e = rng.choice([-127, -90, -51, -50, 0, 50, 51, 90, 126], kb)
    exact(mm, rng, m, n, k, pitch, e + rng.integers(0, 2, (m, kb)), np.tile(-e, (n, 1)))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m", [1, 9, 16, 40, 300])
def test_linear_special_rows_in_the_default_type(mm, dtype, m):
    """Zero rows, infinities and NaN of x, and rows that start at odd places:
    results of x's own 16-bit type."""
    import torch
    n, k = 200, 300
    wide = numbers(m, k + 40, dtype, 3, spread=0.1)
    x = wide[:, 7:7 + k]
    x[0, :] = 0
    if m > 3:
        x[1, 5], x[2, 150], x[3, 299] = float("inf"), float("nan"), -float("inf")
    w, sw, vw = code_matrix(n, k, 4)
    y, tol = ref.product(ref.values(*ref.encode(f64(x))), vw, dtype)
    got = f64(mm.block_linear(x, (w, sw)))
    assert np.array_equal(np.isnan(got), np.isnan(y)) and np.all(got[0] == 0)
    ok = ~np.isnan(y) & ((np.abs(y) + tol < 65504) if dtype == "f16" else True)
    assert np.all(np.abs(got - y)[ok] <= tol[ok])


@pytest.mark.parametrize("dtype", NUMBERS)
@pytest.mark.parametrize("m", [1, 9, 16, 40])
def test_linear_rows_at_odd_starts(mm, dtype, m):
    n, k = 200, 300
    x = numbers(m, k + 40, dtype, 3, spread=0.1)[:, 7:7 + k]
    w, sw, vw = code_matrix(n, k, 4)
    y, tol = ref.product(ref.values(*ref.encode(f64(x))), vw, "f32")
    got = f64(mm.block_linear(x, (w, sw), out_dtype=T("f32")))
    assert np.all(np.abs(got - y) <= tol)


def test_blocks_whose_lower_half_is_another(mm):
    """A block is its whole number, not its lower 32 or 64 bits: scales of one
    per row would be too few for it."""
    import torch
    codes, scales = mm.cache_new(6, 200)
    x, slots = numbers(4, 200, "f32", 1), torch.arange(4, device="cuda")
    pages = codes.view(2, 3, 200), scales[:, :1].contiguous().view(2, 3, 1)
    for block in (2 ** 32 + 128, 2 ** 64 + 128, 0, -128, 8, 24, 272):
        one = scales[:, :1].contiguous()
        for call in (lambda: mm.cache_write(x, slots, codes, one, block=block),
                     lambda: mm.cache_read(codes, one, slots, block=block),
                     lambda: mm.cache_read_pages(*pages, slots.int()[None, :2], slots.int()[:2], 1,
                                                 block=block)):
            with pytest.raises(mm.EmeansError, match="EINVAL.*block"):
                call()


@pytest.mark.parametrize("need", ["x", "w", "both"])
def test_linear_keeps_what_its_gradients_need(mm, need):
    """Between the passes: 1 byte for each value of w if x has a gradient, of x
    if w has one, and their scales; the gradients are those of both together."""
    import torch
    m, n, k = 4096, 640, 1152
    x, w = numbers(m, k, "bf16", 1, 0.1), numbers(n, k, "bf16", 2, 0.1)
    g = numbers(m, n, "bf16", 3, 0.1)
    want = x.clone().requires_grad_(), w.clone().requires_grad_()
    mm.block_linear(*want).backward(g)
    xs = x.clone().requires_grad_(need != "w")
    ws = w.clone().requires_grad_(need != "x")
    y = mm.block_linear(xs, ws)
    kept = sum(t.untyped_storage().nbytes() for t in y.grad_fn.saved_tensors)
    parts = {"x": n * k, "w": m * k, "both": (m + n) * k}
    assert kept <= parts[need] * (1 + 2 / 128) + 4096, (kept, parts[need])
    y.backward(g)
    assert xs.grad is None or torch.equal(xs.grad, want[0].grad)
    assert ws.grad is None or torch.equal(ws.grad, want[1].grad)
    assert (xs.grad is None, ws.grad is None) == (need == "w", need == "x")


@pytest.mark.parametrize("grad", [False, True])
def test_linear_refuses_forward_mode(mm, grad):
    """There is no forward-mode derivative: a tangent is refused, not dropped."""
    import torch
    import torch.autograd.forward_ad as fw
    x, w = numbers(4, 200, "f32", 1), numbers(30, 200, "f32", 2)
    codes = mm.block_encode(w, tiles=True, cols=True)
    with fw.dual_level():
        dx, dw = (fw.make_dual(t.clone().requires_grad_(grad), torch.ones_like(t)) for t in (x, w))
        for call in (lambda: mm.block_linear(dx, codes), lambda: mm.block_linear(dx, w),
                     lambda: mm.block_linear(x, dw), lambda: mm.block_linear(dx, dw)):
            with pytest.raises(mm.EmeansError, match="EINVAL.*forward-mode"):
                call()
        assert mm.block_linear(x, codes[:2]).shape == (4, 30)   # no tangent: fine
    with pytest.raises(mm.EmeansError, match="EINVAL.*forward-mode"):
        torch.func.jvp(lambda t: mm.block_linear(t, codes), (x,), (x,))


def test_tracing_is_refused(mm):
    """A trace records torch operations alone: calls of the library would be lost."""
    import torch
    x, w = numbers(4, 200, "f32", 1), numbers(30, 200, "f32", 2)
    c, s = mm.block_encode(w)
    store, factors = mm.cache_new(8, 200)
    slots = torch.arange(4, device="cuda")
    for call in (lambda t: mm.block_linear(t, w), lambda t: mm.block_linear(t, (c, s)),
                 lambda t: mm.block_encode(t)[0], lambda t: mm.block_matmul(*mm.block_encode(t), c, s),
                 lambda t: mm.cache_write(t, slots, store, factors),
                 lambda t: t + mm.cache_read(store, factors, slots)):
        with pytest.raises(mm.EmeansError, match="EINVAL.*trace"):
            torch.jit.trace(call, (x,), check_trace=False)


def test_negative_total_is_refused(mm):
    import torch
    codes, scales = mm.cache_new((2, 3), 64)
    at = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(mm.EmeansError, match="EINVAL.*total"):
        mm.cache_read_pages(codes, scales, at[None], at, -1)


def test_store_of_numpy_sizes(mm):
    codes, scales = mm.cache_new(np.int64(6), np.int32(200))
    assert codes.shape == (6, 200) and scales.shape == (6, 2)
    codes, scales = mm.cache_new((np.int64(2), 3), 64)
    assert codes.shape == (2, 3, 64) and scales.shape == (2, 3, 1)


def test_linear_without_columns_or_dimensions(mm):
    """k = 0 in any shape gives zeros; a number is no row."""
    import torch
    w = (torch.empty(5, 0, dtype=torch.float8_e4m3fn, device="cuda"),
         torch.empty(5, 0, dtype=torch.uint8, device="cuda"))
    for shape in ((3, 0), (2, 3, 0), (0,)):
        y = mm.block_linear(torch.empty(shape, device="cuda"), w)
        assert y.shape == (*shape[:-1], 5) and torch.all(y == 0)
    with pytest.raises(mm.EmeansError, match="EINVAL"):
        mm.block_linear(torch.ones((), device="cuda"), w)


@pytest.mark.parametrize("block", [0, -16, 8, 100, 272])
def test_store_of_an_impossible_block_is_refused(mm, block):
    with pytest.raises(mm.EmeansError, match="EINVAL.*block"):
        mm.cache_new(4, 64, block=block)
