"""Block codes on the GPU against their definition in 64 bits: encoding and
reading back are exact, products within the bound of fp32 sums and one rounding
(block_ref.product), gradients equal the formula's and central differences."""
import numpy as np
import pytest

import block_ref as ref

pytestmark = pytest.mark.gpu

NUMBERS = ["f32", "bf16", "f16"]


@pytest.fixture(scope="module")
def mm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mini_means_amd
    mini_means_amd.lib()
    return mini_means_amd


def T(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
            "f8": torch.float8_e4m3fn, "i8": torch.int8}[name]


def numbers(n, d, dtype, seed, spread=1.0):
    """n x d tensor on the GPU of values of many sizes."""
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, d, generator=g) * torch.exp2(4 * torch.randn(n, 1, generator=g) * spread)
    return x.to(T(dtype)).cuda()


def f64(t):
    return t.detach().float().cpu().double().numpy()


def expo(s):
    import torch
    return s.view(torch.uint8).cpu().numpy().astype(int) - 127


def check_codes(codes, scales, want):
    assert np.array_equal(f64(codes), want[0], equal_nan=True)
    assert np.array_equal(expo(scales), want[1])


def code_matrix(n, k, seed, tiles=False, pitch=None, offset=0):
    """Random finite codes and scales with rows `pitch` apart, `offset` bytes
    from an aligned address; on the GPU and as 64-bit values."""
    import torch
    rng = np.random.default_rng(seed)
    byte = rng.integers(0, 256, (n, k)).astype(np.uint8)
    byte[(byte & 0x7F) == 0x7F] = 0x40
    kb = -(-k // 128)
    e = rng.integers(-12, 13, (-(-n // 128) if tiles else n, kb))
    pitch = pitch or -(-k // 16) * 16
    room = torch.full((n * pitch + offset + 64,), 0x7F, dtype=torch.uint8, device="cuda")  # NaN around
    codes = room[offset:offset + n * pitch].view(n, pitch)[:, :k]
    codes.copy_(torch.from_numpy(byte))
    return (codes.view(torch.float8_e4m3fn),
            torch.from_numpy((e + 127).astype(np.uint8)).cuda().view(torch.float8_e8m0fnu),
            ref.values(ref.e4m3_values()[byte], e))


# ---- encoding ------------------------------------------------------------------
@pytest.mark.parametrize("dtype", NUMBERS)
@pytest.mark.parametrize("n,d", [(1, 1), (3, 127), (2, 128), (17, 129), (33, 769), (130, 1000)])
def test_encode_rows(mm, dtype, n, d):
    x = numbers(n, d, dtype, n * d)
    codes, scales = mm.block_encode(x)
    assert codes.shape == (n, d) and scales.shape == (n, -(-d // 128))
    check_codes(codes, scales, ref.encode(f64(x)))


@pytest.mark.parametrize("dtype", NUMBERS)
@pytest.mark.parametrize("n,d", [(1, 1), (127, 129), (128, 128), (300, 200), (1, 500), (513, 64)])
def test_encode_both_and_tiles(mm, dtype, n, d):
    x = numbers(n, d, dtype, n + d)
    v = f64(x)
    c, s, ct, st = mm.block_encode(x, cols=True)
    check_codes(c, s, ref.encode(v))
    check_codes(ct, st, ref.encode(v.T))
    a, b, ct, st = mm.block_encode(x, cols=True, rows=False)
    assert a is None and b is None
    check_codes(ct, st, ref.encode(v.T))
    want = ref.encode_tiles(v)
    c, s, ct, st = mm.block_encode(x, tiles=True, cols=True)
    check_codes(c, s, want)
    check_codes(ct, st, (want[0].T, want[1].T))
    check_codes(*mm.block_encode(x, tiles=True), want)


@pytest.mark.parametrize("dtype", NUMBERS)
def test_encode_strides_and_alignment(mm, dtype):
    for first, step in ((1, 1), (3, 2), (8, 1)):
        wide = numbers(50, 400, dtype, first)
        x = wide[::step, first:first + 259]
        v = f64(x)
        check_codes(*mm.block_encode(x), ref.encode(v))
        c, s, ct, st = mm.block_encode(x, cols=True)
        check_codes(c, s, ref.encode(v))
        check_codes(ct, st, ref.encode(v.T))
        check_codes(*mm.block_encode(x, tiles=True), ref.encode_tiles(v))


@pytest.mark.parametrize("form", ["rows", "both", "tiles"])
def test_encode_special_values(mm, form):
    """Zero blocks, infinities, NaN, subnormals, the largest number, ties."""
    import torch
    x = torch.zeros(140, 300)
    inf, nan, big = float("inf"), float("nan"), 3.4028234663852886e38
    x[1, :5] = torch.tensor([inf, -inf, 1.0, nan, -3.0])
    x[2, 200] = nan
    x[3, :3] = inf
    x[4, :3] = torch.tensor([big, -big, 1e30])
    x[5, 130:133] = torch.tensor([1e-45, -3e-42, 2e-39])
    x[6, :6] = torch.tensor([448.0, 17.0, 19.0, 2.0 ** -9, 3 * 2.0 ** -10, -2.0 ** -10])
    x[7, :3] = torch.tensor([448.0001, 1.0, 2.0 ** -10])
    x[8] = 2.0 ** -130
    x[130:, 290:] = 5.0
    v = x.double().numpy()
    if form == "tiles":
        want = ref.encode_tiles(v)
        c, s, ct, st = mm.block_encode(x.cuda(), tiles=True, cols=True)
        check_codes(ct, st, (want[0].T, want[1].T))
    else:
        want = ref.encode(v)
        if form == "rows":
            c, s = mm.block_encode(x.cuda())
        else:
            c, s, ct, st = mm.block_encode(x.cuda(), cols=True)
            check_codes(ct, st, ref.encode(v.T))
    check_codes(c, s, want)


def test_encode_nothing(mm):
    import torch
    c, s, ct, st = mm.block_encode(torch.empty(0, 200, device="cuda"), cols=True)
    assert c.shape == (0, 200) and s.shape == (0, 2) and ct.shape == (200, 0) and st.shape == (200, 0)


# ---- products -------------------------------------------------------------------
SHAPES = [(1, 1, 1), (1, 17, 128), (1, 1000, 769), (2, 256, 4096), (5, 300, 200), (16, 515, 1024),
          (17, 130, 384), (33, 1029, 640), (64, 64, 2048), (65, 129, 257), (100, 520, 1000),
          (130, 250, 128), (200, 333, 1536), (257, 511, 896), (400, 1025, 130), (770, 300, 520)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("tiles", [False, True])
def test_matmul(mm, m, n, k, tiles):
    a, sa, va = code_matrix(m, k, m + k)
    b, sb, vb = code_matrix(n, k, n, tiles)
    for out in NUMBERS:
        y, tol = ref.product(va, vb, out)
        got = mm.block_matmul(a, sa, b, sb, out_dtype=T(out))
        fits = np.abs(y) + tol < 65504 if out == "f16" else np.ones_like(y, bool)
        err = np.abs(f64(got) - y)
        assert got.shape == (m, n)
        assert np.all(err[fits] <= tol[fits]), float(np.max(err[fits] / tol[fits]))


@pytest.mark.parametrize("m,n,k", [(1500, 1490, 200), (1500, 1480, 640), (4096, 4100, 128),
                                   (4100, 4100, 300), (4097, 4096, 512), (4096, 4096, 896),
                                   (5, 131150, 100), (16, 131072, 128), (300, 200, 4000)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_matmul_large(mm, m, n, k, out):
    """Sizes of every tile, k of one stage, of odd and even counts, and with a
    short last stage; k split over workgroups."""
    a, sa, va = code_matrix(m, k, m + k)
    b, sb, vb = code_matrix(n, k, n, True)
    y, tol = ref.product(va, vb, out)
    got = mm.block_matmul(a, sa, b, sb, out_dtype=T(out))
    err = np.abs(f64(got) - y)
    assert np.all(err <= tol), float(np.max(err / tol))


@pytest.mark.parametrize("m,n,k", [(1, 300, 500), (20, 300, 500), (150, 200, 300), (300, 520, 1100)])
@pytest.mark.parametrize("pitch,offset", [(0, 1), (1, 0), (16, 8), (3, 5), (32, 16)])
def test_matmul_alignment_and_tails(mm, m, n, k, pitch, offset):
    """Any pitch, any start, NaN codes in every byte beside the values."""
    a, sa, va = code_matrix(m, k, 1, pitch=-(-k // 16) * 16 + pitch, offset=offset)
    b, sb, vb = code_matrix(n, k, 2, True, pitch=-(-k // 16) * 16 + pitch, offset=offset)
    y, tol = ref.product(va, vb, "f32")
    import torch
    out = torch.full((m, n + 3), 7.0, device="cuda")
    got = mm.block_matmul(a, sa, b, sb, out=out[:, 1:n + 1])
    assert np.all(np.abs(f64(got) - y) <= tol)
    assert torch.all(out[:, 0] == 7) and torch.all(out[:, n + 1:] == 7)


@pytest.mark.parametrize("m,n,k,out", [(4099, 4096, 160, "bf16"), (4196, 4096, 100, "f16"),
                                       (4096, 4103, 256, "bf16"), (4100, 4296, 130, "f16"),
                                       (4098, 4096, 2048, "f32"), (4096, 4196, 2000, "f32"),
                                       (4120, 4100, 2048, "f32"), (4100, 4112, 4096, "bf16")])
@pytest.mark.parametrize("tiles", [False, True])
def test_matmul_a_little_over_whole_rounds(mm, m, n, k, out, tiles):
    """The rows and columns past the large tiles are products of their own: their
    scales, their places in a wider result, and nothing beside it written."""
    import torch
    a, sa, va = code_matrix(m, k, m + k)
    b, sb, vb = code_matrix(n, k, n, tiles)
    y, tol = ref.product(va, vb, out)
    wide = torch.full((m, n + 5), 7.0, device="cuda", dtype=T(out))
    got = mm.block_matmul(a, sa, b, sb, out=wide[:, 2:n + 2])
    err = np.abs(f64(got) - y)
    fits = np.abs(y) + tol < 65504 if out == "f16" else np.ones_like(y, bool)
    assert np.all(err[fits] <= tol[fits]), float(np.max(err[fits] / tol[fits]))
    assert torch.all(wide[:, :2] == 7) and torch.all(wide[:, n + 2:] == 7)


@pytest.mark.parametrize("m", [1, 16, 40, 200, 300])
@pytest.mark.parametrize("out", NUMBERS)
def test_matmul_of_small_integers_is_exact(mm, m, out):
    """Integers whose sums stay below 2^24, products of one group of k within
    2^6 of each other: exact in either unit, so the result is the rounded sum.
    This pins each value and each scale to its place."""
    import torch
    rng = np.random.default_rng(m)
    n, k = 390, 1280
    va = rng.integers(-8, 9, (m, k)).astype(float)
    vb = rng.integers(-8, 9, (n, k)).astype(float)
    ea, eb = rng.integers(0, 2, (m, k // 128)), rng.integers(0, 2, (n, k // 128))
    dev = lambda v: torch.from_numpy(v).float().cuda().to(torch.float8_e4m3fn)  # noqa: E731
    sc = lambda e: torch.from_numpy((e + 127).astype(np.uint8)).cuda()  # noqa: E731
    for e in (eb, eb[::128]):
        got = mm.block_matmul(dev(va), sc(ea), dev(vb), sc(e), out_dtype=T(out))
        want = torch.from_numpy(ref.values(va, ea) @ ref.values(vb, e).T).to(T(out))
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("m,n", [(1, 140), (30, 140), (140, 140), (300, 140), (1500, 1480)])
def test_matmul_nan_and_extreme_scales(mm, m, n):
    import torch
    k = 384
    a, sa, va = code_matrix(m, k, 5)
    b, sb, vb = code_matrix(n, k, 6)
    a.view(torch.uint8)[m - 1, 200] = 0x7F
    b.view(torch.uint8)[3, 383] = 0xFF
    sb.view(torch.uint8)[7, 1] = 255
    got = f64(mm.block_matmul(a, sa, b, sb, out_dtype=torch.float32))
    bad = np.zeros((m, n), bool)
    bad[m - 1] = bad[:, 3] = bad[:, 7] = True
    assert np.array_equal(np.isnan(got), bad)
    y, tol = ref.product(va, vb, "f32")
    assert np.all(np.abs(got - y)[~bad] <= tol[~bad])
    # scales at the ends of their range: 2^-127 against 2^127, and back
    one = torch.full((m, 128), 1.0, device="cuda").to(torch.float8_e4m3fn)
    other = torch.full((n, 128), 2.0, device="cuda").to(torch.float8_e4m3fn)
    for low, high in ((0, 254), (254, 0), (100, 150)):
        got = mm.block_matmul(one, torch.full((m, 1), low, device="cuda", dtype=torch.uint8), other,
                              torch.full((n, 1), high, device="cuda", dtype=torch.uint8),
                              out_dtype=torch.float32)
        assert torch.all(got == 256.0 * 2.0 ** (low + high - 254))


def test_matmul_without_k_is_zero(mm):
    import torch
    c = lambda n: torch.empty(n, 0, dtype=torch.float8_e4m3fn, device="cuda")  # noqa: E731
    s = lambda n: torch.empty(n, 0, dtype=torch.uint8, device="cuda")  # noqa: E731
    got = mm.block_matmul(c(3), s(3), c(5), s(5), out_dtype=torch.float32)
    assert got.shape == (3, 5) and torch.all(got == 0)
    assert mm.block_matmul(c(0), s(0), c(5), s(5)).shape == (0, 5)


def test_matmul_same_result_every_time(mm):
    """No atomics in the sums: two runs agree bit for bit."""
    import torch
    for m, n, k in ((1, 1000, 2048), (48, 700, 4096), (130, 260, 8192), (300, 300, 512),
                    (1500, 1500, 700), (4200, 4100, 384)):
        a, sa, _ = code_matrix(m, k, 1)
        b, sb, _ = code_matrix(n, k, 2, True)
        first = mm.block_matmul(a, sa, b, sb, out_dtype=torch.float32)
        for _ in range(3):
            assert torch.equal(first, mm.block_matmul(a, sa, b, sb, out_dtype=torch.float32))


# ---- linear ---------------------------------------------------------------------
@pytest.mark.parametrize("dtype", NUMBERS)
@pytest.mark.parametrize("m,n,k", [(1, 300, 1000), (3, 515, 256), (16, 260, 777), (17, 260, 1024),
                                   (70, 130, 384), (300, 520, 640)])
def test_linear_with_codes(mm, dtype, m, n, k):
    x = numbers(m, k, dtype, m, spread=0.2)
    w, sw, vw = code_matrix(n, k, 9, True)
    vx = ref.values(*ref.encode(f64(x)))
    for out in ("f32", dtype):
        y, tol = ref.product(vx, vw, out)
        got = mm.block_linear(x, (w, sw), out_dtype=T(out))
        fits = np.abs(y) + tol < 65504 if out == "f16" else np.ones_like(y, bool)
        assert np.all(np.abs(f64(got) - y)[fits] <= tol[fits])


@pytest.mark.parametrize("m", [1, 9, 40])
def test_linear_special_rows_and_layouts(mm, m):
    """Zero rows, infinities, NaN; three dimensions; a column slice."""
    import torch
    n, k = 200, 300
    wide = numbers(m, k + 40, "bf16", 3, spread=0.1)
    x = wide[:, 8:8 + k]
    x[0, :] = 0
    if m > 3:
        x[1, 5], x[2, 150], x[3, 299] = float("inf"), float("nan"), -float("inf")
    w, sw, vw = code_matrix(n, k, 4)
    y, tol = ref.product(ref.values(*ref.encode(f64(x))), vw, "f32")
    got = f64(mm.block_linear(x, (w, sw), out_dtype=torch.float32))
    assert np.array_equal(np.isnan(got), np.isnan(y)) and np.all(got[0] == 0)
    ok = ~np.isnan(y)
    assert np.all(np.abs(got - y)[ok] <= tol[ok])
    y3 = mm.block_linear(x.unsqueeze(0), (w, sw), out_dtype=torch.float32)
    assert y3.shape == (1, m, n) and np.array_equal(f64(y3[0]), got, equal_nan=True)
    off = mm.block_linear(wide[:, 7:7 + k], (w, sw), out_dtype=torch.float32)   # odd start
    assert off.shape == (m, n)


@pytest.mark.parametrize("dtype", NUMBERS)
@pytest.mark.parametrize("m,n,k", [(5, 40, 30), (150, 140, 260), (300, 257, 129)])
def test_linear_gradient_formula(mm, dtype, m, n, k):
    import torch
    x = numbers(m, k, dtype, 1, 0.2).requires_grad_()
    w = numbers(n, k, dtype, 2, 0.2).requires_grad_()
    dy = numbers(m, n, dtype, 3, 0.2)
    y = mm.block_linear(x, w)
    y.backward(dy)
    q = lambda v: ref.values(*ref.encode(v))  # noqa: E731
    qw = ref.values(*ref.encode_tiles(f64(w)))
    for got, a, b in ((y, q(f64(x)), qw), (x.grad, q(f64(dy)), qw.T),
                      (w.grad, q(f64(dy).T), q(f64(x).T))):
        want, tol = ref.product(a, b, dtype)
        assert got.dtype == T(dtype) and got.shape == want.shape
        fits = np.abs(want) + tol < 65504 if dtype == "f16" else np.ones_like(want, bool)
        assert np.all(np.abs(f64(got) - want)[fits] <= tol[fits])


def test_linear_gradient_against_differences(mm):
    """Values on a grid that encoding keeps: the function is linear there, so
    central differences give the gradient exactly."""
    import torch
    m, n, k = 7, 9, 150
    rng = np.random.default_rng(8)
    mk = lambda *s: torch.from_numpy(rng.integers(-3, 4, s)).float().cuda()  # noqa: E731
    x, w, dy = mk(m, k), mk(n, k), mk(m, n)
    loss = lambda a, b: (mm.block_linear(a, b).double() * dy).sum().item()  # noqa: E731
    xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
    mm.block_linear(xg, wg).backward(dy)
    for t, g, at in ((0, xg.grad, (3, 140)), (0, xg.grad, (6, 0)), (1, wg.grad, (8, 149)),
                     (1, wg.grad, (0, 77))):
        pair = [x.clone(), w.clone()]
        pair[t][at] += 1
        up = loss(*pair)
        pair[t][at] -= 2
        assert g[at].item() == (up - loss(*pair)) / 2


def test_linear_gradient_paths(mm):
    """Only x, only w, a frozen w as codes, an expanded gradient, leading
    dimensions, no rows."""
    import torch
    x, w = numbers(24, 200, "f32", 1, 0.1), numbers(30, 200, "f32", 2, 0.1)
    xr, wr = x.clone().requires_grad_(), w.clone().requires_grad_()
    mm.block_linear(xr, wr).sum().backward()          # the gradient is expanded ones
    x1 = x.clone().requires_grad_()
    mm.block_linear(x1, w).sum().backward()
    w1 = w.clone().requires_grad_()
    mm.block_linear(x, w1).sum().backward()
    assert torch.equal(x1.grad, xr.grad) and torch.equal(w1.grad, wr.grad)
    frozen = mm.block_encode(w, tiles=True, cols=True)
    x2 = x.clone().requires_grad_()
    mm.block_linear(x2.view(2, 12, 200), frozen).sum().backward()
    assert torch.equal(x2.grad, xr.grad)
    with pytest.raises(mm.EmeansError, match="EINVAL.*transposed"):
        mm.block_linear(x2, frozen[:2])
    with torch.no_grad():
        assert torch.equal(mm.block_linear(x2, frozen[:2]), mm.block_linear(x, w))
    none = torch.empty(0, 200, device="cuda", requires_grad=True)
    w3 = w.clone().requires_grad_()
    y = mm.block_linear(none, w3)
    assert y.shape == (0, 30)
    y.sum().backward()
    assert none.grad.shape == (0, 200) and torch.all(w3.grad == 0)


# ---- the store ------------------------------------------------------------------
def store_values(codes, scales, block):
    d = codes.shape[-1]
    return ref.values(f64(codes).reshape(-1, d), expo(scales).reshape(-1, scales.shape[-1]), block)


@pytest.mark.parametrize("fmt", ["f8", "i8"])
@pytest.mark.parametrize("dtype", NUMBERS)
@pytest.mark.parametrize("n,d,block", [(1, 1, 16), (7, 100, 32), (33, 96, 96), (20, 240, 80),
                                       (5, 513, 256), (64, 128, 128), (3, 250, 112)])
def test_cache_write_and_read(mm, fmt, dtype, n, d, block):
    import torch
    x = numbers(n, d, dtype, d)
    rows = 3 * n + 4
    codes, scales = mm.cache_new(rows, d, block=block, dtype=T(fmt))
    g = torch.Generator().manual_seed(1)
    for size in (torch.int32, torch.int64):
        slots = torch.randperm(rows, generator=g)[:n].to(size)
        skip = torch.zeros(n, dtype=torch.bool)
        if n > 3:
            slots[1], slots[2] = -1, rows
            skip[1:3] = True
        before = store_values(codes, scales, block)
        mm.cache_write(x, slots.cuda(), codes, scales, block=block)
        c, e = ref.encode(f64(x), fmt, block)
        want = before.copy()
        want[slots[~skip].long().numpy()] = ref.values(c, e, block)[~skip.numpy()]
        assert np.array_equal(store_values(codes, scales, block), want, equal_nan=True)
        ask = torch.cat([slots, torch.tensor([-5, rows, 0, rows - 1], dtype=size)])
        for out in NUMBERS:
            got = mm.cache_read(codes, scales, ask.cuda(), block=block, out_dtype=T(out))
            inside = ((ask >= 0) & (ask < rows)).numpy()
            exact = np.where(inside[:, None], want[np.where(inside, ask.numpy(), 0)], 0.0)
            exact = torch.from_numpy(exact).float().to(T(out))   # fp32 holds every value
            assert torch.equal(got.cpu(), exact)


@pytest.mark.parametrize("dtype", NUMBERS)
def test_cache_write_head_layouts(mm, dtype):
    """Heads as slices of a fused projection, heads first, one head repeated,
    odd starts."""
    import torch
    n, h, w = 19, 3, 80
    g = torch.Generator().manual_seed(2)
    wide = torch.randn(n, 1000, generator=g).to(T(dtype)).cuda()
    first = torch.randn(h, n, w, generator=g).to(T(dtype)).cuda()
    for x, block in ((wide[:, 24:24 + h * w].unflatten(1, (h, w)), 80),
                     (wide[:, 9:9 + h * w].unflatten(1, (h, w)), 128),
                     (first.transpose(0, 1), 80), (first.transpose(0, 1), 16),
                     (first[:1].transpose(0, 1).expand(n, h, w), 80)):
        codes, scales = mm.cache_new((4, 10), h * w, block=block, dtype=torch.int8)
        slots = torch.randperm(40, generator=g)[:n].cuda()
        mm.cache_write(x, slots, codes, scales, block=block)
        want = ref.values(*ref.encode(f64(x).reshape(n, -1), "i8", block), block)
        assert np.array_equal(store_values(codes, scales, block)[slots.cpu().numpy()], want)
    with pytest.raises(mm.EmeansError, match="EINVAL.*multiple of block"):
        codes, scales = mm.cache_new(40, h * w, block=32)
        mm.cache_write(first.transpose(0, 1), slots, codes, scales, block=32)


@pytest.mark.parametrize("fmt", ["f8", "i8"])
def test_cache_special_values(mm, fmt):
    import torch
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[0.0] * 40, [inf, 1.0, -inf, nan] + [0.5] * 36, [3.4e38] * 40,
                      [1e-45] * 40, [nan] * 40, [127.0, 448.0, 126.5, 2.5] + [0.0] * 36])
    codes, scales = mm.cache_new(6, 40, block=32, dtype=T(fmt))
    mm.cache_write(x.cuda(), torch.arange(6).cuda(), codes, scales, block=32)
    check_codes(codes, scales, ref.encode(x.double().numpy(), fmt, 32))
    got = mm.cache_read(codes, scales, torch.arange(6).cuda(), block=32, out_dtype=torch.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        want = ref.values(*ref.encode(x.double().numpy(), fmt, 32), 32).astype(np.float32)
    assert np.array_equal(f64(got), want, equal_nan=True)   # 2^128 rounds to infinity


@pytest.mark.parametrize("page", [1, 16, 24])
@pytest.mark.parametrize("fmt,out,d,block", [("f8", "bf16", 576, 64), ("i8", "f32", 100, 32),
                                             ("f8", "f16", 36, 16)])
def test_cache_read_pages(mm, page, fmt, out, d, block):
    """Lengths of zero and one, a page that ends inside, pages out of range,
    rows of the result past the last sequence."""
    import torch
    lengths = [0, 1, page, page + 1, 0, 3 * page - 1, 37, 0]
    most = max(-(-n // page) for n in lengths)
    pages = sum(-(-n // page) for n in lengths) + 2
    g = torch.Generator().manual_seed(page)
    codes, scales = mm.cache_new((pages, page), d, block=block, dtype=T(fmt))
    mm.cache_write(numbers(pages * page, d, "f32", 4), torch.arange(pages * page).cuda(), codes,
                   scales, block=block)
    order = torch.randperm(pages, generator=g).int()
    table = torch.full((len(lengths), most + 1), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(lengths):
        used = -(-n // page)
        table[i, :used] = order[at:at + used]
        at += used
    lost = table[6, 0].item()
    table[6, 0] = pages            # outside the store: zeros
    starts = np.concatenate([[0], np.cumsum(lengths)])
    total = int(starts[-1]) + 3
    all_rows = store_values(codes, scales, block)
    want = np.zeros((total, d))
    for i, n in enumerate(lengths):
        for p in range(n):
            pg = table[i, p // page].item()
            if 0 <= pg < pages:
                want[starts[i] + p] = all_rows[pg * page + p % page]
    assert lost < pages
    dev = (codes, scales, table.cuda()[:, :most], torch.from_numpy(starts).int().cuda(), total)
    got = mm.cache_read_pages(*dev, block=block, out_dtype=T(out))
    assert torch.equal(got.cpu(), torch.from_numpy(want).float().to(T(out)))
    room = torch.zeros(total, d + 5, dtype=T(out), device="cuda")
    mm.cache_read_pages(*dev, block=block, out=room[:, 3:3 + d])
    assert torch.equal(room[:, 3:3 + d].cpu(), got.cpu()) and torch.all(room[:, :3] == 0)


def test_cache_offsets_past_32_bits(mm):
    """Rows whose byte offset is above 2^32."""
    import torch
    rows, d = 1_200_000, 4096
    codes = torch.empty(rows, d, dtype=torch.int8, device="cuda")
    scales = torch.empty(rows, 32, dtype=torch.uint8, device="cuda")
    slots = torch.tensor([rows - 1, 0, rows // 2, 1_048_577], device="cuda")
    x = numbers(4, d, "bf16", 3)
    mm.cache_write(x, slots, codes, scales)
    want = ref.values(*ref.encode(f64(x), "i8"))
    got = mm.cache_read(codes, scales, slots, out_dtype=torch.float32)
    assert np.array_equal(f64(got), want)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    got = mm.cache_read_pages(codes.view(2, rows // 2, d), scales.view(2, rows // 2, 32), table,
                              starts, 1, out_dtype=torch.float32)
    assert np.array_equal(f64(got[0]), want[2])


# ---- streams, graphs, refusals ----------------------------------------------------
def test_on_another_stream(mm):
    import torch
    s = torch.cuda.Stream()
    x, w = numbers(40, 300, "f32", 1, 0.1), numbers(50, 300, "f32", 2, 0.1)
    s.wait_stream(torch.cuda.current_stream())
    xs, ws = x.clone().requires_grad_(), w.clone().requires_grad_()
    s.wait_stream(torch.cuda.current_stream())
    codes, scales = mm.block_encode(w, tiles=True, stream=s)
    y = mm.block_linear(xs, ws, stream=s)
    z = mm.block_linear(x, (codes, scales), stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, z) and torch.equal(y, mm.block_linear(x, w))


def test_another_stream_waits_for_nothing_else_and_its_gradient(mm):
    """Inputs that have to be copied are copied on the given stream, while the
    current one is busy; a gradient made late on the current stream is waited
    for."""
    import torch
    s = torch.cuda.Stream()
    x, w = numbers(300, 40, "f32", 1, 0.1), numbers(50, 300, "f32", 2, 0.1)
    g = numbers(40, 50, "f32", 3)
    want_x, want_w = x.t().clone().requires_grad_(), w.clone().requires_grad_()
    want = mm.block_linear(want_x, want_w)
    want.backward(g)
    codes = mm.block_encode(w, tiles=True)
    xs, ws = x.clone().requires_grad_(), w.clone().requires_grad_()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)            # the current stream, about 0.1 s
    y = mm.block_linear(xs.t(), ws, stream=s)
    z = mm.block_linear(x.t(), codes, stream=s)
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want) and torch.equal(z, want)
    torch.cuda._sleep(200_000_000)
    late = torch.zeros_like(g)
    late.add_(g)
    y.backward(late)
    torch.cuda.synchronize()
    assert torch.equal(ws.grad, want_w.grad) and torch.equal(xs.grad, want_x.grad.t())


@pytest.mark.parametrize("m", [1, 20, 150])
def test_graph_replays(mm, m):
    """Captured calls, replayed with other inputs between eager work."""
    import torch
    n, k, rows = 300, 512, 40
    w = mm.block_encode(numbers(n, k, "f32", 1, 0.1), tiles=True)
    x = numbers(m, k, "bf16", 2, 0.1)
    codes, scales = mm.cache_new(rows * m, n)
    slots = torch.arange(m, device="cuda") * rows
    out = torch.empty(m, n, dtype=torch.float32, device="cuda")

    def step():
        y = mm.block_linear(x, w)
        mm.cache_write(y, slots, codes, scales)
        mm.cache_read(codes, scales, slots, out=out)
        return y

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step()
    for i in range(4):
        x.copy_(numbers(m, k, "bf16", 10 + i, 0.1))
        out.zero_()
        g.replay()
        got = y.clone(), out.clone()
        torch.cuda.synchronize()
        want = step()
        assert torch.equal(got[0], want) and torch.equal(got[1], out)


def test_example_runs(mm):
    """examples/token_clusters.py: the projection learns, the clustering improves
    pass by pass, and 8-bit scores choose the exact search's centroid."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "token_clusters.py")
    spec = importlib.util.spec_from_file_location("token_clusters", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.main(d_in=512, d_out=200, tokens=6000, k=32, steps=25)
    assert got["losses"][-1] < 0.5 * got["losses"][0]
    assert got["obj"][-1] < got["obj"][0]
    assert got["agree"] > 0.9


def test_refusals(mm):
    import torch
    x = torch.zeros(8, 200, device="cuda")
    c, s = mm.block_encode(x)
    E = mm.EmeansError
    bad = [
        ("EDTYPE", lambda: mm.block_encode(x.double())),
        ("EINVAL", lambda: mm.block_encode(x.t())),
        ("EINVAL", lambda: mm.block_encode(x[0])),
        ("EINVAL", lambda: mm.block_encode(x[:1].expand(8, 200))),
        ("EINVAL", lambda: mm.block_encode(x, rows=False)),
        ("EDTYPE", lambda: mm.block_matmul(x, s, c, s)),
        ("EDTYPE", lambda: mm.block_matmul(c, s.float(), c, s)),
        ("EDTYPE", lambda: mm.block_matmul(c, s, c, s, out_dtype=torch.float64)),
        ("EINVAL", lambda: mm.block_matmul(c, s[:, :1], c, s)),
        ("EINVAL", lambda: mm.block_matmul(c, s[:1], c, s)),
        ("EINVAL", lambda: mm.block_matmul(c, s, c[:, :100], s[:, :1])),
        ("EINVAL", lambda: mm.block_matmul(c, s, c, s, out=torch.zeros(8, 9, device="cuda"))),
        ("EINVAL", lambda: mm.block_linear(x[:, :100], (c, s))),
        ("EINVAL", lambda: mm.block_linear(x, (c, s, c))),
        ("EINVAL", lambda: mm.block_linear(x.requires_grad_(), torch.zeros(4, 100, device="cuda"))),
        ("EDTYPE", lambda: mm.cache_new(4, 8, dtype=torch.uint8)),
    ]
    codes, scales = mm.cache_new((4, 8), 200)
    slots = torch.arange(8, device="cuda")
    x = x.detach()
    bad += [
        ("EINVAL", lambda: mm.cache_write(x[:, :100], slots, codes, scales)),
        ("EINVAL", lambda: mm.cache_write(x, slots[:5], codes, scales)),
        ("EDTYPE", lambda: mm.cache_write(x, slots.float(), codes, scales)),
        ("EINVAL", lambda: mm.cache_write(x, slots, codes, scales, block=64)),
        ("EINVAL", lambda: mm.cache_write(x, slots, codes[:, :, :100], scales)),
        ("EDTYPE", lambda: mm.cache_write(x, slots, codes.view(torch.uint8), scales)),
        ("EINVAL", lambda: mm.cache_read(codes, scales, slots.view(2, 4))),
        ("ENOTDEVICE", lambda: mm.cache_read(codes, scales, slots.cpu())),
        ("EDTYPE", lambda: mm.cache_read(codes, scales, slots, out_dtype=torch.int8)),
        ("EINVAL", lambda: mm.cache_read_pages(codes.view(32, 200), scales.view(32, 2),
                                               slots.int()[None], slots.int()[:2], 3)),
        ("EINVAL", lambda: mm.cache_read_pages(codes, scales, slots.int()[None], slots.int(), 3)),
        ("EDTYPE", lambda: mm.cache_read_pages(codes, scales, slots[None], slots.int()[:2], 3)),
    ]
    for i, (code, call) in enumerate(bad):
        with pytest.raises(E, match=code):
            call()
            pytest.fail(f"refusal {i} did not happen")
