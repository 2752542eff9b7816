"""Block codes at sizes that take several launches: 2^30 rows and more, whose
results repeat with a period that no launch's length is a multiple of."""
import numpy as np
import pytest

from test_gpu_block import f64, mm  # noqa: F401

pytestmark = pytest.mark.gpu

PERIOD, TIMES = 65537, 16400          # PERIOD * TIMES > 2^30
ROWS = PERIOD * TIMES


@pytest.fixture(autouse=True)
def room(mm):  # noqa: F811
    import gc
    import torch
    if torch.cuda.get_device_properties(0).total_memory < 200 << 30:
        pytest.skip("needs 200 GB of device memory")
    yield
    gc.collect()
    torch.cuda.empty_cache()


def repeated(base):
    import torch
    x = torch.empty((TIMES, *base.shape), dtype=base.dtype, device="cuda")
    x.copy_(base)
    return x.flatten(0, 1)


def all_equal(got, base, dim=0):
    """Whether every period of got along dim is base, byte for byte."""
    import torch
    size = base.shape[dim]
    for i in range(0, got.shape[dim], 512 * size):
        part = got.narrow(dim, i, min(512 * size, got.shape[dim] - i)).unflatten(dim, (-1, size))
        if not torch.all(part == base.unsqueeze(dim)):
            return False
    return True


def small(rows, d, seed, dtype):
    import torch
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, d, generator=g).to(dtype).cuda()


def test_encode_rows(mm):  # noqa: F811
    import torch
    base = small(PERIOD, 8, 1, torch.bfloat16)
    want = mm.block_encode(base)
    codes, scales = mm.block_encode(repeated(base))
    assert codes.shape == (ROWS, 8) and scales.shape == (ROWS, 1)
    assert all_equal(codes.view(torch.uint8), want[0].view(torch.uint8))
    assert all_equal(scales.view(torch.uint8), want[1].view(torch.uint8))


@pytest.mark.parametrize("tiles", [False, True])
def test_encode_long_rows(mm, tiles):  # noqa: F811
    import torch
    size = 128 * 513
    base = small(2, size, 2, torch.float32)
    x = torch.empty(2, 16353, size, device="cuda")
    x.copy_(base[:, None])
    x = x.flatten(1)
    assert x.shape[1] > 2 ** 30
    want = [t.view(torch.uint8) for t in mm.block_encode(base, cols=True, tiles=tiles)]
    got = [t.view(torch.uint8) for t in mm.block_encode(x, cols=True, tiles=tiles)]
    for g, w, dim in zip(got, want, (1, 1, 0, 0)):
        assert g.shape[dim] // w.shape[dim] == 16353 and all_equal(g, w, dim)


def test_cache_reads(mm):  # noqa: F811
    import torch
    codes, scales = mm.cache_new((1, PERIOD), 16, block=16, dtype=torch.int8)
    slots = torch.arange(PERIOD, device="cuda", dtype=torch.int32)
    mm.cache_write(small(PERIOD, 16, 3, torch.float32), slots, codes, scales, block=16)
    want = mm.cache_read(codes, scales, slots, block=16).view(torch.int16)
    got = mm.cache_read(codes, scales, repeated(slots), block=16)
    assert got.shape == (ROWS, 16) and all_equal(got.view(torch.int16), want)
    got.zero_()
    table = torch.zeros(TIMES, 1, dtype=torch.int32, device="cuda")
    starts = torch.arange(0, ROWS + 1, PERIOD, dtype=torch.int32, device="cuda")
    mm.cache_read_pages(codes, scales, table, starts, ROWS, block=16, out=got)
    assert all_equal(got.view(torch.int16), want)


def integers(rows, k, seed):
    """Integer values and their codes and scales, products exact in any order."""
    import torch
    rng = np.random.default_rng(seed)
    v, e = rng.integers(-8, 9, (rows, k)).astype(float), rng.integers(0, 2, (rows, 1))
    codes = torch.from_numpy(v).float().to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    return v * 2.0 ** e, codes, torch.from_numpy((e + 127).astype(np.uint8)).cuda()


@pytest.mark.parametrize("m,k,how", [(2, 16, "numbers"), (17, 17, "any pitch")])
def test_products_with_many_rows_of_b(mm, m, k, how):  # noqa: F811
    import torch
    vb, cb, sb = integers(PERIOD, k, 4)
    b, bs = repeated(cb).view(torch.float8_e4m3fn), repeated(sb)
    va, ca, sa = integers(m, k, 5)
    want = torch.from_numpy(va @ vb.T)
    if how == "numbers":
        x = torch.from_numpy(va).bfloat16().cuda()
        got = mm.block_linear(x, (b, bs), out_dtype=torch.float32)
    else:
        got = mm.block_matmul(ca.view(torch.float8_e4m3fn), sa, b, bs)
    assert got.shape == (m, ROWS)
    assert all_equal(got, want.to(got.dtype).cuda(), 1)


@pytest.mark.parametrize("m", [2, 17])
def test_products_with_many_tiles_of_b(mm, m):  # noqa: F811
    """Scales per tile of 128 rows: every launch starts at its own."""
    import torch
    k = 16
    _, cb, _ = integers(PERIOD, k, 6)
    vb = cb.view(torch.float8_e4m3fn).double().cpu().numpy()
    tiles = torch.randint(120, 135, (-(-ROWS // 128), 1), dtype=torch.uint8,
                          generator=torch.Generator().manual_seed(7)).cuda()
    va, ca, sa = integers(m, k, 8)
    want = torch.from_numpy(va @ vb.T).float().cuda()
    got = mm.block_matmul(ca.view(torch.float8_e4m3fn), sa,
                          repeated(cb).view(torch.float8_e4m3fn), tiles, out_dtype=torch.float32)
    for i in range(0, ROWS, PERIOD * 400):
        cols = torch.arange(i, min(i + PERIOD * 400, ROWS), device="cuda")
        factor = torch.exp2(tiles[:, 0].float() - 127)[cols // 128]
        part = (got[:, i:i + PERIOD * 400] / factor).unflatten(1, (-1, PERIOD))
        assert torch.all(part == want[:, None])
