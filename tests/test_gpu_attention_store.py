"""Norms with rotation, attention over the paged store and eviction from it,
against their definitions in 64 bits."""
import numpy as np
import pytest

import attention_ref as ref

pytestmark = pytest.mark.gpu

NUMBERS = ["bf16", "f16", "f32"]


@pytest.fixture(scope="module")
def mm():
    import torch
    assert torch.cuda.is_available(), "these tests need a GPU"
    import mini_means_amd
    return mini_means_amd


def T(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def f64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    import torch
    return torch.randn(*shape, device="cuda", generator=g)


# ---- norms and rotation ------------------------------------------------------

def rotate_inputs(n, hq, hk, w, turned, dtype, seed, wtype=None):
    import torch
    g = gen(seed)
    wide = (randn(g, n, (hq + 2 * hk) * w + 8) * torch.exp(randn(g, n, 1))).to(T(dtype))
    q = wide[:, 8:8 + hq * w].unflatten(1, (hq, w))
    k = wide[:, 8 + hq * w:8 + (hq + hk) * w].unflatten(1, (hk, w))
    gq, gk = (1 + 0.3 * randn(g, 2, w)).to(T(wtype or dtype)).unbind(0)
    pos = torch.randint(0, 1 << 20, (n,), device="cuda", generator=g)
    if n:
        pos[0] = 2 ** 31 - 1
    return q, k, gq, gk, pos


SHAPES = [(1, 1, 1, 8, 8), (5, 32, 8, 128, 128), (3, 3, 1, 64, 64), (7, 2, 1, 80, 40), (2, 4, 4, 96, 48),
          (9, 3, 2, 112, 112), (2, 5, 3, 128, 0), (3, 2, 1, 256, 256), (2, 2, 2, 256, 24), (4, 7, 1, 72, 72),
          (5, 1, 2, 24, 8), (4100, 3, 1, 64, 32)]


@pytest.mark.parametrize("n,hq,hk,w,turned", SHAPES)
@pytest.mark.parametrize("dtype", NUMBERS)
def test_norm_rotate(mm, n, hq, hk, w, turned, dtype):
    q, k, gq, gk, pos = rotate_inputs(n, hq, hk, w, turned, dtype, n + w)
    freqs = mm.rotary_freqs(turned)
    got = mm.norm_rotate(q, k, gq, gk, pos, freqs)
    for x, gain, y in ((q, gq, got[0]), (k, gk, got[1])):
        want, size = ref.rotate(f64(x), f64(gain), pos.cpu().numpy(), f64(freqs))
        tol = ref.rotate_tol(want, size, dtype)
        assert y.dtype == x.dtype and y.is_contiguous() and y.shape == x.shape
        assert np.all(np.abs(f64(y) - want) <= tol)


@pytest.mark.parametrize("n,hq,hk,w,turned", SHAPES)
@pytest.mark.parametrize("dtype,wtype", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_norm_rotate_gradients(mm, n, hq, hk, w, turned, dtype, wtype):
    import torch
    q, k, gq, gk, pos = rotate_inputs(n, hq, hk, w, turned, dtype, n + w + 1, wtype)
    g = gen(5)
    dq = randn(g, hq, n, w).to(T(dtype)).transpose(0, 1)       # heads outside, as a caller may have it
    dk = randn(g, n, hk, w).to(T(dtype))
    freqs = mm.rotary_freqs(turned)
    leaves = [t.detach().requires_grad_() for t in (q, k, gq, gk)]
    y = mm.norm_rotate(*leaves, pos.int(), freqs)
    plain = mm.norm_rotate(q, k, gq, gk, pos.int(), freqs)
    assert all(torch.equal(a, b) for a, b in zip(y, plain))
    got = torch.autograd.grad(y, leaves, (dq, dk))
    again = torch.autograd.grad(mm.norm_rotate(*leaves, pos, freqs), leaves, (dq, dk))
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    for x, gain, dy, dx, dg in ((q, gq, dq, got[0], got[2]), (k, gk, dk, got[1], got[3])):
        wx, tx, wg, tg = ref.rotate_grad(f64(x), f64(gain), pos.cpu().numpy(), f64(freqs), f64(dy))
        tx = tx + ref.HALF_ULP[dtype] * 1.01 * np.abs(wx) + ref.TINY[dtype]
        tg = tg + ref.HALF_ULP[wtype] * 1.01 * np.abs(wg) + ref.TINY[wtype]
        assert np.all(np.abs(f64(dx) - wx) <= tx) and np.all(np.abs(f64(dg) - wg) <= tg)


def test_norm_rotate_gradient_against_differences(mm):
    import torch
    q, k, gq, gk, pos = rotate_inputs(3, 2, 1, 16, 16, "f32", 3)
    freqs = mm.rotary_freqs(16)
    cq, ck = randn(gen(8), 3, 2, 16), randn(gen(9), 3, 1, 16)

    def loss(*a):
        y = mm.norm_rotate(*a, pos, freqs)
        return (y[0] * cq).sum() + (y[1] * ck).sum()

    leaves = [t.detach().clone().requires_grad_() for t in (q, k, gq, gk)]
    grads = torch.autograd.grad(loss(*leaves), leaves)
    for i, x in enumerate(leaves):
        way = randn(gen(20 + i), *x.shape)
        way /= way.norm()
        step = 2.0 ** -7 * float(x.detach().norm())
        ends = []
        for sign in (1, -1):
            a = [t.detach() for t in leaves]
            a[i] = x.detach() + sign * step * way
            ends.append(float(loss(*a)))
        # the third derivative's part is step^2 relative; the losses' rounding 2^-20 of their size
        slope = (ends[0] - ends[1]) / (2 * step)
        want = float((grads[i] * way).sum())
        size = float(cq.abs().sum() + ck.abs().sum())
        assert abs(slope - want) <= 2.0 ** -10 * size / float(x.detach().norm()) + 2.0 ** -20 * size / step


def test_norm_rotate_of_nothing_zeros_and_broadcast_heads(mm):
    import torch
    freqs = mm.rotary_freqs(64)
    gain = torch.ones(64, device="cuda", requires_grad=True)
    q = torch.zeros(0, 4, 64, device="cuda", requires_grad=True)
    y = mm.norm_rotate(q, q, gain, gain, torch.zeros(0, device="cuda", dtype=torch.int64), freqs)
    d = torch.autograd.grad(y, (q, gain), (q.detach(), q.detach()))
    assert y[0].shape == (0, 4, 64) and not d[1].any()
    pos = torch.arange(3, device="cuda")
    zero = torch.zeros(3, 2, 64, device="cuda", requires_grad=True)
    y = mm.norm_rotate(zero, zero, gain, gain, pos, freqs)
    assert not y[0].any()
    assert all(torch.isfinite(t).all() for t in torch.autograd.grad(y, (zero, gain), (zero + 1, zero + 1)))
    one = randn(gen(1), 3, 1, 64).requires_grad_()      # the gradient of a head that is used four times
    y = mm.norm_rotate(one.expand(3, 4, 64), one, gain, gain, pos, freqs)
    part = torch.autograd.grad(y, one, (torch.ones(3, 4, 64, device="cuda"),
                                        torch.zeros(3, 1, 64, device="cuda")))[0]
    y = mm.norm_rotate(one, one, gain, gain, pos, freqs)
    single = torch.autograd.grad(y, one, (torch.ones_like(one), torch.zeros_like(one)))[0]
    assert torch.allclose(part, 4 * single, rtol=1e-5, atol=1e-6)


# ---- one new token -----------------------------------------------------------

def make_store(rng, pages, page, d, block, fmt, poison=True):
    """Stores whose every row is a NaN, to be overwritten where a sequence has rows."""
    nb = -(-d // block)
    codes = np.full((pages * page, d), 0x7F if fmt == "f8" else 0x80, np.uint8)
    scales = np.full((pages * page, nb), 255, np.uint8)
    return codes, scales


def fill(rng, store, rows, fmt):
    codes, scales = store
    c = rng.integers(0, 256, (len(rows), codes.shape[1])).astype(np.uint8)
    if fmt == "f8":
        c[(c & 0x7F) == 0x7F] = 0x30
        mid = 120
    else:
        c[c == 0x80] = 0x11
        mid = 121
    codes[rows] = c
    scales[rows] = rng.integers(mid - 3, mid + 1, (len(rows), scales.shape[1]))


def to_gpu(store, pages, page, fmt):
    import torch
    c = torch.from_numpy(store[0]).cuda().view(torch.int8 if fmt == "i8" else torch.float8_e4m3fn)
    s = torch.from_numpy(store[1]).cuda().view(torch.float8_e8m0fnu)
    return c.view(pages, page, -1), s.view(pages, page, -1)


def lay_out(rng, lengths, page, columns=None):
    """A page table of pages in any order, and each sequence's rows."""
    used = [-(-n // page) for n in lengths]
    columns = columns or max(max(used), 1)
    pages = sum(used) + 3
    order = rng.permutation(pages)
    table, at = np.full((len(lengths), columns), -1, np.int32), 0
    rows = []
    for s, (n, u) in enumerate(zip(lengths, used)):
        table[s, :u] = order[at:at + u]
        at += u
        p = np.arange(n)
        rows.append(table[s, p // page].astype(np.int64) * page + p % page)
    return pages, table, rows


def check_decode(mm, rng, lengths, hq, hk, w, page, block, fmt, dtype, weights=False, scale=None,
                 given=None, columns=None, gaps=()):
    import torch
    pages, table, rows = lay_out(rng, lengths, page, columns)
    d = hk * w
    k, v = (make_store(rng, pages, page, d, block, fmt) for _ in range(2))
    for r in rows:
        fill(rng, k, r, fmt)
        fill(rng, v, r, fmt)
    for s, c, value in gaps:                     # pages that are not in the store
        table[s, c] = value
    rows = [r[[table[s, i // page] in range(pages) for i in range(len(r))]] for s, r in enumerate(rows)]
    q = torch.from_numpy(rng.normal(size=(len(lengths), hq + 2, w + 16)) * 0.5).cuda().to(T(dtype))
    q = q[:, 1:hq + 1, 8:w + 8]
    total = torch.from_numpy(rng.random((len(lengths), table.shape[1] * page + 3)).astype(np.float32)).cuda()
    before = total.clone()
    used = total[:, :table.shape[1] * page] if weights else None
    lens = torch.tensor(lengths if given is None else given, dtype=torch.int32, device="cuda")
    call = lambda: mm.cache_attend(q, to_gpu(k, pages, page, fmt), to_gpu(v, pages, page, fmt),  # noqa: E731
                                   torch.from_numpy(table).cuda(), lens, block=block, scale=scale,
                                   weights=used)
    got = call()
    assert got.dtype == q.dtype and got.shape == q.shape and got.is_contiguous()
    added = f64(total)
    for s, r in enumerate(rows):
        kv, vv = (ref.store_values(x[0][r], x[1][r], block, fmt).reshape(-1, hk, w) for x in (k, v))
        out, tol, wt, wtol = ref.decode(f64(q[s]), kv, vv, w ** -0.5 if scale is None else scale, dtype)
        off = np.abs(f64(got[s]) - out)
        assert bool(np.all(off <= tol)), (s, off.max())
        if weights:
            b = f64(before[s])
            want, wide = b.copy(), np.full(len(b), 0.0)
            place = {int(x): i for i, x in enumerate(r)}
            for p in range(min(len(b), lengths[s])):
                if p // page < table.shape[1] and 0 <= table[s, p // page] < pages:
                    i = place[int(table[s, p // page]) * page + p % page]
                    want[p] += wt[i]
                    wide[p] = wtol[i] + ref.SUM_ULP * want[p]
            assert np.all(np.abs(added[s] - want) <= wide)
    if not weights:
        assert torch.equal(total, before)
        assert torch.equal(got, call())          # the same call, the same bits
    return got


LENGTHS = [0, 1, 31, 32, 33, 127, 128, 129, 200]


@pytest.mark.parametrize("hq,hk,w,page,block", [
    (8, 2, 128, 16, 128), (4, 4, 64, 1, 64), (6, 2, 96, 24, 96), (5, 1, 80, 7, 16), (16, 16, 96, 16, 96),
    (3, 3, 112, 64, 128), (32, 1, 128, 16, 64), (17, 1, 16, 16, 16), (40, 2, 48, 16, 256), (2, 1, 32, 300, 32)])
@pytest.mark.parametrize("fmt,dtype", [("f8", "bf16"), ("f8", "f32"), ("i8", "f16"), ("i8", "bf16")])
def test_cache_attend(mm, hq, hk, w, page, block, fmt, dtype):
    rng = np.random.default_rng(hq + w)
    check_decode(mm, rng, LENGTHS, hq, hk, w, page, block, fmt, dtype)
    check_decode(mm, rng, LENGTHS, hq, hk, w, page, block, fmt, dtype, weights=True)


@pytest.mark.parametrize("fmt,dtype", [("f8", "bf16"), ("f8", "f16"), ("i8", "f32")])
@pytest.mark.parametrize("weights", [False, True])
def test_cache_attend_long_sequences_are_split_and_joined(mm, fmt, dtype, weights):
    rng = np.random.default_rng(4)
    check_decode(mm, rng, [5000, 0, 1, 4097, 2049], 8, 2, 128, 16, 128, fmt, dtype, weights)
    check_decode(mm, rng, [20011], 3, 1, 64, 64, 64, fmt, dtype, weights)
    check_decode(mm, rng, [700] * 70, 8, 8, 64, 16, 64, fmt, dtype, weights)


@pytest.mark.parametrize("weights", [False, True])
def test_cache_attend_pages_outside_the_store_and_lengths_outside_the_table(mm, weights):
    rng = np.random.default_rng(6)
    gaps = [(0, 0, -1), (0, 3, 1 << 30), (1, 1, -7), (3, 0, 9999)]
    check_decode(mm, rng, [150, 40, 9, 16, 300], 4, 2, 64, 16, 64, "f8", "bf16", weights, gaps=gaps)
    check_decode(mm, rng, [150, 40, 9, 16, 300], 4, 2, 64, 16, 64, "i8", "f16", weights, gaps=gaps)
    # negative lengths are none, those past the table's places are all of them
    check_decode(mm, rng, [0, 64, 64], 4, 2, 64, 16, 64, "f8", "f32", weights, given=[-5, 1 << 30, 65],
                 columns=4)


def test_cache_attend_large_scores_and_scales(mm):
    """Scores of some hundreds: all weight on few places; no overflow on the way."""
    rng = np.random.default_rng(7)
    check_decode(mm, rng, [300, 33], 4, 2, 64, 16, 64, "f8", "f32", True, scale=3.0)
    check_decode(mm, rng, [300, 33], 4, 2, 64, 16, 64, "f8", "f32", True, scale=-1.5)
    check_decode(mm, rng, [300, 33], 4, 2, 64, 16, 64, "i8", "f32", True, scale=0.0)


def test_cache_attend_nan_rows_of_a_sequence_show_in_it_alone(mm):
    import torch
    rng = np.random.default_rng(8)
    pages, table, rows = lay_out(rng, [70, 70, 70], 16)
    k, v = (make_store(rng, pages, 16, 128, 64, "f8") for _ in range(2))
    for r in rows:
        fill(rng, k, r, "f8")
        fill(rng, v, r, "f8")
    k[0][rows[0][40], 3] = 0x7F                 # a key of head 0
    v[1][rows[1][69], 1] = 255                  # a value of head 1
    q = torch.randn(3, 4, 64, device="cuda")
    got = mm.cache_attend(q, to_gpu(k, pages, 16, "f8"), to_gpu(v, pages, 16, "f8"),
                          torch.from_numpy(table).cuda(), torch.tensor([70] * 3, device="cuda").int(),
                          block=64)
    bad = torch.isnan(got).all(2).cpu().numpy()
    assert np.array_equal(bad, [[True, True, False, False], [False, False, True, True], [False] * 4])
    assert not torch.isnan(got[~torch.isnan(got).all(2)]).any()


def test_cache_attend_and_evict_past_4_gib(mm):
    """Rows whose bytes lie past 32 bits of offset."""
    import torch
    page, d, pages = 64, 1024, 70000              # 4.6 GB of codes
    keys, values = (mm.cache_new((pages, page), d) for _ in range(2))
    n = 300
    table = (pages - 1 - torch.arange(5, dtype=torch.int32, device="cuda"))[None]
    p = torch.arange(n, device="cuda")
    slots = table[0].long()[p // page] * page + p % page
    x, y = (torch.randn(n, d, device="cuda", generator=gen(i)) for i in range(2))
    mm.cache_write(x, slots, *keys)
    mm.cache_write(y, slots, *values)
    q = torch.randn(1, 8, 128, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    weights = torch.zeros(1, 5 * page, device="cuda")
    kv, vv = (f64(mm.cache_read(*s, slots, out_dtype=torch.float32)).reshape(n, 8, 128) for s in (keys, values))
    got = mm.cache_attend(q, keys, values, table, lens, weights=weights)
    out, tol, wt, wtol = ref.decode(f64(q[0]), kv, vv, 128 ** -0.5, "f32")
    assert np.all(np.abs(f64(got[0]) - out) <= tol)
    _, _, kept = mm.cache_evict((keys, values), table, lens, weights, 100, recent=10)
    stay = ref.evict(f64(weights[0]), n, 100, 10)
    assert kept[0].tolist() == stay
    now = f64(mm.cache_read(*keys, slots[:100], out_dtype=torch.float32)).reshape(100, 8, 128)
    assert np.array_equal(now, kv[stay])


# ---- eviction ----------------------------------------------------------------

def check_evict(mm, rng, lengths, keep, recent, d, page, block, fmt, stores=2, weights=None, columns=None):
    import torch
    pages, table, rows = lay_out(rng, lengths, page, columns)
    cap = table.shape[1] * page
    host = []
    for i in range(stores):
        codes = rng.integers(0, 256, (pages * page, d + 16 * i)).astype(np.uint8)
        scales = rng.integers(0, 256, (pages * page, -(-(d + 16 * i) // block))).astype(np.uint8)
        host.append((codes, scales))
    if weights is None:
        weights = rng.random((len(lengths), cap)).astype(np.float32)
    wide = torch.from_numpy(np.concatenate([weights, weights], 1)).cuda()[:, :cap]
    gpu = [to_gpu(s, pages, page, fmt) for s in host]
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    new, new_w, kept = mm.cache_evict(gpu, torch.from_numpy(table).cuda(), lens, wide, keep, recent=recent,
                                      block=block)
    assert torch.equal(lens.cpu(), torch.tensor(lengths, dtype=torch.int32))
    for s, n in enumerate(lengths):
        stay = ref.evict(weights[s].astype(np.float64), n, keep, recent)
        assert int(new[s]) == len(stay)
        assert kept[s].tolist() == stay + [-1] * (keep - len(stay))
        want = np.zeros(cap, np.float32)
        want[:len(stay)] = weights[s][stay]
        assert np.array_equal(new_w[s].cpu().numpy(), want, equal_nan=True)
        for codes, scales in host:
            codes[rows[s][:len(stay)]] = codes[rows[s][stay]]
            scales[rows[s][:len(stay)]] = scales[rows[s][stay]]
    for (codes, scales), (c, s) in zip(host, gpu):
        assert np.array_equal(c.view(torch.uint8).flatten(0, 1).cpu().numpy(), codes)
        assert np.array_equal(s.view(torch.uint8).flatten(0, 1).cpu().numpy(), scales)


@pytest.mark.parametrize("keep,recent", [(0, 0), (1, 0), (1, 1), (64, 64), (100, 7), (256, 32), (999, 0), (5000, 9)])
@pytest.mark.parametrize("d,page,block,fmt", [(256, 16, 64, "i8"), (1024, 16, 128, "f8"), (100, 1, 16, "f8"),
                                              (36, 24, 32, "i8"), (1001, 7, 256, "i8")])
def test_cache_evict(mm, keep, recent, d, page, block, fmt):
    rng = np.random.default_rng(keep + d)
    check_evict(mm, rng, [0, 1, 63, 64, 65, 100, 101, 700, 1500], keep, recent, d, page, block, fmt)


def test_cache_evict_of_weights_that_are_equal_or_no_numbers(mm):
    rng = np.random.default_rng(2)
    lengths = [1200, 1200, 1200, 1200, 1200]
    w = np.ones((5, 1200), np.float32)
    w[1] = rng.integers(0, 3, 1200)
    w[2] = rng.choice(np.array([0.0, -0.0, 1e-45, -1.0], np.float32), 1200)
    w[3] = rng.choice(np.array([np.nan, -np.inf, np.inf, 3.0, -2.0], np.float32), 1200)
    w[4] = np.nan
    for keep, recent in ((300, 50), (1199, 3), (7, 0)):
        check_evict(mm, rng, lengths, keep, recent, 64, 16, 64, "f8", weights=w)


@pytest.mark.parametrize("stores", [1, 3, 4])
def test_cache_evict_of_several_stores_and_long_sequences(mm, stores):
    rng = np.random.default_rng(3)
    check_evict(mm, rng, [9000, 0, 4097], 3000, 100, 128, 16, 128, "i8", stores, columns=600)


def test_refusals_of_the_store_calls(mm):
    """What a caller can get wrong with tensors on the GPU: refused before any device work."""
    import torch
    keys, values = (mm.cache_new((4, 16), 128, block=64) for _ in range(2))
    other = mm.cache_new((4, 8), 128, block=64)
    i8 = mm.cache_new((4, 16), 128, block=64, dtype=torch.int8)
    q = torch.zeros(2, 4, 64, device="cuda")
    table, lens = torch.zeros(2, 3, device="cuda").int(), torch.zeros(2, device="cuda").int()
    w = torch.zeros(2, 48, device="cuda")
    attend = lambda q=q, k=keys, v=values, t=table, n=lens, **kw: mm.cache_attend(q, k, v, t, n, block=64, **kw)  # noqa: E731
    evict = lambda s=(keys, values), t=table, n=lens, w=w, keep=5, **kw: mm.cache_evict(s, t, n, w, keep, block=64, **kw)  # noqa: E731
    attend(weights=w)
    evict()
    for call, word in (
            (lambda: attend(q=q.double()), "EDTYPE"), (lambda: attend(q=q[:, :3]), "EINVAL"),
            (lambda: attend(q=q[:, :, :40]), "EINVAL"), (lambda: attend(q=q[:1]), "EINVAL"),
            (lambda: attend(q=q.transpose(1, 2)), "EINVAL"), (lambda: attend(v=other), "EINVAL"),
            (lambda: attend(v=i8), "EINVAL"), (lambda: attend(v=values[0]), "EINVAL"),
            (lambda: attend(t=table.long()), "EDTYPE"), (lambda: attend(n=lens.long()), "EDTYPE"),
            (lambda: attend(n=lens[:1]), "EINVAL"), (lambda: attend(weights=w[:, :40]), "EINVAL"),
            (lambda: attend(weights=w.half()), "EDTYPE"), (lambda: attend(weights=w[:1].expand(2, 48)), "EINVAL"),
            (lambda: attend(scale=float("nan")), "EINVAL"), (lambda: attend(k=keys[0].cpu()), "EINVAL"),
            (lambda: attend(n=lens.cpu()), "ENOTDEVICE"),
            (lambda: evict(s=()), "EINVAL"), (lambda: evict(s=(keys, keys)), "EINVAL"),
            (lambda: evict(s=(keys, other)), "EINVAL"), (lambda: evict(w=w[:, 1:]), "EINVAL"),
            (lambda: evict(keep=-1), "EINVAL"), (lambda: evict(keep=3, recent=4), "EINVAL"),
            (lambda: evict(n=lens.cpu()), "ENOTDEVICE")):
        with pytest.raises(mm.EmeansError, match=word):
            call()


# ---- streams, graphs ---------------------------------------------------------

def test_on_a_given_stream_and_in_graphs(mm):
    """Two captured graphs over one store, replayed in turn with eager calls between,
    against eager results; and the calls on a stream of their own."""
    import torch
    rng = np.random.default_rng(1)
    pages, table, rows = lay_out(rng, [900, 50, 0], 16)
    k, v = (make_store(rng, pages, 16, 256, 64, "f8") for _ in range(2))
    for r in rows:
        fill(rng, k, r, "f8")
        fill(rng, v, r, "f8")
    keys, values = to_gpu(k, pages, 16, "f8"), to_gpu(v, pages, 16, "f8")
    table, lens = torch.from_numpy(table).cuda(), torch.tensor([900, 50, 0], device="cuda").int()
    freqs, gain = mm.rotary_freqs(64), torch.ones(64, device="cuda")
    pos = torch.arange(3, device="cuda")
    places = table.shape[1] * 16
    x = [torch.randn(3, 8, 64, device="cuda").bfloat16() for _ in range(2)]
    w = [torch.zeros(3, places, device="cuda") for _ in range(2)]

    def step(i, stream=None):
        q, _ = mm.norm_rotate(x[i], x[i][:, :4], gain, gain, pos, freqs, stream=stream)
        return mm.cache_attend(q, keys, values, table, lens, block=64, weights=w[i], stream=stream)

    want = [step(i) for i in range(2)]
    one = [t.clone() for t in w]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(0, side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[0])
    for t in w:
        t.zero_()
    graphs, outs = [], []
    side.wait_stream(torch.cuda.current_stream())
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(i))
        graphs.append(graph)
    for t in w:
        t.zero_()
    for turn in range(4):
        for i in (0, 1):
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        for o in outs:
            o.zero_()
        for i in range(2):
            # turn + 1 additions of the same numbers, each rounded once
            assert torch.allclose(w[i], one[i] * (turn + 1), rtol=2.0 ** -20, atol=0)
        other = mm.cache_attend(x[0], keys, values, table, lens, block=64)
        assert torch.isfinite(other).all()
