"""Attention around the store at the far ends of what its calls take: rows nearly 2^24 values apart,
millions of places, thousands of heads, many sequences of nothing."""
import numpy as np
import pytest

import attention_ref as ref
from test_gpu_attend import inputs
from test_gpu_attention_store import check_decode, f64, gen, mm, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_far_apart(mm, dtype):  # noqa: F811
    """Offsets of a tile's rows up to 2^31 bytes and past 4 GiB in the tensor."""
    import torch
    far, lens = (1 << 24) - 8, [97, 40]
    q, k, v, do, starts, _ = inputs(lens, lens, 2, 1, 64, dtype, 3, 0, 0)
    room = torch.empty(sum(lens) * far, device="cuda", dtype=q.dtype)
    views = []
    for i, x in enumerate((q, k, v, do)):
        y = room.as_strided(x.shape, (far, 64, 1), 256 * i)
        y.copy_(x)
        views.append(y)
    results = []
    for a, b, c, d in ((q, k, v, do), views):
        leaves = [t.detach().requires_grad_() for t in (a, b, c)]
        o = mm.attend(*leaves, starts)
        results.append((o.detach(), *torch.autograd.grad(o, leaves, d)))
    assert all(torch.equal(x, y) for x, y in zip(*results))


def test_a_million_places(mm):  # noqa: F811
    """One sequence of 1.5 million places in pages of any order: attention, weights, eviction."""
    import torch
    n, page, w = 1_500_001, 16, 16
    pages = -(-n // page)
    rng = np.random.default_rng(1)
    table = rng.permutation(pages).astype(np.int32)[None]
    codes = [rng.integers(0, 0x60, (pages * page, 2 * w)).astype(np.uint8) for _ in range(2)]
    scales = [rng.integers(123, 127, (pages * page, 2)).astype(np.uint8) for _ in range(2)]
    stores = [(torch.from_numpy(c).cuda().view(torch.float8_e4m3fn).view(pages, page, -1),
               torch.from_numpy(s).cuda().view(torch.float8_e8m0fnu).view(pages, page, -1)) for c, s in zip(codes, scales)]
    q = 0.05 * randn(gen(2), 1, 4, w)
    weights = torch.zeros(1, pages * page, device="cuda")
    lens, tab = torch.tensor([n], device="cuda").int(), torch.from_numpy(table).cuda()
    got = mm.cache_attend(q, *stores, tab, lens, block=w, weights=weights)
    rows = (table[0].astype(np.int64)[:, None] * page + np.arange(page)).reshape(-1)
    kv = [ref.store_values(c[rows[:n]], s[rows[:n]], w, "f8").reshape(n, 2, w) for c, s in zip(codes, scales)]
    want, tol, wt, wtol = ref.decode(f64(q[0]), *kv, w ** -0.5, "f32")
    assert np.all(np.abs(f64(got[0]) - want) <= tol)
    assert np.all(np.abs(f64(weights[0])[:n] - wt) <= wtol) and not weights[0, n:].any()
    keep, recent = 400_000, 1000
    new, held, kept = mm.cache_evict(stores, tab, lens, weights, keep, recent=recent, block=w)
    h = weights[0, :n].cpu().numpy()
    order = np.argsort(-h[:n - recent], kind="stable")[:keep - recent]
    stay = np.concatenate([np.sort(order), np.arange(n - recent, n)])
    assert new.tolist() == [keep] and np.array_equal(kept[0].cpu().numpy(), stay)
    assert np.array_equal(held[0, :keep].cpu().numpy(), h[stay]) and not held[0, keep:].any()
    for c, s, (gc, gs) in zip(codes, scales, stores):
        for host, dev in ((c, gc), (s, gs)):
            host[rows[:keep]] = host[rows[stay]]
            assert np.array_equal(dev.view(torch.uint8).flatten(0, 1).cpu().numpy(), host)


@pytest.mark.parametrize("hq,hk,weights", [(1024, 1, True), (1024, 64, True), (1040, 8, False), (4096, 2, False)])
def test_many_heads_over_the_store(mm, hq, hk, weights):  # noqa: F811
    check_decode(mm, np.random.default_rng(hq + hk), [33, 0, 600], hq, hk, 16, 16, 16, "f8", "bf16", weights)


def test_many_heads_and_sequences_of_nothing(mm):  # noqa: F811
    import torch
    # 20000 sequences of which two have rows, 160 heads
    q, k, v, do, _, _ = inputs([70, 3], [70, 3], 160, 32, 16, "f16", 5, 0, 0)
    ends = torch.zeros(20001, device="cuda", dtype=torch.int32)
    ends[7001:] = 70
    ends[15001:] = 73
    two = torch.tensor([0, 70, 73], device="cuda").int()
    results = []
    for starts in (two, ends):
        leaves = [t.clone().requires_grad_() for t in (q, k, v)]
        o = mm.attend(*leaves, starts)
        results.append((o.detach(), *torch.autograd.grad(o, leaves, do)))
    # keys' sums may be cut differently, as that goes by the number of sequences
    for i, (a, b) in enumerate(zip(*results)):
        assert torch.equal(a, b) if i < 2 else bool(((a.float() - b.float()).abs() <= 2.0 ** -10 * a.float().abs() + 2.0 ** -9).all())
    # the same for tokens one by one: 20000 sequences of a place or none
    from test_gpu_attention_calls import small_store
    store, n = small_store(mm), 20000
    lens = (torch.arange(n, device="cuda") % 2).int()
    table = (torch.arange(n, device="cuda") % 3).int()[:, None]
    x = randn(gen(6), n, 2, 64)
    got = mm.cache_attend(x, store, store, table, lens, block=64)
    rows = mm.cache_read(*store, table[:, 0].long() * 16, block=64, out_dtype=torch.float32).view(n, 2, 64)
    want = rows * lens[:, None, None]
    assert bool(((got - want).abs() <= 2.0 ** -22 * want.abs()).all())
    y = mm.norm_rotate(x, x[:, :1], *(torch.ones(64, device="cuda"),) * 2, -torch.arange(n, device="cuda"), mm.rotary_freqs(64))[0]
    want, size = ref.rotate(f64(x[-50:]), np.ones(64), -np.arange(n)[-50:], f64(mm.rotary_freqs(64)))
    assert np.all(np.abs(f64(y[-50:]) - want) <= ref.rotate_tol(want, size, "f32"))
