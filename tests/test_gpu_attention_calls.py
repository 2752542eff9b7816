"""Attention around the store: calls that the documentation allows, and what is refused."""
import numpy as np
import pytest

import attention_ref as ref
from test_gpu_attend import inputs
from test_gpu_attention_store import T, f64, gen, mm, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,heads", [(1, 2), (1, 1), (0, 2), (3, 1), (2, 2)])
def test_rows_and_heads_at_any_distance_where_there_is_one(mm, rows, heads, dtype):  # noqa: F811
    """torch calls a tensor contiguous whatever the distance of what there is one of: rows of a prompt of
    one token out of an odd buffer, a single head, a gradient like these."""
    import torch
    base = randn(gen(rows + heads), 8, 131 * 3).to(T(dtype))

    def view(i):
        return base[2:2 + rows, 131 * i:131 * i + 64 * heads].unflatten(1, (heads, 64))

    def apart(x):                  # the same values, heads 67 apart
        room = torch.zeros(x.shape[0], heads, 67, device="cuda", dtype=x.dtype)
        room[:, :, :64] = x
        return room[:, :, :64]

    def far(x):                    # rows 2^24 values apart, as a slice across a large buffer is
        return x.as_strided(x.shape, (1 << 24, 64, 1)) if x.shape[0] == 1 and x.is_contiguous() else x

    starts = torch.tensor([0, rows], device="cuda").int()
    plain = [view(i).clone(memory_format=torch.contiguous_format) for i in range(3)]
    do = randn(gen(9), rows, heads, 64).to(T(dtype))
    results = []
    for make, of in ((lambda x: x, plain), (lambda x: x, [view(i) for i in range(3)]), (apart, plain), (far, plain)):
        leaves = [make(x.detach()).requires_grad_() for x in of]
        o = mm.attend(*leaves, starts)
        results.append((o, *torch.autograd.grad(o, leaves, make(do))))
        with torch.no_grad():
            assert torch.equal(mm.attend(*leaves, starts), o)
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], r))


def test_the_same_starts_for_keys_of_a_longer_buffer(mm):  # noqa: F811
    """k_starts given, and the same tensor as starts: keys behind the last sequence are not read."""
    import torch
    q, k, v, _, starts, _ = inputs([30, 9], [30, 9], 2, 1, 64, "bf16", 4, 0, 0)
    pad = torch.full((7, 1, 64), float("nan"), device="cuda", dtype=k.dtype)
    got = mm.attend(q, torch.cat([k, pad]), torch.cat([v, pad]), starts, k_starts=starts)
    assert torch.equal(got, mm.attend(q, k, v, starts))
    with pytest.raises(mm.EmeansError, match="EINVAL"):
        mm.attend(q, torch.cat([k, pad]), torch.cat([v, pad]), starts)


def small_store(mm, d=128, block=64):  # noqa: F811
    import torch
    store = mm.cache_new((3, 16), d, block=block)
    mm.cache_write(randn(gen(1), 48, d), torch.arange(48, device="cuda"), *store, block=block)
    return store


def test_what_has_no_gradient_is_refused_for_inputs_that_ask_for_one(mm):  # noqa: F811
    import torch
    import torch.autograd.forward_ad as fwd
    store, table = small_store(mm), torch.arange(3, device="cuda").int().view(1, 3)
    lens, q = torch.tensor([40], device="cuda").int(), randn(gen(2), 1, 4, 64)
    w = torch.zeros(1, 48, device="cuda")
    call = lambda q, w=None: mm.cache_attend(q, store, store, table, lens, block=64, weights=w)  # noqa: E731
    want = call(q)
    leaf = q.clone().requires_grad_()
    with pytest.raises(mm.EmeansError, match="EINVAL.*gradient"):
        call(leaf)
    with pytest.raises(mm.EmeansError, match="EINVAL.*gradient"):
        call(q, w.clone().requires_grad_())
    with torch.no_grad():
        assert torch.equal(call(leaf), want) and torch.equal(call(leaf, w), want)
    assert torch.equal(call(leaf.detach()), want)
    with fwd.dual_level(), pytest.raises(mm.EmeansError, match="forward-mode"):
        call(fwd.make_dual(q, torch.ones_like(q)))
    evict = lambda w: mm.cache_evict([store], table, lens, w, 8, block=64)  # noqa: E731
    with pytest.raises(mm.EmeansError, match="EINVAL.*gradient"):
        evict(w.clone().requires_grad_())
    with fwd.dual_level(), pytest.raises(mm.EmeansError, match="forward-mode"):
        evict(fwd.make_dual(w, torch.ones_like(w)))
    # the angles' frequencies have none either
    x, gain, pos, f = q.expand(3, 4, 64), torch.ones(64, device="cuda"), torch.arange(3, device="cuda"), mm.rotary_freqs(64)
    with pytest.raises(mm.EmeansError, match="EINVAL.*gradient"):
        mm.norm_rotate(x, x, gain, gain, pos, f.clone().requires_grad_())
    with torch.no_grad():
        mm.norm_rotate(x, x, gain, gain, pos, f.clone().requires_grad_())
    with fwd.dual_level(), pytest.raises(mm.EmeansError, match="forward-mode"):
        mm.norm_rotate(x, x, gain, gain, pos, fwd.make_dual(f, torch.ones_like(f)))


def test_a_generous_budget_takes_no_memory(mm):  # noqa: F811
    """keep far over what the table holds: beside the results no list of that length."""
    import torch
    store, table = small_store(mm), torch.arange(3, device="cuda").int().view(1, 3)
    lens, w = torch.tensor([40], device="cuda").int(), torch.rand(1, 48, device="cuda")
    before, keep = [s.view(torch.uint8).clone() for s in store], 40 * 10 ** 6
    torch.cuda.synchronize()
    at = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    new, held, kept = mm.cache_evict([store], table, lens, w, keep, recent=5, block=64)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - at <= 4 * keep + (1 << 20)
    assert new.tolist() == [40] and torch.equal(held[:, :40], w[:, :40]) and not held[:, 40:].any()
    assert kept.shape == (1, keep) and kept[0, :40].tolist() == list(range(40)) and bool((kept[0, 40:] == -1).all())
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(before, store))


@pytest.mark.parametrize("keep", [47, 48, 49, 39, 40, 41, 0, 1])
def test_eviction_around_the_places_of_the_table(mm, keep):  # noqa: F811
    import torch
    store, table = small_store(mm), torch.tensor([[2, 0, 1]], device="cuda").int()
    lens, w = torch.tensor([40], device="cuda").int(), torch.rand(1, 48, device="cuda", generator=gen(3))
    rows = table[0].long().repeat_interleave(16) * 16 + torch.arange(48, device="cuda") % 16
    before = [s.view(torch.uint8).flatten(0, 1)[rows].clone() for s in store]
    new, held, kept = mm.cache_evict([store], table, lens, w, keep, block=64)
    stay = ref.evict(f64(w[0]), 40, keep, 0)
    assert new.tolist() == [len(stay)] and kept[0].tolist() == stay + [-1] * (keep - len(stay))
    assert np.array_equal(f64(held[0]), np.concatenate([f64(w[0])[stay], np.zeros(48 - len(stay))]))
    now = [s.view(torch.uint8).flatten(0, 1)[rows] for s in store]
    assert all(torch.equal(a[stay], b[:len(stay)]) for a, b in zip(before, now))


def test_stores_that_share_memory_are_refused(mm):  # noqa: F811
    """Rows would be moved once for each of them."""
    import torch
    (codes, scales), table = small_store(mm), torch.arange(3, device="cuda").int().view(1, 3)
    lens, w = torch.tensor([40], device="cuda").int(), torch.rand(1, 48, device="cuda")
    other, wide = codes.clone(), mm.cache_new((4, 16), 128, block=64)
    for stores in ([(codes, scales), (other, scales)], [(codes, scales), (codes, scales.clone())],
                   [tuple(t[:3] for t in wide), tuple(t[1:] for t in wide)]):
        before = [t.view(torch.uint8).clone() for s in stores for t in s]
        with pytest.raises(mm.EmeansError, match="EINVAL"):
            mm.cache_evict(stores, table, lens, w, 8, block=64)
        assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(before, (t for s in stores for t in s)))
    halves = mm.cache_new((6, 16), 128, block=64)        # two of one allocation that do not
    mm.cache_evict([tuple(t[:3] for t in halves), tuple(t[3:] for t in halves)], table, lens, w, 8, block=64)


@pytest.mark.parametrize("fmt,block", [("f8", 128), ("f8", 16), ("i8", 128), ("i8", 32)])
@pytest.mark.parametrize("width", [128, 48])
@pytest.mark.parametrize("places", [20, 700])
def test_softmax_weights_of_bf16_queries_keep_16_bits(mm, fmt, block, width, places):  # noqa: F811
    """Values of both signs, so that the result is small beside the sum of its terms and the weights'
    rounding would show: off by 2^-16 of that sum at most, beside the score's error, that
    of the sums and the result's own rounding."""
    import torch
    from test_gpu_attention_store import fill, lay_out, make_store, to_gpu
    rng = np.random.default_rng(places + width)
    d = 2 * width
    if block == 128:
        block = width
    pages, table, rows = lay_out(rng, [places], 16)
    k, v = (make_store(rng, pages, 16, d, block, fmt) for _ in range(2))
    for s in (k, v):
        fill(rng, s, rows[0], fmt)
    codes = v[0].reshape(-1, d)
    half = rows[0][1::2]                       # each second place has the value of the one before, negative
    prev = rows[0][:-1:2][:len(half)]
    codes[half] = codes[prev] ^ 0x80 if fmt == "f8" else (-codes[prev].view(np.int8)).view(np.uint8)
    v[1].reshape(-1, v[1].shape[-1])[half] = v[1].reshape(-1, v[1].shape[-1])[prev]
    kc, vc = (ref.store_values(s[0].reshape(-1, d)[rows[0]], s[1].reshape(-1, s[1].shape[-1])[rows[0]], block, fmt)
              .reshape(places, 2, width) for s in (k, v))
    q = (0.02 * randn(gen(3), 1, 8, width)).bfloat16()
    got = f64(mm.cache_attend(q, to_gpu(k, pages, 16, fmt), to_gpu(v, pages, 16, fmt), torch.from_numpy(table).cuda(),
                              torch.tensor([places], device="cuda").int(), block=block))[0]
    want, tol, _, _ = ref.decode(f64(q[0]), kc, vc, width ** -0.5, "bf16")
    size = np.stack([ref.softmax(kc[:, h // 4] @ f64(q[0, h]) * width ** -0.5) @ np.abs(vc[:, h // 4]) for h in range(8)])
    tol = tol - (2.0 ** -8 - 2.0 ** -16) * 1.01 * size
    off = np.abs(got - want)
    assert np.all(off <= tol), (off / size).max()


def test_gradients_with_saved_tensors_elsewhere_and_recomputed(mm):  # noqa: F811
    """Saved tensors kept in host memory come back with strides of their own; a checkpoint makes them
    anew."""
    import torch
    from torch.utils.checkpoint import checkpoint
    base = randn(gen(7), 80, 5 * 67).half()
    parts = [base[:, a * 67:b * 67].unflatten(1, (b - a, 67))[:, :, :64] for a, b in ((0, 3), (3, 4), (4, 5))]
    starts, pos, f = torch.tensor([0, 50, 80], device="cuda").int(), torch.arange(80, device="cuda"), mm.rotary_freqs(64)
    gain = torch.ones(64, device="cuda")

    def layer(q, k, v, g):
        return mm.attend(*mm.norm_rotate(q, k, g, g, pos, f), v, starts)

    def grads(run, *, offload=False):
        leaves = [t.detach().requires_grad_() for t in (*parts, gain)]
        with torch.autograd.graph.save_on_cpu() if offload else torch.enable_grad():
            o = run(*leaves)
        return (o.detach(), *torch.autograd.grad(o, leaves, torch.ones_like(o)))

    want = grads(layer)
    for got in (grads(layer, offload=True), grads(lambda *a: checkpoint(layer, *a, use_reentrant=False))):
        assert all(torch.equal(a, b) for a, b in zip(want, got))
