"""The attention operators together, as a layer uses them: prompts, new tokens over the
store, eviction, a training step (examples/token_attention.py)."""
import os
import sys

import numpy as np
import pytest

import attention_ref as ref
from test_gpu_attention_store import f64, mm  # noqa: F401

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex(mm):  # noqa: F811
    import token_attention
    return token_attention


def stored(mm, cache, seq, n):  # noqa: F811
    """Keys and values of a sequence's first n places as they are in the store (bf16: exact)."""
    import torch
    place = torch.arange(n, device="cuda")
    at = cache.slots(torch.full_like(place, seq), place)
    return [f64(mm.cache_read(*s, at, block=cache.block)) for s in (cache.keys, cache.values)]


def test_new_tokens_attend_over_what_the_store_holds(mm, ex):  # noqa: F811
    import torch
    layer = ex.Layer()
    weights = [mm.block_encode(w, tiles=True) for w in (layer.w_in, layer.w_out)]
    lengths = [70, 1, 33, 0]
    cache = ex.Cache(layer, 4, 8)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(sum(lengths), layer.d, device="cuda", generator=g).bfloat16()
    _, (q, k, v, o) = ex.prompt(layer, weights, cache, x, lengths)
    at = np.cumsum([0] + lengths)
    for s, n in enumerate(lengths):              # the prompt itself, and what was written of it
        for h in range(layer.hq):
            a, b = at[s], at[s + 1]
            want, tol, _ = ref.attend(f64(q[a:b, h]), f64(k[a:b, h // 4]), f64(v[a:b, h // 4]), 0.125, True, "bf16")
            assert np.all(np.abs(f64(o[a:b, h]) - want) <= tol)
        if n == 0:
            continue
        kc, vc = stored(mm, cache, s, n)
        for c, t in ((kc, k), (vc, v)):          # E4M3: half a step is 2^-4 of a value, 2^-10 of the block's scale
            t = f64(t[at[s]:at[s + 1]]).reshape(n, -1)
            big = np.abs(t.reshape(n, layer.hk, -1)).max(2).repeat(layer.width, 1)
            assert np.all(np.abs(c - t) <= 2.0 ** -4 * np.abs(t) + 2.0 ** -10 * big / 224)
    total = np.zeros((4, 8 * cache.page))
    for _ in range(3):
        before = f64(cache.weights)
        _, (q, o) = ex.step(layer, weights, cache, torch.randn(4, layer.d, device="cuda", generator=g).bfloat16())
        for s in range(4):
            n = int(cache.lengths[s])
            kc, vc = (t.reshape(n, layer.hk, -1) for t in stored(mm, cache, s, n))
            want, tol, w, wtol = ref.decode(f64(q[s]), kc, vc, 0.125, "bf16")
            assert np.all(np.abs(f64(o[s]) - want) <= tol)
            got = f64(cache.weights[s]) - before[s]
            assert np.all(np.abs(got[:n] - w) <= wtol + ref.SUM_ULP * f64(cache.weights[s])[:n]) and not got[n:].any()
            total[s, :n] += w
    # eviction: rows, weights and lengths move together, and attention goes on over them
    old = [stored(mm, cache, s, int(cache.lengths[s])) for s in range(4)]
    held, lens = f64(cache.weights), cache.lengths.tolist()
    kept = ex.trim(cache, 40, 8)
    for s in range(4):
        stay = ref.evict(held[s], lens[s], 40, 8)
        assert kept[s].tolist() == stay + [-1] * (40 - len(stay)) and int(cache.lengths[s]) == len(stay)
        now = stored(mm, cache, s, len(stay))
        assert all(np.array_equal(a, b[stay]) for a, b in zip(now, old[s]))
        assert np.array_equal(f64(cache.weights[s])[:len(stay)], held[s][stay])
    _, (q, o) = ex.step(layer, weights, cache, torch.randn(4, layer.d, device="cuda", generator=g).bfloat16())
    for s in range(4):
        n = int(cache.lengths[s])
        kc, vc = (t.reshape(n, layer.hk, -1) for t in stored(mm, cache, s, n))
        want, tol, _, _ = ref.decode(f64(q[s]), kc, vc, 0.125, "bf16")
        assert np.all(np.abs(f64(o[s]) - want) <= tol)


def test_training_step(ex):
    """A step gives finite gradients of all weights, the same ones each time."""
    import torch
    layer = ex.Layer(d=256, hq=4, hk=2, width=64)
    lengths = [50, 3, 20]
    x = torch.randn(73, 256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9)).bfloat16()
    loss, grads = ex.train_step(layer, x, lengths, torch.zeros_like(x))
    assert all(torch.isfinite(t).all() and t.abs().max() > 0 for t in grads)
    again = ex.train_step(layer, x, lengths, torch.zeros_like(x))[1]
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_gradients_through_attention_and_norms(mm):  # noqa: F811
    """dO to the gains and to the projected queries and keys, through both operators: the 64-bit
    chain on the same rounded queries and keys, with the tolerance of one carried through
    the other."""
    import torch
    n, hq, hk, w = 90, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    y = torch.randn(n, hq + 2 * hk, w, device="cuda", generator=g).bfloat16().requires_grad_()
    gains = [(1 + 0.2 * torch.randn(w, device="cuda", generator=g)).requires_grad_() for _ in range(2)]
    do = (0.1 * torch.randn(n, hq, w, device="cuda", generator=g)).bfloat16()
    pos, freqs = torch.arange(n, device="cuda"), mm.rotary_freqs(w)
    starts = torch.tensor([0, 60, 60, n], device="cuda").int()
    q, k, v = y.split([hq, hk, hk], 1)
    qr, kr = mm.norm_rotate(q, k, *gains, pos, freqs)
    dy, *dgains = torch.autograd.grad(mm.attend(qr, kr, v, starts), (y, *gains), do)
    Q, K, V, DO = f64(qr), f64(kr), f64(v), f64(do)
    grads = [np.zeros(t.shape) for t in (Q, K, V)]
    tols = [np.zeros(t.shape) for t in (Q, K, V)]
    for a, b in ((0, 60), (60, n)):
        for h in range(hq):
            got, tol = ref.attend_grad(Q[a:b, h], K[a:b, h // 2], V[a:b, h // 2], DO[a:b, h], w ** -0.5, True, "bf16")
            for i, hh in enumerate((h, h // 2, h // 2)):
                grads[i][a:b, hh] += got[i]
                tols[i][a:b, hh] += tol[i]
    for t, e in zip(grads, tols):
        e += (ref.HALF_ULP["bf16"] * 1.01 + 4 * ref.SUM_ULP) * np.abs(t) + ref.TINY["bf16"]
    P, F = pos.cpu().numpy(), f64(freqs)
    for i, (x, gain, at) in enumerate(((q, gains[0], slice(0, hq)), (k, gains[1], slice(hq, hq + hk)))):
        X, G = f64(x), f64(gain)
        dx, dx_tol, dg, dg_tol = ref.rotate_grad(X, G, P, F, grads[i])
        carried = ref.turn(tols[i], P, F)[1]                 # a turned value is off by both of its pair's
        r = 1 / np.sqrt((X * X).mean(-1, keepdims=True) + 1e-6)
        dg_tol = dg_tol + (carried * np.abs(X) * r).sum((0, 1)) * (1 + 2.0 ** -8)
        dx_tol = dx_tol + (r * np.abs(G) * carried + np.abs(X) * r ** 3 * (carried * np.abs(G * X)).mean(-1, keepdims=True)) \
            * (1 + 2.0 ** -8) + ref.HALF_ULP["bf16"] * 1.01 * np.abs(dx) + ref.TINY["bf16"]
        assert np.all(np.abs(f64(dgains[i]) - dg) <= dg_tol + 2.0 ** -24 * np.abs(dg))
        assert np.all(np.abs(f64(dy[:, at]) - dx) <= dx_tol)
    assert np.all(np.abs(f64(dy[:, hq + hk:]) - grads[2]) <= tols[2])


def test_example_runs(ex):
    out = ex.main(steps=30)
    assert out["cache"].positions.tolist() == [100, 31, 63]
    assert out["kept"] is not None and int(out["cache"].lengths.max()) < 64 + 16
