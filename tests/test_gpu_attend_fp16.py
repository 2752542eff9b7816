"""Digits of fp16 attention: what is rounded to fp16 on the way keeps them whatever else the call
holds."""
import numpy as np
import pytest

import attention_ref as ref
from test_gpu_attend import inputs
from test_gpu_attention_store import f64, gen, mm, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def step(mm, q, k, v, do, starts, causal=True):  # noqa: F811
    import torch
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, v)]
    return torch.autograd.grad(mm.attend(*leaves, starts, causal=causal), leaves, do)


@pytest.mark.parametrize("w,hq,hk", [(128, 4, 2), (64, 2, 2), (96, 3, 1), (40, 2, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_gradients_do_not_depend_on_rows_outside_sequences(mm, w, hq, hk, causal):  # noqa: F811
    import torch
    q, k, v, do, starts, _ = inputs([200, 64, 1], [200, 64, 1], hq, hk, w, "f16", 1)
    got = []
    for fill in (0.0, 6e4, -6e4):
        for t in (q, k, v, do):
            t[:3] = t[-5:] = fill
        got.append(step(mm, q, k, v, do, starts, causal))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
    assert all(not g[:3].any() and not g[-5:].any() for g in got[0])


def test_gradients_do_not_depend_on_other_sequences_and_heads(mm):  # noqa: F811
    import torch
    q, k, v, do, starts, _ = inputs([150, 70, 90], [150, 70, 90], 4, 2, 64, "f16", 2, 0, 0)
    want = step(mm, q, k, v, do, starts)
    v2, do2 = v.clone(), do.clone()
    v2[150:220], do2[150:220] = 6e4, 6e4            # the sequence between
    for a, b in zip(want, step(mm, q, k, v2, do2, starts)):
        assert torch.equal(a[:150], b[:150]) and torch.equal(a[220:], b[220:])
    v2, do2 = v.clone(), do.clone()
    v2[:, 1], do2[:, 2:] = 6e4, 6e4                 # the other key-value head
    for a, b in zip(want, step(mm, q, k, v2, do2, starts)):
        assert torch.equal(a[:, :a.shape[1] // 2], b[:, :a.shape[1] // 2])


def test_gradients_do_not_depend_on_rows_that_are_not_seen(mm):  # noqa: F811
    """Causal: values behind a query, and queries before a key."""
    import torch
    q, k, v, do, starts, _ = inputs([210], [210], 2, 1, 128, "f16", 3, 0, 0)
    want = step(mm, q, k, v, do, starts)
    late = v.clone()
    late[77:] = 6e4
    assert torch.equal(want[0][:77], step(mm, q, k, late, do, starts)[0][:77])
    early = do.clone()
    early[:77] = 6e4
    got = step(mm, q, k, v, early, starts)
    assert torch.equal(want[1][77:], got[1][77:]) and torch.equal(want[2][77:], got[2][77:])


def score_grads(q, k, v, do, scale, causal):
    p = ref.softmax(np.where(ref.seen(len(q), len(k), causal), q @ k.T * scale, -np.inf))
    return np.abs(p * (do @ v.T - (do * (p @ v)).sum(1, keepdims=True)))


@pytest.mark.parametrize("n,w,causal", [(230, 128, True), (65, 64, False), (130, 96, True), (33, 32, False)])
def test_gradients_of_rows_of_any_size_side_by_side(mm, n, w, causal):  # noqa: F811
    """dO and V of rows from 2^-13 to 1 and from 2^-6 to 2^6. Scores' gradients are fp16 numbers times a
    power of two that leaves the largest of a query's (for dQ) or of a key's (for dK) at
    least 2^11, where the step at zero is 2^-24: off by 2^-25 2^-11 of the largest at most
    beside half a unit of their own."""
    q, k, v, do, starts, _ = inputs([n], [n], 2, 1, w, "f16", n, 0, 0)
    g = gen(n + 1)
    import torch
    do = (do.float() * torch.exp2(-13 * torch.rand(n, 1, 1, device="cuda", generator=g))).half()
    v = (v.float() * torch.exp2(6 - 12 * torch.rand(n, 1, 1, device="cuda", generator=g))).half()
    got = [f64(t) for t in step(mm, q, k, v, do, starts, causal)]
    scale = w ** -0.5
    total = [np.zeros((n, w)) for _ in range(2)]
    tols = [np.zeros((n, w)) for _ in range(2)]
    mask = ref.seen(n, n, causal)
    sizes = [score_grads(f64(q[:, h]), f64(k[:, 0]), f64(v[:, 0]), f64(do[:, h]), scale, causal) for h in range(2)]
    step_of = 2.0 ** -25 * 2.0 ** -11 * 1.01
    by_key = np.maximum(*sizes).max(0, keepdims=True) * step_of * mask
    for h in range(2):
        want, tol = ref.attend_grad(f64(q[:, h]), f64(k[:, 0]), f64(v[:, 0]), f64(do[:, h]), scale, causal, "f16", 0.0)
        more = scale * (sizes[h].max(1, keepdims=True) * step_of * mask) @ np.abs(f64(k[:, 0]))
        t = tol[0] + more + ref.HALF_ULP["f16"] * 1.01 * np.abs(want[0]) + ref.TINY["f16"]
        off = np.abs(got[0][:, h] - want[0])
        assert np.all(off <= t), (h, np.argwhere(off > t)[:3].tolist())
        for i in range(2):
            total[i] += want[i + 1]
            tols[i] += tol[i + 1]
        tols[0] += scale * by_key.T @ np.abs(f64(q[:, h]))
    for i in range(2):
        t = tols[i] + (ref.HALF_ULP["f16"] * 1.01 + 4 * ref.SUM_ULP) * np.abs(total[i]) + ref.TINY["f16"]
        off = np.abs(got[i + 1][:, 0] - total[i])
        assert np.all(off <= t), (i, np.argwhere(off > t)[:3].tolist())


@pytest.mark.parametrize("w,at,below", [(64, 0, 15.0), (64, 4096, 15.0), (128, 2000, 12.0), (96, 70, 15.0)])
def test_many_small_weights_keep_their_digits(mm, w, at, below):  # noqa: F811
    """One key holds nearly all of the weight and has a value of 0; 4096 others weigh e^-12 or e^-15
    each (2^-17.3, 2^-21.6: fp16 has its smallest normal number at 2^-14 and a step of 2^-24
    there) and make up the result."""
    import torch
    n = 40
    q, k, v = (torch.zeros(r, 1, w, device="cuda", dtype=torch.float16) for r in (n, 4097, 4097))
    q[:, 0, 0] = 1.0
    k[at, 0, 0] = below
    v[:] = randn(gen(5), 1, 1, w)
    v[at] = 0.0
    starts, ks = (torch.tensor([0, r], device="cuda").int() for r in (n, 4097))
    o = mm.attend(q, k, v, starts, k_starts=ks, causal=False, scale=1.0)
    want, tol, _ = ref.attend(f64(q[:, 0]), f64(k[:, 0]), f64(v[:, 0]), 1.0, False, "f16")
    off = np.abs(f64(o[:, 0]) - want)
    assert np.all(off <= tol), (off / np.abs(want)).max()
    # the gradients go by the same weights
    do = torch.ones_like(q)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    dv = torch.autograd.grad(mm.attend(*leaves, starts, k_starts=ks, causal=False, scale=1.0), leaves, do)[2]
    (_, _, dv_want), (_, _, dv_tol) = ref.attend_grad(f64(q[:, 0]), f64(k[:, 0]), f64(v[:, 0]), f64(do[:, 0]), 1.0, False, "f16")
    assert np.all(np.abs(f64(dv[:, 0]) - dv_want) <= dv_tol + ref.HALF_ULP["f16"] * 1.01 * np.abs(dv_want) + ref.TINY["f16"])
