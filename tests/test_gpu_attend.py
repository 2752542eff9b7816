"""Attention over packed sequences and its gradients against the definition in 64 bits."""
import numpy as np
import pytest

import attention_ref as ref
from test_gpu_attention_store import T, f64, gen, mm, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def inputs(lq, lk, hq, hk, w, dtype, seed, lead=3, tail=5):
    """Packed q, k, v, dO of sequences of lq queries and lk keys, with rows of NaN before the
    first and behind the last; starts and k_starts."""
    import torch
    g = gen(seed)
    n, nk = sum(lq) + lead + tail, sum(lk) + lead + tail
    q, k, v, do = (x.to(T(dtype)) for x in (1.5 * randn(g, n, hq, w), randn(g, nk, hk, w), randn(g, nk, hk, w),
                                            0.1 * randn(g, n, hq, w)))
    for t in (q, k, v, do):
        t[:lead] = float("nan")
        t[len(t) - tail:] = float("inf")
    starts, k_starts = (torch.tensor([lead] + [lead + sum(x[:i + 1]) for i in range(len(x))], device="cuda").int()
                        for x in (lq, lk))
    return q, k, v, do, starts, k_starts


def check(mm, lq, lk, hq, hk, w, dtype, causal, seed=0, grad=True, scale=None, view=None):
    import torch
    q, k, v, do, starts, k_starts = inputs(lq, lk, hq, hk, w, dtype, seed)
    if view:
        q, k, v, do = (view(t) for t in (q, k, v, do))
    same = lq == lk
    leaves = [t.detach().requires_grad_(grad) for t in (q, k, v)]
    call = lambda: mm.attend(*leaves, starts, k_starts=None if same else k_starts, causal=causal, scale=scale)  # noqa: E731
    o = call()
    assert o.dtype == q.dtype and o.shape == q.shape and o.is_contiguous()
    if grad:
        with torch.no_grad():
            assert torch.equal(o, call())
        grads = torch.autograd.grad(o, leaves, do)
        again = torch.autograd.grad(call(), leaves, do)
        assert all(torch.equal(a, b) for a, b in zip(grads, again))
        got = [f64(t) for t in grads]
        want = [np.zeros(t.shape) for t in got]
        tols = [np.zeros(t.shape) for t in got]
    f = w ** -0.5 if scale is None else scale
    Q, K, V, DO, O = (f64(t) for t in (q, k, v, do, o))
    cq, ck = starts.tolist(), k_starts.tolist()
    assert not O[:cq[0]].any() and not O[cq[-1]:].any()
    top = np.abs(DO[cq[0]:cq[-1]]).max(initial=0) * np.abs(V[ck[0]:ck[-1]]).max(initial=0)
    for s in range(len(lq)):
        a, b, c, d = cq[s], cq[s + 1], ck[s], ck[s + 1]
        for h in range(hq):
            kv = h // (hq // hk)
            out, tol, _ = ref.attend(Q[a:b, h], K[c:d, kv], V[c:d, kv], f, causal, dtype)
            off = np.abs(O[a:b, h] - out)
            assert bool(np.all(off <= tol)), (s, h, off.max())
            if grad:
                x, t = ref.attend_grad(Q[a:b, h], K[c:d, kv], V[c:d, kv], DO[a:b, h], f, causal, dtype, top)
                for i, (lo, hi, hh) in enumerate(((a, b, h), (c, d, kv), (c, d, kv))):
                    want[i][lo:hi, hh] += x[i]
                    tols[i][lo:hi, hh] += t[i]
    if grad:
        for name, x, y, t in zip("qkv", got, want, tols):
            t = t + (ref.HALF_ULP[dtype] * 1.01 + hq // hk * ref.SUM_ULP) * np.abs(y) + (y != 0) * ref.TINY[dtype]
            off = np.abs(x - y)
            assert bool(np.all(off <= t)), (name, off.max(), np.argwhere(off > t)[:3].tolist())
    return o


EDGES = [0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 2, 300]


@pytest.mark.parametrize("hq,hk,w", [(2, 2, 64), (4, 1, 128), (3, 3, 96), (6, 2, 80), (1, 1, 8), (8, 8, 16),
                                     (7, 1, 40), (16, 2, 72), (5, 5, 104), (2, 1, 120), (9, 3, 32)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [True, False])
def test_attend(mm, hq, hk, w, dtype, causal):
    check(mm, EDGES, EDGES, hq, hk, w, dtype, causal, hq + w)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("w", [64, 96, 128])
def test_attend_with_more_or_fewer_keys_than_queries(mm, dtype, causal, w):
    """Chunks of prompts behind cached keys; queries that see no key; sequences that have
    only queries or only keys."""
    lq = [1, 1, 40, 130, 200, 70, 0, 5, 65, 64]
    lk = [1, 300, 333, 130, 60, 0, 50, 1, 1, 129]
    check(mm, lq, lk, 4, 2, w, dtype, causal, 3)


@pytest.mark.parametrize("w,hq,hk,causal", [(128, 4, 1, True), (64, 2, 2, False)])
def test_attend_long(mm, w, hq, hk, causal):
    check(mm, [2100, 1], [2100, 1], hq, hk, w, "bf16", causal, 5)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attend_scales(mm, scale, dtype):
    check(mm, [100, 7], [100, 7], 2, 1, 64, dtype, True, 6, scale=scale)


def test_attend_takes_any_strides(mm):
    import torch

    def fused(t):                      # a slice of a wider row
        return torch.cat([t.flatten(1), t.flatten(1)[:, :8 * 3]], 1)[:, :t.shape[1] * t.shape[2]].unflatten(1, t.shape[1:])

    def heads_first(t):
        return t.transpose(0, 1).contiguous().transpose(0, 1)

    def odd(t):                        # rows at no multiple of 16 bytes
        room = torch.zeros(t.shape[0], t.shape[1], t.shape[2] + 3, device="cuda", dtype=t.dtype)
        room[:, :, 1:-2] = t
        return room[:, :, 1:-2]

    def values_apart(t):
        return t.transpose(1, 2).contiguous().transpose(1, 2)

    outs = [check(mm, [40, 65], [40, 65], 2, 2, 64, "bf16", True, 7, view=f)
            for f in (lambda t: t, fused, heads_first, odd, values_apart)]
    assert all(torch.equal(outs[0], o) for o in outs[1:])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("dtype,w", [("bf16", 128), ("f16", 64), ("bf16", 96)])
def test_what_a_row_does_not_see_does_not_show(mm, bad, which, dtype, w):
    """From some row on keys or values are no numbers: the rows before are as without them, to
    the bit; the rows that see them are no numbers where the definition says so."""
    import torch
    n, at = 300, 77
    q, k, v, _, starts, _ = inputs([n], [n], 2, 1, w, dtype, 8, 0, 0)
    clean = mm.attend(q, k, v, starts)
    k2, v2 = k.clone(), v.clone()
    if which != "v":
        k2[at:, :, 3] = bad
    if which != "k":
        v2[at:, :, 5] = bad
        v2[at + 100, :, 6] = -bad
    got = mm.attend(q, k2, v2, starts)
    assert torch.equal(got[:at], clean[:at])
    if which == "v":
        assert torch.equal(got[:, :, 7:], clean[:, :, 7:])
        col = got[at:, :, 5].float()
        assert bool((torch.isnan(col) if bad != bad else col == bad).all())
        assert torch.isfinite(got[:at + 100, :, 6]).all() and not torch.isfinite(got[at + 100:, :, 6]).any()
    elif bad == bad and which == "k":     # a score of +infinity makes its row NaN, one of -infinity drops a key
        plus = (q[at:, :, 3].float() * bad) > 0
        assert torch.isnan(got[at:][plus]).all()
    elif bad != bad:
        assert torch.isnan(got[at:]).all()


def test_mixed_infinities_in_values(mm):
    import torch
    q, k, v, _, starts, _ = inputs([70], [70], 1, 1, 64, "bf16", 9, 0, 0)
    v[10, 0, 0], v[20, 0, 0] = float("inf"), -float("inf")
    v[69, 0, 1] = float("nan")
    o = mm.attend(q, k, v, starts)[:, 0].float()
    assert torch.isfinite(o[:10]).all() and bool((o[10:20, 0] == float("inf")).all()) and torch.isnan(o[20:, 0]).all()
    assert torch.isfinite(o[:69, 1]).all() and torch.isnan(o[69, 1]) and torch.isfinite(o[:, 2:]).all()


def test_gradients_of_other_sequences_are_untouched_by_a_nan(mm):
    import torch
    q, k, v, do, starts, _ = inputs([100, 60, 100], [100, 60, 100], 2, 1, 64, "f16", 10, 0, 0)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    clean = torch.autograd.grad(mm.attend(*leaves, starts), leaves, do)
    k[130] = float("nan")
    do[140] = float("inf")
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    got = torch.autograd.grad(mm.attend(*leaves, starts), leaves, do)
    for a, b in zip(clean, got):
        assert torch.equal(a[:100], b[:100]) and torch.equal(a[160:], b[160:])


@pytest.mark.parametrize("size", [2.0 ** -14, 1.0, 2.0 ** 9])
def test_fp16_gradients_of_any_size(mm, size):
    """dO and V from fp16's smallest normal numbers to large ones: the weights' gradients keep
    their digits."""
    import torch
    q, k, v, do, starts, _ = inputs([200], [200], 2, 1, 64, "f16", 11, 0, 0)
    for x, y in ((do * size * 10, v), (do, v * size)):
        leaves = [t.clone().requires_grad_() for t in (q, k, y)]
        got = torch.autograd.grad(mm.attend(*leaves, starts), leaves, x)
        top = float(x.abs().max() * y.abs().max())
        total = [np.zeros((200, 64)) for _ in range(2)]
        tols = [np.zeros((200, 64)) for _ in range(2)]
        for h in range(2):
            want, tol = ref.attend_grad(f64(q[:, h]), f64(k[:, 0]), f64(y[:, 0]), f64(x[:, h]), 0.125, True, "f16", top)
            t = tol[0] + ref.HALF_ULP["f16"] * 1.01 * np.abs(want[0]) + ref.TINY["f16"]
            assert bool(np.all(np.abs(f64(got[0][:, h]) - want[0]) <= t))
            for i in range(2):
                total[i] += want[i + 1]
                tols[i] += tol[i + 1]
        for i in range(2):
            t = tols[i] + (ref.HALF_ULP["f16"] * 1.01 + 4 * ref.SUM_ULP) * np.abs(total[i]) + ref.TINY["f16"]
            assert bool(np.all(np.abs(f64(got[i + 1][:, 0]) - total[i]) <= t))


def test_gradients_against_differences(mm):
    """The change of a weighted sum of the results along the gradient: as the gradient says, up
    to what the definition's own change differs from it and what the results may be off by."""
    import torch
    q, k, v, do, starts, _ = inputs([90], [90], 2, 1, 64, "f16", 12, 0, 0)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    grads = torch.autograd.grad(mm.attend(*leaves, starts), leaves, do)
    for i in range(3):
        way = grads[i].float() / grads[i].float().norm()
        ends, exact, tol, points = [], [], 0.0, []
        for sign in (1, -1):
            x = [t.detach() for t in (q, k, v)]
            x[i] = (x[i].float() + sign * 2.0 * way).half()
            points.append(f64(x[i]))
            ends.append((f64(mm.attend(*x, starts)) * f64(do)).sum())
            e = 0.0
            for h in range(2):
                out, t, _ = ref.attend(f64(x[0][:, h]), f64(x[1][:, 0]), f64(x[2][:, 0]), 0.125, True, "f16")
                e += (out * f64(do[:, h])).sum()
                tol += (t * np.abs(f64(do[:, h]))).sum()
            exact.append(e)
        said = ((points[0] - points[1]) * f64(grads[i])).sum()
        assert abs(said) > 4 * tol or i == 2
        assert abs((ends[0] - ends[1]) - said) <= abs((exact[0] - exact[1]) - said) + tol


def test_attend_of_nothing_and_of_starts_outside_the_tensors(mm):
    import torch
    none = torch.zeros(0, 2, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    zero = torch.zeros(1, device="cuda").int()
    o = mm.attend(none, none, none, zero)
    assert o.shape == (0, 2, 64) and torch.autograd.grad(o, none, o.detach())[0].shape == none.shape
    q = torch.randn(40, 2, 64, device="cuda").bfloat16().requires_grad_()
    o = mm.attend(q, none, none, torch.tensor([0, 40], device="cuda").int(), k_starts=torch.zeros(2, device="cuda").int())
    assert not o.any() and not torch.autograd.grad(o, q, o.detach())[0].any()
    for rows in (40, 300):                 # no sequence at all
        x = torch.ones(rows, 2, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
        o = mm.attend(x, x, x, zero)
        assert not o.any() and not torch.autograd.grad(o, x, torch.ones_like(o))[0].any()
    # starts are cut to the tensors: no row outside them is read
    for s in ([-5, 1000], [0, 50], [39, 20, 45]):
        starts = torch.tensor(s, device="cuda").int()
        assert torch.isfinite(mm.attend(q, q, q, starts)).all()
    with torch.no_grad():
        assert torch.equal(mm.attend(q, q, q, torch.tensor([-5, 1000], device="cuda").int()),
                           mm.attend(q, q, q, torch.tensor([0, 40], device="cuda").int()))


def test_attend_on_a_given_stream_and_in_graphs(mm):
    """A captured training step replayed with eager work between, while an eager graph of the
    same leaves lives; two graphs in turn."""
    import torch
    q, k, v, do, starts, _ = inputs([300, 33], [300, 33], 4, 2, 64, "f16", 13, 0, 0)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]

    def step(scale=None):
        o = mm.attend(*leaves, starts, scale=scale)
        return (o.detach(), *torch.autograd.grad(o, leaves, do))

    want = [[t.clone() for t in step(s)] for s in (None, 0.5)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mm.attend(*leaves, starts, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[0][0])
    del got
    graphs, outs = [], []
    for s in (None, 0.5):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(s))
        graphs.append(graph)
    for _ in range(4):
        for t in (*outs[0], *outs[1]):
            t.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for o, w in zip(outs, want) for a, b in zip(o, w))
        assert all(torch.equal(a, b) for a, b in zip(step(), want[0]))
