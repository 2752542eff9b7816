"""Attention around the store: calls that its documentation allows and that are easily
forgotten, and refusals that need tensors on the GPU."""
import numpy as np
import pytest

import attention_ref as ref
from test_gpu_attend import inputs
from test_gpu_attention_store import f64, fill, gen, lay_out, make_store, mm, randn, rotate_inputs, to_gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def test_refusals_of_norm_rotate_and_attend(mm):  # noqa: F811
    import torch
    q, k, gq, gk, pos = rotate_inputs(4, 4, 2, 64, 64, "bf16", 1)
    f = mm.rotary_freqs(64)
    turn = lambda q=q, k=k, gq=gq, gk=gk, pos=pos, f=f, **kw: mm.norm_rotate(q, k, gq, gk, pos, f, **kw)  # noqa: E731
    starts = torch.tensor([0, 4], device="cuda").int()
    att = lambda q=q, k=k, v=k, s=starts, **kw: mm.attend(q, k, v, s, **kw)  # noqa: E731
    turn()
    att()
    for call, word in (
            (lambda: turn(q=q.double()), "EDTYPE"), (lambda: turn(k=k.half()), "EDTYPE"), (lambda: turn(k=k[:3]), "EINVAL"),
            (lambda: turn(k=k[..., :56]), "EINVAL"), (lambda: turn(gq=gq[:63]), "EINVAL"), (lambda: turn(gk=gk.float()), "EDTYPE"),
            (lambda: turn(pos=pos.float()), "EDTYPE"), (lambda: turn(pos=pos[:2]), "EINVAL"), (lambda: turn(f=f.float()), "EDTYPE"),
            (lambda: turn(f=mm.rotary_freqs(128)), "EINVAL"), (lambda: turn(q=q[:, :, 0]), "EINVAL"), (lambda: turn(eps=-1.0), "EINVAL"),
            (lambda: turn(gq=gq.cpu()), "ENOTDEVICE"), (lambda: turn(q=q[..., ::2], k=k[..., ::2]), "EINVAL"),
            (lambda: att(q=q.float(), k=k.float(), v=k.float()), "EDTYPE"), (lambda: att(k=k.half()), "EDTYPE"),
            (lambda: att(v=k[:3]), "EINVAL"), (lambda: att(q=q[:3]), "EINVAL"), (lambda: att(q=q[:, :3]), "EINVAL"),
            (lambda: att(q=q[..., :60], k=k[..., :60], v=k[..., :60]), "EINVAL"), (lambda: att(s=starts.long()), "EDTYPE"),
            (lambda: att(s=starts[:0]), "EINVAL"), (lambda: att(k_starts=starts[:1]), "EINVAL"), (lambda: att(q=q[0]), "EINVAL"),
            (lambda: att(scale=float("inf")), "EINVAL"), (lambda: att(s=starts.cpu()), "ENOTDEVICE"),
            (lambda: att(q=torch.cat([q] * 3, 2), k=torch.cat([k] * 3, 2), v=torch.cat([k] * 3, 2)), "EINVAL")):
        with pytest.raises(mm.EmeansError, match=word):
            call()


def test_tangents_traces_and_second_derivatives_are_refused(mm):  # noqa: F811
    import torch
    import torch.autograd.forward_ad as fwd
    q, k, gq, gk, pos = rotate_inputs(4, 2, 2, 64, 64, "bf16", 2)
    f, starts = mm.rotary_freqs(64), torch.tensor([0, 4], device="cuda").int()
    calls = (lambda x: mm.norm_rotate(x, k, gq, gk, pos, f)[0], lambda x: mm.attend(x, k, k, starts))
    for call in calls:
        with fwd.dual_level(), pytest.raises(mm.EmeansError, match="forward-mode"):
            call(fwd.make_dual(q, torch.ones_like(q)))
        with pytest.raises(mm.EmeansError, match="traced"):
            torch.jit.trace(call, (q,), check_trace=False)
        x = q.detach().clone().requires_grad_()
        g, = torch.autograd.grad(call(x), x, torch.ones_like(q), create_graph=True)
        with pytest.raises(RuntimeError, match="differentiate twice|does not require grad"):
            g.sum().backward()


def test_gradients_of_one_result_alone_and_of_a_graph_kept(mm):  # noqa: F811
    import torch
    q, k, gq, gk, pos = rotate_inputs(9, 3, 1, 64, 32, "f32", 3)
    f = mm.rotary_freqs(32)
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, gq, gk)]
    y = mm.norm_rotate(*leaves, pos, f)
    d = randn(gen(4), 9, 3, 64)
    one = torch.autograd.grad(y[0], leaves, d, retain_graph=True)
    both = torch.autograd.grad(y, leaves, (d, torch.zeros_like(y[1])))
    assert all(torch.equal(a, b) for a, b in zip(one, both))
    assert not one[1].any() and not one[3].any()
    # inputs of which only some have a gradient, and a gradient that is an expanded number
    y = mm.norm_rotate(q, k, leaves[2], gk, pos, f)
    g, = torch.autograd.grad(y[0].sum(), leaves[2])
    want = ref.rotate_grad(f64(q), f64(gq), pos.cpu().numpy(), f64(f), np.ones((9, 3, 64)))
    assert np.all(np.abs(f64(g) - want[2]) <= want[3] + 2.0 ** -24 * np.abs(want[2]))
    a, b, c, _, starts, _ = inputs([40, 9], [40, 9], 4, 2, 64, "bf16", 5, 0, 0)
    v = c.clone().requires_grad_()
    o = mm.attend(a, b, v, starts)
    first, = torch.autograd.grad(o.sum(), v, retain_graph=True)
    second, = torch.autograd.grad(o, v, torch.ones_like(o))
    assert torch.equal(first, second)


def test_shared_and_broadcast_inputs(mm):  # noqa: F811
    """One tensor as queries, keys and values, and keys that are one head expanded: gradients are the
    sums of those of separate tensors."""
    import torch
    x, _, _, do, starts, _ = inputs([70, 33], [70, 33], 2, 2, 64, "f16", 6, 0, 0)
    x = x.requires_grad_()
    shared, = torch.autograd.grad(mm.attend(x, x, x, starts), x, do)
    parts = [x.detach().clone().requires_grad_() for _ in range(3)]
    grads = torch.autograd.grad(mm.attend(*parts, starts), parts, do)
    total = sum(t.float() for t in grads)
    # 16-bit sums of three numbers: two roundings of partial sums
    assert bool(((shared.float() - total).abs() <= 2 * 2.0 ** -11 * sum(t.float().abs() for t in grads) + 2.0 ** -24).all())
    one = x.detach()[:, :1].clone().requires_grad_()
    wide = one.detach().expand(-1, 2, -1).contiguous().requires_grad_()
    o = mm.attend(x.detach(), one.expand(-1, 2, -1), one.expand(-1, 2, -1), starts)
    p = mm.attend(x.detach(), wide, wide, starts)
    assert torch.equal(o, p)
    a, = torch.autograd.grad(o, one, do)
    apart = [wide.detach().clone().requires_grad_() for _ in range(2)]
    grads = torch.autograd.grad(mm.attend(x.detach(), *apart, starts), apart, do)
    terms = torch.cat(grads, 1).float()
    # four 16-bit numbers added in some order: three roundings of partial sums
    assert bool(((a.float() - terms.sum(1, keepdim=True)).abs()
                 <= 3.1 * 2.0 ** -11 * terms.abs().sum(1, keepdim=True) + 2.0 ** -23).all())


def test_two_calls_at_once(mm):  # noqa: F811
    """Calls on two streams over one store, with their own working memory, and a training step beside
    them."""
    import torch
    rng = np.random.default_rng(7)
    lengths = [3000, 700, 0, 64]
    pages, table, rows = lay_out(rng, lengths, 16)
    k, v = (make_store(rng, pages, 16, 256, 64, "f8") for _ in range(2))
    for r in rows:
        fill(rng, k, r, "f8")
        fill(rng, v, r, "f8")
    keys, values = to_gpu(k, pages, 16, "f8"), to_gpu(v, pages, 16, "f8")
    table, lens = torch.from_numpy(table).cuda(), torch.tensor(lengths, device="cuda").int()
    q = [torch.randn(4, 8, 64, device="cuda").bfloat16() for _ in range(2)]
    x, y, z, do, starts, _ = inputs([200, 100], [200, 100], 4, 2, 64, "f16", 8, 0, 0)
    leaves = [t.clone().requires_grad_() for t in (x, y, z)]
    call = lambda i, **kw: mm.cache_attend(q[i], keys, values, table, lens, block=64, **kw)  # noqa: E731
    step = lambda: torch.autograd.grad(mm.attend(*leaves, starts), leaves, do)  # noqa: E731
    want, grads = [call(i) for i in range(2)], step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [call(i, stream=s) for i, s in enumerate(streams)]
        now = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got + list(now), want + list(grads)))


def test_backward_on_the_stream_of_the_forward_pass(mm):  # noqa: F811
    import torch
    x, y, z, do, starts, _ = inputs([150], [150], 2, 2, 64, "bf16", 9, 0, 0)
    leaves = [t.clone().requires_grad_() for t in (x, y, z)]
    want = torch.autograd.grad(mm.attend(*leaves, starts), leaves, do)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = mm.attend(*leaves, starts, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    got = torch.autograd.grad(o, leaves, do)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("seqs", [64, 65, 1000, 5000])
def test_many_short_sequences(mm, seqs):  # noqa: F811
    """A tile finds its sequence among any number of them, empty ones too."""
    import torch
    rng = np.random.default_rng(seqs)
    lengths = rng.integers(0, 4, seqs)
    lengths[rng.integers(0, seqs)] = 140
    starts = np.concatenate([[0], lengths.cumsum()])
    n = int(starts[-1])
    q, k, v = (randn(gen(i), n, 1, 16).bfloat16() for i in range(3))
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    o = mm.attend(*leaves, torch.from_numpy(starts).int().cuda())
    d = torch.ones_like(o)
    dq, dk, dv = torch.autograd.grad(o, leaves, d)
    Q, K, V, O, DV = (f64(t)[:, 0] for t in (q, k, v, o, dv))
    for s in rng.choice(seqs, min(seqs, 200), replace=False).tolist() + [int(lengths.argmax())]:
        a, b = starts[s], starts[s + 1]
        want, tol, _ = ref.attend(Q[a:b], K[a:b], V[a:b], 0.25, True, "bf16")
        assert np.all(np.abs(O[a:b] - want) <= tol)
        (_, _, gv), (_, _, tv) = ref.attend_grad(Q[a:b], K[a:b], V[a:b], np.ones((b - a, 16)), 0.25, True, "bf16")
        assert np.all(np.abs(DV[a:b] - gv) <= tv + ref.HALF_ULP["bf16"] * 1.01 * np.abs(gv))
    m = rng.integers(0, 3, seqs).astype(np.int32)            # as many sequences of one place or two in a store
    rows = 2 * seqs
    codes, scales = (t.view(torch.uint8) for t in mm.cache_new((rows, 1), 16, block=16))
    codes.copy_(torch.from_numpy(rng.integers(0, 0x70, (rows, 1, 16)).astype(np.uint8)))
    store = codes.view(torch.float8_e4m3fn), scales
    table = torch.arange(rows, device="cuda").int().view(seqs, 2)
    w = torch.zeros(seqs, 2, device="cuda")
    x = randn(gen(9), seqs, 1, 16)
    got = mm.cache_attend(x, store, store, table, torch.from_numpy(m).cuda(), block=16, weights=w)
    assert not got[torch.from_numpy(m == 0).cuda()].any()
    assert torch.allclose(w.sum(1), torch.from_numpy((m > 0).astype(np.float32)).cuda(), atol=2.0 ** -20)
    new, _, kept = mm.cache_evict([store], table, torch.from_numpy(m).cuda(), w, 1, block=16)
    assert np.array_equal(new.cpu().numpy(), np.minimum(m, 1))
    best = np.where(m == 0, -1, np.where((m == 2) & (f64(w)[:, 1] > f64(w)[:, 0]), 1, 0))
    assert np.array_equal(kept[:, 0].cpu().numpy(), best)


def test_wide_tables_and_odd_pages(mm):  # noqa: F811
    """A table far wider than the sequences, pages that end inside a wave's places, and a
    view of a table's columns."""
    import torch
    rng = np.random.default_rng(11)
    pages, table, rows = lay_out(rng, [37, 5, 0], 7, columns=3000)
    k, v = (make_store(rng, pages, 7, 64, 32, "i8") for _ in range(2))
    for r in rows:
        fill(rng, k, r, "i8")
        fill(rng, v, r, "i8")
    keys, values = to_gpu(k, pages, 7, "i8"), to_gpu(v, pages, 7, "i8")
    table, lens = torch.from_numpy(table).cuda(), torch.tensor([37, 5, 0], device="cuda").int()
    q = torch.randn(3, 4, 32, device="cuda")
    w = torch.zeros(3, 3000 * 7, device="cuda")
    wide = mm.cache_attend(q, keys, values, table, lens, block=32, weights=w)
    narrow = mm.cache_attend(q, keys, values, table[:, :6], lens, block=32)
    assert torch.allclose(wide, narrow, rtol=2.0 ** -18, atol=2.0 ** -18)
    assert not w[:, 37:].any() and torch.allclose(w.sum(1), torch.tensor([4.0, 4.0, 0.0], device="cuda"), atol=1e-5)
    new, w2, kept = mm.cache_evict((keys, values), table, lens, w, 10, recent=2, block=32)
    assert new.tolist() == [10, 5, 0] and kept[0].tolist() == ref.evict(f64(w[0]), 37, 10, 2)
