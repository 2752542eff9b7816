"""Attention around the store without a GPU: the 64-bit references against each
other, and every refusal of the C ABI and the binding that precedes device work."""
import ctypes

import numpy as np
import pytest

import attention_ref as ref
import mini_means_amd as mm


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(mm.LIB_PATH):
        from mini_means_amd import build
        build.build(verbose=False)
    return mm.lib()


def test_rotation_is_a_complex_product_and_goes_back():
    rng = np.random.default_rng(1)
    y, pos, f = rng.normal(size=(5, 3, 20)), rng.integers(0, 10 ** 6, 5), 10.0 ** -np.arange(8.0)
    z = (y[..., :8] + 1j * y[..., 8:16]) * np.exp(1j * pos[:, None] * f)[:, None]
    got, size = ref.turn(y, pos, f)
    assert np.allclose(got, np.concatenate([z.real, z.imag, y[..., 16:]], -1), atol=1e-12)
    assert np.all(np.abs(got) <= size + 1e-12)
    assert np.allclose(ref.turn(got, pos, f, back=True)[0], y, atol=1e-12)


def test_rotation_gradients_are_differences():
    rng = np.random.default_rng(2)
    x, g, dy = rng.normal(size=(2, 3, 12)), rng.normal(size=12), rng.normal(size=(2, 3, 12))
    pos, f = np.array([3, 900]), np.array([1.0, 0.1, 0.01, 0.5])
    dx, _, dg, _ = ref.rotate_grad(x, g, pos, f, dy)
    loss = lambda a, b: (ref.rotate(a, b, pos, f)[0] * dy).sum()  # noqa: E731
    for t, d in ((x, dx), (g, dg)):
        for i in np.ndindex(*t.shape):
            e = np.zeros_like(t)
            e[i] = 1e-5
            ends = [loss(x + e, g) - loss(x - e, g)] if t is x else [loss(x, g + e) - loss(x, g - e)]
            assert abs(ends[0] / 2e-5 - d[i]) < 1e-7


def test_softmax_of_nothing_and_of_masked_rows():
    assert ref.softmax(np.zeros((2, 0))).shape == (2, 0)
    assert not ref.softmax(np.full((2, 3), -np.inf)).any()
    assert ref.evict(np.array([1, 2, 2, 0, 5.0]), 5, 3, 1) == [1, 2, 4]
    assert ref.evict(np.array([1, np.nan, 2]), 3, 2, 0) == [0, 2]


FAKE = 4096   # never dereferenced: the checks run before any device work


def _rotate(L, **kw):
    a = dict(q=FAKE, qr=512, qh=64, k=FAKE, kr=512, kh=64, dt=1, n=3, hq=4, hk=2, w=64, gq=FAKE, gk=FAKE,
             gt=0, pos=FAKE, pb=8, f=FAKE, half=32, eps=1e-6, qo=FAKE, ko=FAKE)
    a.update(kw)
    return L.emeans_norm_rotate(*a.values(), None)


def _rotate_back(L, **kw):
    a = dict(q=FAKE, qr=512, qh=64, k=FAKE, kr=512, kh=64, dt=1, n=3, hq=4, hk=2, w=64, gq=FAKE, gk=FAKE,
             gt=0, pos=FAKE, pb=8, f=FAKE, half=32, eps=1e-6, dq=FAKE, dqr=1, dqh=1, dk=FAKE, dkr=1, dkh=1,
             qo=FAKE, ko=FAKE, dgq=FAKE, dgk=FAKE, work=None)
    a.update(kw)
    return L.emeans_norm_rotate_gradient(*a.values(), None)


ROTATE = [
    (dict(n=-1), -1, b"n out"), (dict(n=1 << 31), -1, b"n out"), (dict(dt=3), -2, b"dtype"),
    (dict(gt=9), -2, b"weight_dtype"), (dict(hq=0), -1, b"hq"), (dict(hk=1 << 20), -1, b"hk"),
    (dict(w=12), -1, b"width"), (dict(w=264), -1, b"width"), (dict(w=2 ** 32 + 64), -1, b"width"),
    (dict(half=36), -1, b"half"), (dict(half=6), -1, b"half"), (dict(half=-4), -1, b"half"),
    (dict(pb=2), -1, b"position_bytes"), (dict(eps=-1.0), -1, b"eps"), (dict(eps=float("nan")), -1, b"eps"),
    (dict(qr=-1), -1, b"strides"), (dict(kh=-1), -1, b"strides"), (dict(q=None), -1, b"NULL"),
    (dict(gk=None), -1, b"NULL"), (dict(f=None), -1, b"NULL"), (dict(ko=None), -1, b"NULL")]


@pytest.mark.parametrize("change,code,word", ROTATE)
def test_norm_rotate_refuses(L, change, code, word):
    more = {} if "dq" in change else {"dq": FAKE}
    assert _rotate(L, **change) == code and word in L.emeans_last_error()
    assert _rotate_back(L, **change, **more) == code


@pytest.mark.parametrize("change,word", [
    (dict(dq=None), b"dq_out"), (dict(dk=None), b"dk_out"), (dict(dgq=None), b"dq_weight"),
    (dict(dkr=-1), b"strides"), (dict(work=8), b"aligned")])
def test_norm_rotate_gradient_refuses(L, change, word):
    assert _rotate_back(L, **change) == -1 and word in L.emeans_last_error()


def _attend(L, **kw):
    a = dict(q=FAKE, dt=1, qr=512, qh=64, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, pages=10, page=16, block=64,
             fmt=3, table=FAKE, ld=4, tp=4, lens=FAKE, seqs=3, hq=4, hk=2, w=64, scale=0.1, out=FAKE,
             weights=None, wld=0, work=None)
    a.update(kw)
    return L.emeans_cache_attend(*a.values(), None)


@pytest.mark.parametrize("change,code,word", [
    (dict(dt=2), -2, b"dtype"), (dict(hq=0), -1, b"hq"), (dict(hk=0), -1, b"hk"), (dict(hq=5), -1, b"multiple"),
    (dict(w=72), -1, b"width"), (dict(w=144), -1, b"width"), (dict(w=0), -1, b"width"),
    (dict(page=0), -1, b"page_rows"), (dict(pages=-1), -1, b"pages"), (dict(seqs=-1), -1, b"seqs"),
    (dict(ld=3), -1, b"table_ld"), (dict(tp=-1), -1, b"table_pages"), (dict(tp=1 << 30, ld=1 << 30), -1, b"places"),
    (dict(pages=(1 << 31) - 1, page=1 << 20, tp=1), -1, b"rows"), (dict(block=8), -1, b"block"),
    (dict(fmt=1), -2, b"fmt"), (dict(qr=-1), -1, b"strides"), (dict(scale=float("nan")), -1, b"scale"),
    (dict(weights=FAKE, wld=63), -1, b"weights_ld"), (dict(weights=FAKE, wld=64, hq=2048), -1, b"1024"),
    (dict(work=8), -1, b"aligned"), (dict(q=None), -1, b"NULL"), (dict(out=None), -1, b"NULL"),
    (dict(lens=None), -1, b"NULL"), (dict(table=None), -1, b"NULL"), (dict(vs=None), -1, b"NULL")])
def test_cache_attend_refuses(L, change, code, word):
    assert _attend(L, **change) == code and word in L.emeans_last_error()


def _evict(L, stores=2, codes=FAKE, scales=FAKE, rc=128, rs=1, **kw):
    m = max(stores, 1)
    a = dict(c=(ctypes.c_void_p * m)(*[codes] * m), s=(ctypes.c_void_p * m)(*[scales] * m),
             rc=(ctypes.c_int64 * m)(*[rc] * m), rs=(ctypes.c_int64 * m)(*[rs] * m), m=stores, pages=10, page=16,
             table=FAKE, ld=4, tp=4, lens=FAKE, seqs=3, weights=FAKE, wld=64, keep=32, recent=8, nl=FAKE, nw=FAKE,
             kept=FAKE, work=None)
    a.update(kw)
    return L.emeans_cache_evict(*a.values(), None)


@pytest.mark.parametrize("change,word", [
    (dict(stores=0), b"stores"), (dict(stores=5), b"stores"), (dict(rc=0), b"row_codes"), (dict(rs=0), b"row_scales"),
    (dict(codes=None), b"NULL"), (dict(scales=None), b"NULL"), (dict(page=0), b"page_rows"),
    (dict(keep=-1), b"keep"), (dict(recent=33), b"recent"), (dict(recent=-1), b"recent"), (dict(wld=63), b"weights_ld"),
    (dict(ld=3), b"table_ld"), (dict(seqs=1 << 30, ld=4, rc=10 ** 6), b"too many"), (dict(work=4), b"aligned"),
    (dict(lens=None), b"NULL"), (dict(nl=None), b"NULL"), (dict(nw=None), b"NULL"), (dict(kept=None), b"NULL"),
    (dict(table=None), b"NULL"), (dict(c=None), b"NULL")])
def test_cache_evict_refuses(L, change, word):
    assert _evict(L, **change) == -1 and word in L.emeans_last_error()


def test_cache_evict_refuses_planes_that_overlap(L):
    """Before any device work: in all pairs, by a byte, and none of planes that only touch."""
    size = 10 * 16 * 128                                   # of codes; scales are 10 x 16
    at = [FAKE, FAKE + size, FAKE + size + 160, FAKE + 2 * size + 160]
    planes = lambda c0, s0, c1, s1: dict(c=(ctypes.c_void_p * 2)(c0, c1), s=(ctypes.c_void_p * 2)(s0, s1))  # noqa: E731
    assert _evict(L, **planes(*at)) != 0 and b"overlap" not in L.emeans_last_error()      # no GPU memory
    for i in range(4):
        for j in range(4):
            if i != j:
                same = list(at)
                same[i] = at[j]
                assert _evict(L, **planes(*same)) == -1 and b"overlap" in L.emeans_last_error()
    for i in range(1, 4):
        near = list(at)
        near[i] -= 1
        assert _evict(L, **planes(*near)) == -1 and b"overlap" in L.emeans_last_error()
    _evict(L, pages=0)                                     # a store of no rows has none to overlap
    assert b"overlap" not in L.emeans_last_error()
    # lengths whose product passes 64 bits
    assert _evict(L, **planes(*at), pages=(1 << 31) - 1, page=512, rc=1 << 25, wld=2048) == -1
    assert b"overlap" in L.emeans_last_error()


def test_nothing_to_do_is_fine(L):
    assert _rotate(L, n=0, q=None) == 0 and _attend(L, seqs=0, q=None) == 0 and _evict(L, seqs=0) == 0
    assert L.emeans_cache_evict_work(0, 5) == L.emeans_cache_attend_work(0, 4, 2, 64, 16, 4, 1) == 0
    assert L.emeans_norm_rotate_work(5, 300) == 0
    assert L.emeans_cache_attend_work(2, 4, 3, 64, 16, 4, 1) == 0


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x, g = torch.zeros(4, 2, 64), torch.zeros(64)
    store = (torch.zeros(3, 16, 128, dtype=torch.int8), torch.zeros(3, 16, 1, dtype=torch.uint8))
    table, lens = torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: mm.norm_rotate(x, x, g, g, lens, g.double()),
                 lambda: mm.cache_attend(x, store, store, table, lens),
                 lambda: mm.cache_evict([store], table, lens, torch.zeros(4, 48), 3)):
        with pytest.raises(mm.EmeansError, match="ENOTDEVICE"):
            call()
    with pytest.raises(mm.EmeansError, match="EINVAL"):
        mm.rotary_freqs(12)
    f = mm.rotary_freqs(64, 500.0, device="cpu").numpy()
    assert np.allclose(f, 500.0 ** (-2 * np.arange(32) / 64), rtol=1e-14, atol=0)


# ---- packed sequences ----------------------------------------------------------

def test_attention_gradients_are_differences():
    rng = np.random.default_rng(3)
    for lq, lk, causal in ((5, 5, True), (3, 6, True), (6, 3, True), (4, 5, False)):
        x = [rng.normal(size=(n, 8)) for n in (lq, lk, lk)]
        do = rng.normal(size=(lq, 8))
        grads, _ = ref.attend_grad(*x, do, 0.4, causal, "bf16")
        for i, t in enumerate(x):
            for j in np.ndindex(*t.shape):
                ends = []
                for e in (1e-5, -1e-5):
                    y = [a.copy() for a in x]
                    y[i][j] += e
                    ends.append((ref.attend(*y, 0.4, causal, "bf16")[0] * do).sum())
                assert abs((ends[0] - ends[1]) / 2e-5 - grads[i][j]) < 1e-7


@pytest.mark.parametrize("dtype,sharp", [("bf16", 0.2), ("f16", 0.03)])
def test_slopes_find_wrong_gradients(dtype, sharp):
    """What the GPU's gradients are held against accepts the definition's and finds them 5% too large or
    too small (bf16 25%: every rounding may be as large as it can be), with D left out, of another
    mask, of one head of a group alone."""
    rng = np.random.default_rng(6)
    q, do = rng.normal(size=(90, 2, 64)) * 1.5, rng.normal(size=(90, 2, 64)) * 0.1
    k, v = rng.normal(size=(2, 90, 1, 64))

    def grads(causal=True, heads=(0, 1)):
        out = [np.zeros(t.shape) for t in (q, k, v)]
        for h in heads:
            for o, x, at in zip(out, ref.attend_grad(q[:, h], k[:, 0], v[:, 0], do[:, h], 0.125, causal, dtype, 0.0)[0], (h, 0, 0)):
                o[:, at] += x
        return out

    def fits(g):
        return [abs(a - b) <= off for a, b, off in ref.grad_slopes(q, k, v, do, g, 0.125, True, dtype)]

    right = grads()
    for a, b, off in ref.grad_slopes(q, k, v, do, right, 0.125, True, dtype):
        assert abs(a - b) <= 1e-6 * abs(b) and off <= sharp * abs(b)
    wrong = 0.05 if dtype == "f16" else 0.25
    assert fits([(1 + wrong) * g for g in right]) == [False] * 3
    assert fits([(1 - wrong) * g for g in right]) == [False] * 3
    assert fits(grads(causal=False)) == [False] * 3
    assert fits(grads(heads=(0,)))[1:] == [False] * 2
    without = [np.zeros(t.shape) for t in (q, k)]
    for h in range(2):
        p = ref.softmax(np.where(ref.seen(90, 90, True), q[:, h] @ k[:, 0].T * 0.125, -np.inf))
        ds = p * (do[:, h] @ v[:, 0].T)
        without[0][:, h] += 0.125 * ds @ k[:, 0]
        without[1][:, 0] += 0.125 * ds.T @ q[:, h]
    assert fits([*without, right[2]])[:2] == [False] * 2


def test_attention_of_one_token_is_the_last_row_of_causal_attention():
    rng = np.random.default_rng(4)
    q, k, v = (rng.normal(size=(7, 16)) for _ in range(3))
    full = ref.attend(q, k, v, 0.25, True, "bf16")[0]
    one = ref.decode(q[6:7], k[:, None], v[:, None], 0.25, "bf16")[0]
    assert np.allclose(full[6], one[0], atol=1e-14)
    assert not ref.attend(q, k[:3], v[:3], 0.25, True, "bf16")[0][:4].any()      # no key seen


def _packed(L, **kw):
    a = dict(q=FAKE, qr=256, qh=64, k=FAKE, kr=128, kh=64, v=FAKE, vr=128, vh=64, dt=1, n=10, nk=10, hq=4, hk=2,
             w=64, starts=FAKE, ks=FAKE, seqs=2, causal=1, scale=0.1, out=FAKE, lse=None, rest=None)
    a.update(kw)
    return L.emeans_attend(*a.values(), None)


def _packed_back(L, **kw):
    a = dict(q=FAKE, qr=256, qh=64, k=FAKE, kr=128, kh=64, v=FAKE, vr=128, vh=64, dt=1, n=10, nk=10, hq=4, hk=2,
             w=64, starts=FAKE, ks=FAKE, seqs=2, causal=1, scale=0.1, out=FAKE, lse=FAKE, rest=FAKE, do=FAKE, dr=256,
             dh=64, dq=FAKE, dk=FAKE, dv=FAKE, work=None)
    a.update(kw)
    return L.emeans_attend_gradient(*a.values(), None)


PACKED = [
    (dict(dt=0), -2, b"dtype"), (dict(dt=3), -2, b"dtype"), (dict(n=-1), -1, b"n out"), (dict(nk=1 << 31), -1, b"nk out"),
    (dict(hq=0), -1, b"hq"), (dict(hk=0), -1, b"hk"), (dict(hq=3), -1, b"multiple of hk"), (dict(w=4), -1, b"width"),
    (dict(w=136), -1, b"width"), (dict(w=65), -1, b"width"), (dict(seqs=-1), -1, b"seqs"), (dict(qr=-8), -1, b"strides"),
    (dict(kh=4), -1, b"strides"), (dict(v=FAKE + 8), -1, b"16 bytes"), (dict(out=FAKE + 2), -1, b"16 bytes"),
    (dict(scale=float("inf")), -1, b"scale"), (dict(q=None), -1, b"NULL"), (dict(v=None), -1, b"NULL"),
    (dict(starts=None), -1, b"NULL"), (dict(ks=None), -1, b"NULL"), (dict(out=None), -1, b"NULL")]


@pytest.mark.parametrize("change,code,word", PACKED)
def test_attend_refuses(L, change, code, word):
    assert _packed(L, **change) == code and word in L.emeans_last_error()
    assert _packed_back(L, **change) == code and word in L.emeans_last_error()


@pytest.mark.parametrize("change,word", [
    (dict(lse=None), b"NULL"), (dict(rest=None), b"NULL"), (dict(do=None), b"NULL"), (dict(dq=None), b"NULL"),
    (dict(dk=None), b"NULL"), (dict(dv=None), b"NULL"), (dict(dr=12), b"strides"), (dict(do=FAKE + 8), b"16 bytes"),
    (dict(work=8), b"aligned")])
def test_attend_gradient_refuses(L, change, word):
    assert _packed_back(L, **change) == -1 and word in L.emeans_last_error()


def test_attend_of_nothing_is_fine(L):
    assert _packed(L, n=0, q=None, out=None) == 0 and _packed_back(L, n=0, nk=0, q=None) == 0
    assert L.emeans_attend_work(-1, 5, 4, 2, 64, 1) == 0 and L.emeans_attend_work(10, 10, 4, 2, 64, 1) >= 160


def test_scalar_bases_of_direct_loads_are_waited_for():
    """The shared load into LDS whose address is in scalar registers: a vector instruction may have
    written them right before, and the hardware needs five wait states then, which only the
    asm block itself can give."""
    import glob
    import os
    import re
    found = 0
    for path in glob.glob(os.path.join(os.path.dirname(os.path.abspath(mm.__file__)), "csrc", "common.hpp")):
        with open(path) as f:
            text = f.read()
        for block in re.findall(r'asm volatile\(\s*((?:"[^"]*"\s*)+)', text):
            steps = [s.strip() for s in re.sub(r'"\s*"', "", block).strip('" \n').split(r"\n\t")]
            for i, s in enumerate(steps):
                if "_load_lds_" in s and not s.endswith("off"):
                    found += 1
                    waits = sum(1 + int(x.split()[1]) if x.startswith("s_nop") else 1 for x in steps[:i])
                    assert waits >= 5, (path, steps)
    assert found >= 1
