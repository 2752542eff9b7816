"""Block codes without a GPU: the 64-bit reference against the definition, and
every refusal of the C ABI and the binding that precedes device work."""
import numpy as np
import pytest

import mini_means_amd as mm
import block_ref as ref


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(mm.LIB_PATH):
        from mini_means_amd import build
        build.build(verbose=False)
    return mm.lib()


def test_grid_is_nearest_e4m3():
    """grid() against a search of all E4M3 values: nearest, ties to even."""
    v = ref.e4m3_values()
    order = np.argsort(v[:127])                   # the non-negative finite codes
    pos = v[:127][order]
    rng = np.random.default_rng(1)
    y = np.concatenate([pos, (pos[1:] + pos[:-1]) / 2, rng.uniform(0, 460, 2000),
                        np.exp2(rng.uniform(-12, 9, 2000))])
    y = np.concatenate([y, -y])
    for x in y:
        a = abs(x)
        d = np.abs(pos - a)
        near = np.flatnonzero(d == d.min())
        want = near[0] if len(near) == 1 else next(i for i in near if order[i] % 2 == 0)
        assert abs(ref.grid(np.array([x]), "f8")[0]) == pos[want], x


def test_exponent_is_smallest():
    a = np.array([0.0, 448.0, 448.0001, 1e-45, 3.4e38, 1.0, 0.875, 0.8750001, 2.0 ** -120])
    e = ref.exponent(a, 448.0)
    assert e[0] == 0
    for x, q in zip(a[1:], e[1:]):
        assert x <= 448 * 2.0 ** q and (q == -127 or x > 448 * 2.0 ** (q - 1))


FAKE = 4096   # never dereferenced: the checks run before any device work


def _encode(L, **kw):
    a = dict(X=FAKE, dtype=0, n=4, d=200, ldx=200, tiles=0, c=FAKE, ldc=208, s=FAKE, lds=4,
             ct=None, ldct=0, st=None, ldst=0)
    a.update(kw)
    return L.emeans_block_encode(*a.values(), None)


@pytest.mark.parametrize("change,code,word", [
    (dict(n=-1), -1, b"n out of range"), (dict(n=1 << 31), -1, b"n out of range"),
    (dict(d=0), -1, b"d must"), (dict(dtype=2), -2, b"dtype"), (dict(dtype=9), -2, b"dtype"),
    (dict(ldx=199), -1, b"ldx"), (dict(ldc=199), -1, b"ldc"), (dict(lds=1), -1, b"lds"),
    (dict(c=None), -1, b"NULL"), (dict(s=None), -1, b"together"),
    (dict(ct=FAKE), -1, b"together"), (dict(ct=FAKE, st=FAKE, ldct=3, ldst=1), -1, b"ldct"),
    (dict(X=None), -1, b"X must"),
])
def test_encode_refuses(L, change, code, word):
    assert _encode(L, **change) == code
    assert word in L.emeans_last_error()


def _matmul(L, **kw):
    a = dict(A=FAKE, lda=256, As=FAKE, ldas=2, B=FAKE, ldb=256, Bs=FAKE, ldbs=2, tiles=0,
             m=4, n=5, k=200, out=FAKE, ot=0, ldo=5, work=None)
    a.update(kw)
    return L.emeans_block_matmul(*a.values(), None)


@pytest.mark.parametrize("change,code,word", [
    (dict(m=-1), -1, b"m out"), (dict(n=1 << 31), -1, b"n out"), (dict(k=-1), -1, b"k out"),
    (dict(ot=3), -2, b"out_dtype"), (dict(lda=199), -1, b"lda"), (dict(ldas=1), -1, b"ldas"),
    (dict(ldb=10), -1, b"ldb"), (dict(ldbs=0), -1, b"ldbs"), (dict(ldo=4), -1, b"ldo"),
    (dict(A=None), -1, b"NULL"), (dict(Bs=None), -1, b"NULL"), (dict(out=None), -1, b"NULL"),
    (dict(work=8), -1, b"aligned"),
])
def test_matmul_refuses(L, change, code, word):
    assert _matmul(L, **change) == code
    assert word in L.emeans_last_error()


def test_matmul_of_nothing_is_fine(L):
    assert _matmul(L, m=0) == 0 and _matmul(L, n=0, A=None) == 0


def _linear(L, **kw):
    a = dict(X=FAKE, dtype=1, ldx=200, B=FAKE, ldb=256, Bs=FAKE, ldbs=2, tiles=1, m=4, n=5,
             k=200, out=FAKE, ot=0, ldo=5, work=None)
    a.update(kw)
    return L.emeans_block_linear(*a.values(), None)


@pytest.mark.parametrize("change,code,word", [
    (dict(dtype=2), -2, b"dtype"), (dict(ldx=100), -1, b"ldx"), (dict(X=None), -1, b"X must"),
    (dict(work=8), -1, b"aligned"), (dict(ot=5), -2, b"out_dtype"), (dict(B=None), -1, b"NULL"),
])
def test_linear_refuses(L, change, code, word):
    assert _linear(L, **change) == code
    assert word in L.emeans_last_error()


def test_work_sizes(L):
    """Codes and scales of X come on top of the product's own working memory."""
    for m, n, k in ((300, 200, 200), (100, 100, 8192), (40, 256, 1000)):
        own = L.emeans_block_matmul_work(m, n, k)
        assert own % 16 == 0 and own >= 0
        assert L.emeans_block_linear_work(m, n, k) == own + m * (-(-k // 16) * 16
                                                                + -(-(-(-k // 128)) // 4) * 4)
    assert L.emeans_block_linear_work(0, 5, 200) == 0 and L.emeans_block_matmul_work(3, 5, 0) == 0


def test_train_refuses(L):
    def forward(X=FAKE, xt=0, ldx=200, W=FAKE, wt=1, ldw=200, m=4, n=5, k=200, need=3, out=FAKE,
                ot=0, ldo=5, saved=FAKE, work=None):
        return L.emeans_block_train_forward(X, xt, ldx, W, wt, ldw, m, n, k, need, out, ot, ldo,
                                            saved, work, None)

    def gradient(dY=FAKE, t=0, ld=5, saved=FAKE, m=4, n=5, k=200, dX=FAKE, xt=0, ldx=200, dW=FAKE,
                 wt=0, ldw=200, work=None):
        return L.emeans_block_train_gradient(dY, t, ld, saved, m, n, k, dX, xt, ldx, dW, wt, ldw,
                                             work, None)

    for call, cases in (
        (forward, [(dict(m=-1), -1), (dict(n=0), -1), (dict(k=0), -1), (dict(xt=2), -2),
                   (dict(wt=3), -2), (dict(ot=9), -2), (dict(ldx=9), -1), (dict(ldw=9), -1),
                   (dict(ldo=4), -1), (dict(need=4), -1), (dict(saved=None), -1),
                   (dict(saved=8), -1), (dict(work=4), -1), (dict(X=None), -1), (dict(W=None), -1),
                   (dict(out=None), -1)]),
        (gradient, [(dict(t=2), -2), (dict(xt=2), -2), (dict(wt=5), -2), (dict(ld=4), -1),
                    (dict(ldx=9), -1), (dict(ldw=9), -1), (dict(dX=None, dW=None), -1),
                    (dict(dY=None), -1), (dict(saved=None), -1), (dict(work=8), -1),
                    (dict(n=0), -1), (dict(m=1 << 31), -1)])):
        for change, code in cases:
            assert call(**change) == code, (call, change)
            assert L.emeans_last_error() and b"device" not in L.emeans_last_error()
    assert forward(m=0) == 0 and gradient(m=0, dW=None) == 0
    assert L.emeans_block_train_saved(300, 200, 130) > 2 * 130 * 200
    assert L.emeans_block_train_saved(0, 5, 5) == L.emeans_block_train_work(5, 5, 0, 1) == 0


def _write(L, **kw):
    a = dict(X=FAKE, dtype=0, n=3, heads=2, width=96, rs=192, hs=96, slots=FAKE, sb=4, c=FAKE,
             s=FAKE, rows=10, block=96, fmt=3)
    a.update(kw)
    return L.emeans_cache_write(*a.values(), None)


@pytest.mark.parametrize("change,code,word", [
    (dict(n=-1), -1, b"n out"), (dict(dtype=3), -2, b"dtype"), (dict(heads=0), -1, b"heads"),
    (dict(width=0), -1, b"width"), (dict(rows=-1), -1, b"rows"), (dict(block=0), -1, b"block"),
    (dict(block=40), -1, b"block"), (dict(block=272), -1, b"block"), (dict(fmt=0), -2, b"fmt"),
    (dict(rs=-1), -1, b"strides"), (dict(sb=2), -1, b"slot_bytes"),
    (dict(hs=128, block=64), -1, b"multiple of block"), (dict(c=None), -1, b"NULL"),
    (dict(X=None), -1, b"NULL"), (dict(slots=None), -1, b"NULL"),
    (dict(heads=1 << 20, width=1 << 20), -1, b"d out of range"),
])
def test_cache_write_refuses(L, change, code, word):
    assert _write(L, **change) == code
    assert word in L.emeans_last_error()


def _read(L, **kw):
    a = dict(c=FAKE, s=FAKE, rows=10, d=100, block=32, fmt=2, slots=FAKE, sb=8, n=3, out=FAKE,
             ot=1, ldo=100)
    a.update(kw)
    return L.emeans_cache_read(*a.values(), None)


@pytest.mark.parametrize("change,code,word", [
    (dict(d=0), -1, b"d out"), (dict(block=8), -1, b"block"), (dict(fmt=1), -2, b"fmt"),
    (dict(sb=1), -1, b"slot_bytes"), (dict(n=-2), -1, b"n out"), (dict(ot=2), -2, b"out_dtype"),
    (dict(ldo=99), -1, b"ldo"), (dict(slots=None), -1, b"slots"), (dict(out=None), -1, b"out"),
    (dict(s=None), -1, b"NULL"),
])
def test_cache_read_refuses(L, change, code, word):
    assert _read(L, **change) == code
    assert word in L.emeans_last_error()


def _pages(L, **kw):
    a = dict(c=FAKE, s=FAKE, pages=10, page=16, d=100, block=32, fmt=2, table=FAKE, ldt=4, tp=4,
             starts=FAKE, seqs=2, n=3, out=FAKE, ot=1, ldo=100)
    a.update(kw)
    return L.emeans_cache_read_pages(*a.values(), None)


@pytest.mark.parametrize("change,code,word", [
    (dict(page=0), -1, b"page_rows"), (dict(pages=-1), -1, b"pages"), (dict(seqs=-1), -1, b"seqs"),
    (dict(ldt=3), -1, b"table_ld"), (dict(tp=-1), -1, b"table_pages"),
    (dict(table=None), -1, b"table"), (dict(starts=None), -1, b"starts"),
    (dict(ldo=0), -1, b"ldo"), (dict(pages=(1 << 31) - 1, page=1 << 20), -1, b"rows"),
])
def test_cache_read_pages_refuses(L, change, code, word):
    assert _pages(L, **change) == code
    assert word in L.emeans_last_error()


def test_host_memory_is_refused(L):
    x = np.zeros((4, 256), np.float32)
    assert _encode(L, X=x.ctypes.data) == -5
    assert _matmul(L, A=x.ctypes.data) == -5


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 128)
    c = torch.zeros(4, 128, dtype=torch.float8_e4m3fn)
    s = torch.zeros(4, 1, dtype=torch.uint8)
    i = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: mm.block_encode(x), lambda: mm.block_matmul(c, s, c, s),
                 lambda: mm.block_linear(x, (c, s)), lambda: mm.cache_write(x, i, c, s),
                 lambda: mm.cache_read(c, s, i),
                 lambda: mm.cache_read_pages(c[None], s[None], i[None], i, 3)):
        with pytest.raises(mm.EmeansError, match="ENOTDEVICE"):
            call()


@pytest.mark.parametrize("d", [2 ** 31 - 1023, 2 ** 31 - 1])
def test_rows_too_long_for_their_last_block(L, d):
    """The end of a row's last block has to fit 31 bits; nothing is computed from
    a longer length."""
    assert _encode(L, d=d, ldx=d, ldc=d, lds=d) == -1 and b"d out" in L.emeans_last_error()
    assert _matmul(L, k=d, lda=d, ldb=d, ldas=d, ldbs=d) == -1 and b"k out" in L.emeans_last_error()
    assert L.emeans_block_matmul_work(4, 5, d) == 0 and L.emeans_block_linear_work(40, 5, d) == 0
    for m, n, k in ((d, 5, 5), (5, d, 5), (5, 5, d)):
        assert L.emeans_block_train_saved(m, n, k) == 0
        assert L.emeans_block_train_work(m, n, k, 0) == L.emeans_block_train_work(m, n, k, 1) == 0


FAR = 2 ** 32 + 128   # 128 in its lower half


def test_lengths_keep_their_upper_bits(L):
    """Lengths past 32 bits are refused by every entry, not taken for what their
    lower half says; so is a block, whose lower half would give the store's rows
    more scales than they have room for."""
    assert _encode(L, d=FAR, ldx=FAR, ldc=FAR, lds=FAR) == -1 and b"d out" in L.emeans_last_error()
    big = dict(k=FAR, ldb=FAR, ldbs=FAR)
    assert _matmul(L, lda=FAR, ldas=FAR, **big) == -1 and b"k out" in L.emeans_last_error()
    assert _linear(L, ldx=FAR, **big) == -1 and b"k out" in L.emeans_last_error()
    assert L.emeans_block_matmul_work(40, 5, FAR) == L.emeans_block_linear_work(40, 5, FAR) == 0
    assert L.emeans_block_train_saved(40, 5, FAR) == 0
    for gradient in (0, 1):
        assert L.emeans_block_train_work(40, 5, FAR, gradient) == 0
    assert L.emeans_block_train_forward(FAKE, 0, FAR, FAKE, 0, FAR, 4, 5, FAR, 3, FAKE, 0, 5, FAKE,
                                        None, None) == -1
    assert b"k out" in L.emeans_last_error()
    assert L.emeans_block_train_gradient(FAKE, 0, 5, FAKE, 4, 5, FAR, FAKE, 0, FAR, FAKE, 0, FAR,
                                         None, None) == -1
    assert b"k out" in L.emeans_last_error()
    for change, word in ((dict(heads=2 ** 32 + 2), b"heads"), (dict(width=2 ** 32 + 96), b"width"),
                         (dict(heads=1, width=FAR, rs=FAR), b"width"),
                         (dict(heads=2 ** 33, width=2 ** 33), b"heads"),
                         (dict(block=2 ** 32 + 96), b"block")):
        assert _write(L, **change) == -1 and word in L.emeans_last_error(), change
    for change, word in ((dict(d=FAR, ldo=FAR), b"d out"), (dict(block=2 ** 32 + 32), b"block")):
        assert _read(L, **change) == -1 and word in L.emeans_last_error(), change
        assert _pages(L, **change) == -1 and word in L.emeans_last_error(), change
    for change, word in ((dict(page=2 ** 32 + 16), b"page_rows"), (dict(seqs=2 ** 32 + 2), b"seqs"),
                         (dict(tp=2 ** 32 + 4, ldt=2 ** 33), b"table_pages")):
        assert _pages(L, **change) == -1 and word in L.emeans_last_error(), change


def test_saved_size_by_need(L):
    """X^T comes first, so a forward pass whose x needs no gradient saves that
    alone; the gradient pass with dX = NULL reads no more."""
    m, n, k = 300, 200, 130
    whole, x = L.emeans_block_train_saved(m, n, k), 130 * 304 + 130 * 4
    assert [L.emeans_block_train_saved_for(m, n, k, need) for need in range(4)] \
        == [0, whole, -(-x // 16) * 16, whole]
    assert L.emeans_block_train_saved_for(0, n, k, 2) == L.emeans_block_train_saved_for(m, n, k, 4) == 0
    assert L.emeans_block_train_saved_for(m, n, FAR, 2) == 0
