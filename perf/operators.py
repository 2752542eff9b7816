"""Cases of the block-scaled 8-bit operators: what is measured, their plain
forms in elementary torch operations, and their definition in 64 bits.

Five operators share one code format: E4M3 (or int8) codes with one
power-of-two scale, an E8M0 byte, for each block of values.

  encode        rows of numbers to codes and scales (along rows, along columns
                transposed, or in 128 x 128 tiles)
  matmul        product of two code matrices, fp32 sums
  linear        y = x w^T with both sides encoded; for serving with w kept as
                codes, for training with the gradients of x and w
  cache_write   rows encoded into the slots of a store
  cache_read    rows of a store decoded, by slot or through a page table

The scale of a block whose largest finite magnitude is a: the smallest power
of two s = 2^e with a <= L s (L = 448 for E4M3, 127 for int8), e clamped to
[-127, 127], s = 1 where a = 0. A code is the nearest representable value of
x / s, ties to even, saturating at +-L.
"""
import math

import torch

own = False  # True: run() calls the framework's operators

BLOCK = 128
TOP = {"f8": 448.0, "i8": 127.0}
CODE = {"f8": torch.float8_e4m3fn, "i8": torch.int8}
NUM = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # embeddings of odd width, encoded as they arrive
        dict(name="encode_f32_1237x769", op="encode", n=1237, d=769, dtype="f32", form="rows"),
        # activations of a training step: both orders from one read
        dict(name="encode_bf16_16384x4096_both", op="encode", n=16384, d=4096, dtype="bf16",
             form="both"),
        # an odd batch of embeddings scored against 4096 centroids
        dict(name="matmul_4099x4096x768", op="matmul", m=4099, n=4096, k=768, bscale="rows",
             out="f32"),
        # a few queries scored against every row of a store of short vectors
        dict(name="matmul_16x200003x128", op="matmul", m=16, n=200003, k=128, bscale="rows",
             out="f32"),
        # a large product, weights in tiles: matrix rate
        dict(name="matmul_8192x8192x8192", op="matmul", m=8192, n=8192, k=8192, bscale="tiles",
             out="bf16"),
        # one token through a projection: latency and the weight's bytes
        dict(name="linear_serve_1x4096x4096", op="serve", m=1, n=4096, k=4096, dtype="bf16"),
        # a training step of a small head with odd sizes, fp32
        dict(name="linear_train_777x1000x768", op="train", m=777, n=1000, k=768, dtype="f32"),
        # a training step of a projection
        dict(name="linear_train_8192x4096x4096", op="train", m=8192, n=4096, k=4096, dtype="bf16"),
        # one step of serving: a few tokens' keys and values, heads of 96, int8
        dict(name="cache_write_33x16x96_i8", op="write", rows=4096, n=33, heads=16, width=96,
             block=96, fmt="i8", dtype="f16"),
        # a prompt's keys and values, heads of 128, scattered over the store
        dict(name="cache_write_32768x16x128_f8", op="write", rows=65536, n=32768, heads=16,
             width=128, block=128, fmt="f8", dtype="bf16"),
        # a batch of stored embeddings for a clustering step, by row id
        dict(name="cache_read_65536x768_f32", op="read", rows=262144, n=65536, d=768, block=128,
             fmt="f8", out="f32"),
        # ragged sequences through a page table, empty ones among them
        dict(name="cache_read_pages_33x4000x2048", op="pages", seqs=33, longest=4000, page=16,
             d=2048, block=128, fmt="f8", out="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["encode", "matmul", "matmul", "serve", "train", "write", "read", "pages"])
    number = rng.choice(["f32", "bf16", "f16"])
    if op == "encode":
        return dict(op=op, n=_log(rng, 1, 16384), d=_log(rng, 16, 4096), dtype=number,
                    form=rng.choice(["rows", "both", "tiles"]))
    if op == "matmul":
        return dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 64, 8192), k=_log(rng, 96, 8192),
                    bscale=rng.choice(["rows", "tiles"]), out=number)
    if op == "serve":
        return dict(op=op, m=_log(rng, 1, 256), n=_log(rng, 256, 16384), k=_log(rng, 256, 8192),
                    dtype=number)
    if op == "train":
        return dict(op=op, m=_log(rng, 64, 8192), n=_log(rng, 128, 4096), k=_log(rng, 128, 4096),
                    dtype=number)
    fmt = rng.choice(["f8", "i8"])
    if op == "write":
        width = rng.choice([64, 80, 96, 112, 128])
        n = _log(rng, 1, 32768)
        return dict(op=op, rows=n + _log(rng, 1, 32768), n=n, heads=rng.randint(1, 16),
                    width=width, block=width, fmt=fmt, dtype=number)
    if op == "read":
        n = _log(rng, 1, 65536)
        return dict(op=op, rows=_log(rng, 64, 262144), n=n, d=_log(rng, 32, 1024),
                    block=rng.choice([32, 64, 96, 128]), fmt=fmt, out=number)
    return dict(op=op, seqs=rng.randint(1, 48), longest=_log(rng, 1, 4000),
                page=rng.choice([1, 16, 24, 64]), d=rng.choice([576, 1000, 1024, 2048]),
                block=rng.choice([64, 128]), fmt=fmt, out=number)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _numbers(n, d, dtype, g, spread=1.0):
    """Hidden states: normal values, row by row of another size, a few large
    columns, as activations have."""
    x = torch.randn(n, d, device="cuda", generator=g)
    x *= torch.exp(0.5 * torch.randn(n, 1, device="cuda", generator=g)) * spread
    x *= torch.where(torch.rand(1, d, device="cuda", generator=g) < 0.01, 12.0, 1.0)
    return x.to(NUM[dtype])


def _pitched(t, unit):
    """t with rows that start a multiple of `unit` bytes apart (1-byte values)."""
    n, d = t.shape
    pitch = -(-d // unit) * unit
    if pitch == d:
        return t
    room = torch.zeros(n, pitch, device=t.device, dtype=torch.uint8)
    room[:, :d] = t.view(torch.uint8)
    return room.view(t.dtype)[:, :d]


def _code_matrix(n, d, g, tiles=False, spread=1.0):
    codes, scales = _plain_encode(_numbers(n, d, "f32", g, spread), "tiles" if tiles else "rows")
    return _pitched(codes, 16), _pitched(scales, 4)


def _store(rows, d, block, fmt, g):
    codes = torch.empty(rows, d, device="cuda", dtype=CODE[fmt])
    scales = torch.empty(rows, -(-d // block), device="cuda", dtype=torch.float8_e8m0fnu)
    at = 0
    while at < rows:  # in pieces: a store is larger than its rows in fp32 should be at once
        m = min(rows - at, 65536)
        x = _numbers(m, d, "f32", g)
        c, s = _plain_blocks(x, block, fmt)
        codes[at:at + m], scales[at:at + m] = c, s
        at += m
    return codes, scales


def _lengths(case):
    """Lengths of the ragged sequences, 0 and the longest among them, whose
    order the seed gives."""
    n, most = case["seqs"], case["longest"]
    return [most] + [0] * (n > 2) + [int(most * (i * 0.6180339887 % 1.0))
                                     for i in range(1, n - (n > 2))]


def prepare(case, seed):
    g = _generator(seed)
    c, op = case, case["op"]
    s = dict(case=case)
    if op == "encode":
        s["x"] = _numbers(c["n"], c["d"], c["dtype"], g)
    elif op == "matmul":
        s["a"], s["a_scales"] = _code_matrix(c["m"], c["k"], g)
        s["b"], s["b_scales"] = _code_matrix(c["n"], c["k"], g, c["bscale"] == "tiles",
                                             c["k"] ** -0.5)
    elif op == "serve":
        s["x"] = _numbers(c["m"], c["k"], c["dtype"], g)
        s["w"], s["w_scales"] = _code_matrix(c["n"], c["k"], g, True, c["k"] ** -0.5)
    elif op == "train":
        s["x"] = _numbers(c["m"], c["k"], c["dtype"], g).requires_grad_()
        s["w"] = _numbers(c["n"], c["k"], c["dtype"], g, c["k"] ** -0.5).requires_grad_()
        s["dy"] = _numbers(c["m"], c["n"], c["dtype"], g, 0.01)
    elif op == "write":
        # the keys and values are the tail of a wider row, as a fused projection leaves them
        d = c["heads"] * c["width"]
        wide = _numbers(c["n"], d + 256, c["dtype"], g)
        s["x"] = wide[:, 256:].unflatten(1, (c["heads"], c["width"]))
        s["slots"] = torch.randperm(c["rows"], device="cuda", generator=g)[:c["n"]]
        s["slots"][torch.rand(c["n"], device="cuda", generator=g) < 0.02] = -1
        s["codes"] = torch.zeros(c["rows"], d, device="cuda", dtype=CODE[c["fmt"]])
        s["scales"] = torch.full((c["rows"], -(-d // c["block"])), 127, device="cuda",
                                 dtype=torch.uint8).view(torch.float8_e8m0fnu)
    elif op == "read":
        s["codes"], s["scales"] = _store(c["rows"], c["d"], c["block"], c["fmt"], g)
        s["slots"] = torch.randint(0, c["rows"], (c["n"],), device="cuda", generator=g,
                                   dtype=torch.int32)
    else:
        lengths = torch.tensor(_lengths(c), device="cuda")
        lengths = lengths[torch.randperm(c["seqs"], device="cuda", generator=g)]
        used = -(-lengths // c["page"])
        most = int(used.max())
        pages = int(used.sum()) + 7
        order = torch.randperm(pages, device="cuda", generator=g).int()
        first = torch.cumsum(used, 0) - used
        at = torch.arange(most, device="cuda")
        s["table"] = torch.where(at < used[:, None],
                                 order[(first[:, None] + at).clamp(max=pages - 1)], -1)
        s["starts"] = torch.cat([lengths.new_zeros(1), torch.cumsum(lengths, 0)]).int()
        s["total"] = int(lengths.sum())
        codes, scales = _store(pages * c["page"], c["d"], c["block"], c["fmt"], g)
        s["codes"] = codes.view(pages, c["page"], -1)
        s["scales"] = scales.view(pages, c["page"], -1)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import mini_means_amd as em
    c, op = s["case"], s["case"]["op"]
    if op == "encode":
        return em.block_encode(s["x"], tiles=c["form"] == "tiles", cols=c["form"] != "rows")
    if op == "matmul":
        return em.block_matmul(s["a"], s["a_scales"], s["b"], s["b_scales"],
                               out_dtype=NUM[c["out"]])
    if op == "serve":
        return em.block_linear(s["x"], (s["w"], s["w_scales"]))
    if op == "train":
        y = em.block_linear(s["x"], s["w"])
        return y.detach(), *torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])
    if op == "write":
        em.cache_write(s["x"], s["slots"], s["codes"], s["scales"], block=c["block"])
        return s["codes"], s["scales"]
    if op == "read":
        return em.cache_read(s["codes"], s["scales"], s["slots"], block=c["block"],
                             out_dtype=NUM[c["out"]])
    return em.cache_read_pages(s["codes"], s["scales"], s["table"], s["starts"], s["total"],
                               block=c["block"], out_dtype=NUM[c["out"]])


def _exponent(a, top):
    """The smallest e with a <= top 2^e, in [-127, 127]; 0 where a is 0."""
    m, e = torch.frexp(a)
    mt, et = math.frexp(top)
    e = e - et + (m > mt).to(e.dtype)
    return torch.where(a > 0, e.clamp(-127, 127), 0)


def _round_codes(y, fmt):
    y = y.clamp(-TOP[fmt], TOP[fmt])
    return torch.round(y).nan_to_num(0.0).to(torch.int8) if fmt == "i8" \
        else y.to(torch.float8_e4m3fn)


def _e8m0(e):
    return (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _finite_abs(x):
    return torch.where(torch.isfinite(x), x.abs(), 0.0)


def _plain_blocks(x, block, fmt="f8"):
    """Codes and scales of the rows of x (fp32), blocks along the row."""
    n, d = x.shape
    nb = -(-d // block)
    p = torch.nn.functional.pad(x, (0, nb * block - d)).view(n, nb, block)
    e = _exponent(_finite_abs(p).amax(2), TOP[fmt])
    y = p * torch.exp2(-e.float())[:, :, None]
    return _round_codes(y, fmt).view(n, nb * block)[:, :d], _e8m0(e)


def _plain_tiles(x):
    n, d = x.shape
    nb, db = -(-n // BLOCK), -(-d // BLOCK)
    p = torch.nn.functional.pad(x, (0, db * BLOCK - d, 0, nb * BLOCK - n))
    p = p.view(nb, BLOCK, db, BLOCK)
    e = _exponent(_finite_abs(p).amax((1, 3)), TOP["f8"])
    y = p * torch.exp2(-e.float())[:, None, :, None]
    return _round_codes(y, "f8").view(nb * BLOCK, db * BLOCK)[:n, :d], _e8m0(e)


def _plain_encode(x, form):
    x = x.float()
    if form == "tiles":
        return _plain_tiles(x)
    if form == "rows":
        return _plain_blocks(x, BLOCK)
    return *_plain_blocks(x, BLOCK), *_plain_blocks(x.t().contiguous(), BLOCK)


def _plain_values(codes, scales, block):
    """fp32 values of codes whose scales stand per row and block, or per tile."""
    n, d = codes.shape
    f = torch.exp2(scales.view(torch.uint8).float() - 127.0)
    f = f.repeat_interleave(block, 1)[:, :d]
    if f.shape[0] != n:
        f = f.repeat_interleave(BLOCK, 0)[:n]
    return codes.float() * f


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "encode":
        if c["form"] != "tiles":
            return _plain_encode(s["x"], c["form"])
        codes, scales = _plain_encode(s["x"], "tiles")
        return codes, scales, codes.view(torch.uint8).t().contiguous().view(codes.dtype), \
            scales.view(torch.uint8).t().contiguous().view(scales.dtype)
    if op == "matmul":
        a = _plain_values(s["a"], s["a_scales"], BLOCK)
        b = _plain_values(s["b"], s["b_scales"], BLOCK)
        return (a @ b.t()).to(NUM[c["out"]])
    if op == "serve":
        x = _plain_values(*_plain_encode(s["x"], "rows"), BLOCK)
        return (x @ _plain_values(s["w"], s["w_scales"], BLOCK).t()).to(s["x"].dtype)
    if op == "train":
        with torch.no_grad():
            x, w, dy = s["x"].detach(), s["w"].detach(), s["dy"]
            xr, xs, xc, xcs = _plain_encode(x, "both")
            gr, gs, gc, gcs = _plain_encode(dy, "both")
            qw = _plain_values(*_plain_encode(w, "tiles"), BLOCK)
            y = _plain_values(xr, xs, BLOCK) @ qw.t()
            dx = _plain_values(gr, gs, BLOCK) @ qw
            dw = _plain_values(gc, gcs, BLOCK) @ _plain_values(xc, xcs, BLOCK).t()
            return y.to(x.dtype), dx.to(x.dtype), dw.to(w.dtype)
    if op == "write":
        codes, scales = _plain_blocks(s["x"].float().flatten(1), c["block"], c["fmt"])
        keep = s["slots"] >= 0
        at = s["slots"][keep]
        s["codes"].view(torch.uint8)[at] = codes.view(torch.uint8)[keep]
        s["scales"].view(torch.uint8)[at] = scales.view(torch.uint8)[keep]
        return s["codes"], s["scales"]
    codes, scales = s["codes"].flatten(0, -2), s["scales"].flatten(0, -2)
    if op == "read":
        at = s["slots"].long()
    else:
        starts = s["starts"].long()
        i = torch.arange(s["total"], device="cuda")
        seq = torch.searchsorted(starts, i, right=True) - 1
        pos = i - starts[seq]
        at = s["table"].long()[seq, pos // c["page"]] * c["page"] + pos % c["page"]
    rows = codes.view(torch.uint8)[at].view(codes.dtype)
    factors = scales.view(torch.uint8)[at].view(scales.dtype)
    return _plain_values(rows, factors, c["block"]).to(NUM[c["out"]])


# --------------------------------------------------------------------------
# the bytes and operations that a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    c, op = case, case["op"]

    def blocks(n, d, b=BLOCK):
        return n * -(-d // b)

    if op == "encode":
        n, d = c["n"], c["d"]
        forms = 1 if c["form"] == "rows" else 2
        scales = blocks(n, d) if c["form"] == "rows" else blocks(n, d) + blocks(d, n)
        if c["form"] == "tiles":
            scales = 2 * -(-n // BLOCK) * -(-d // BLOCK)
        return dict(bytes=n * d * (SIZE[c["dtype"]] + forms) + scales, flops=2 * n * d)
    if op == "matmul":
        m, n, k = c["m"], c["n"], c["k"]
        scales = blocks(m, k) + (blocks(n, k) if c["bscale"] == "rows" else
                                 -(-n // BLOCK) * -(-k // BLOCK))
        return dict(bytes=(m + n) * k + scales + m * n * SIZE[c["out"]], flops=2 * m * n * k)
    if op == "serve":
        m, n, k = c["m"], c["n"], c["k"]
        return dict(bytes=n * k + -(-n // BLOCK) * -(-k // BLOCK)
                    + (m * k + m * n) * SIZE[c["dtype"]], flops=2 * m * n * k)
    if op == "train":  # x, w and dy read, y, dx and dw written
        m, n, k = c["m"], c["n"], c["k"]
        return dict(bytes=2 * (m * k + n * k + m * n) * SIZE[c["dtype"]], flops=6 * m * n * k)
    if op == "write":
        d = c["heads"] * c["width"]
        return dict(bytes=c["n"] * (d * (SIZE[c["dtype"]] + 1) + -(-d // c["block"]) + 8),
                    flops=2 * c["n"] * d)
    rows = c["n"] if op == "read" else sum(_lengths(c))
    return dict(bytes=rows * (c["d"] * (1 + SIZE[c["out"]]) + -(-c["d"] // c["block"]) + 4),
                flops=rows * c["d"])


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def _exact_grid(x, factor, fmt):
    """Nearest code value of x / factor, ties to even, saturating."""
    y = x / factor
    if fmt == "i8":
        return torch.round(y).clamp(-127, 127)
    size = y.abs().clamp(min=2.0 ** -6, max=448.0)
    step = torch.exp2(torch.floor(torch.log2(size)) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _exact_factor(a, top):
    """The smallest power of two s >= 2^-127 with a <= top s; 1 where a is 0."""
    s = torch.exp2(torch.ceil(torch.log2(a / top)).clamp(-127, 127))
    s = torch.where((s > 2.0 ** -127) & (a <= top * s / 2), s / 2, s)
    s = torch.where(a > top * s, s * 2, s)
    return torch.where(a > 0, s, 1.0)


def _exact_blocks(x, block, axis, fmt="f8"):
    """Code values and the factor of every value; blocks along `axis` of the
    2-D x, or tiles where axis is None."""
    n, d = x.shape
    big = torch.empty_like(x)
    for i in range(0, n, n if axis == 1 else block):
        for j in range(0, d, d if axis == 0 else block):
            part = x[i:(n if axis == 1 else i + block), j:(d if axis == 0 else j + block)]
            m = part.abs().amax() if axis is None else part.abs().amax(axis, keepdim=True)
            big[i:i + part.shape[0], j:j + part.shape[1]] = _exact_factor(m, TOP[fmt])
    return _exact_grid(x, big, fmt), big


def _exact_values(codes, scales):
    """64-bit values of a code matrix given with its scales."""
    n, d = codes.shape
    f = torch.pow(2.0, scales.view(torch.uint8).double() - 127)
    rows = torch.arange(n, device="cuda")
    if f.shape[0] != n:
        rows = rows // BLOCK
    return codes.double() * f[rows][:, torch.arange(d, device="cuda") // BLOCK]


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "encode":
        x = s["x"].double()
        if c["form"] == "tiles":
            v, f = _exact_blocks(x, BLOCK, None)
            f = f[::BLOCK, ::BLOCK]
            return v, f, v.t(), f.t()
        v, f = _exact_blocks(x, BLOCK, 1)
        if c["form"] == "rows":
            return v, f[:, ::BLOCK]
        vt, ft = _exact_blocks(x, BLOCK, 0)
        return v, f[:, ::BLOCK], vt.t(), ft[::BLOCK].t()
    if op == "matmul":
        return _exact_values(s["a"], s["a_scales"]) @ _exact_values(s["b"], s["b_scales"]).t()
    if op == "serve":
        v, f = _exact_blocks(s["x"].double(), BLOCK, 1)
        return (v * f) @ _exact_values(s["w"], s["w_scales"]).t()
    if op == "train":
        x, w, dy = (s[name].detach().double() for name in ("x", "w", "dy"))

        def q(t, axis):
            v, f = _exact_blocks(t, BLOCK, axis)
            return v * f
        return q(x, 1) @ q(w, None).t(), q(dy, 1) @ q(w, None), q(dy, 0).t() @ q(x, 0)
    if op == "write":
        v, f = _exact_blocks(s["x"].double().flatten(1), c["block"], 1, c["fmt"])
        f = f[:, ::c["block"]]
        codes = torch.zeros(c["rows"], v.shape[1], device="cuda", dtype=torch.float64)
        factors = torch.ones(c["rows"], f.shape[1], device="cuda", dtype=torch.float64)
        for source, to in ((v, codes), (f, factors)):
            used = s["slots"] >= 0
            to.index_copy_(0, s["slots"][used], source[used])
        return codes.to(torch.int8) if c["fmt"] == "i8" else codes, factors
    if op == "read":
        at = s["slots"].tolist()
    else:
        starts, table = s["starts"].tolist(), s["table"].tolist()
        at = [table[q][p // c["page"]] * c["page"] + p % c["page"]
              for q in range(c["seqs"]) for p in range(starts[q + 1] - starts[q])]
    at = torch.tensor(at, device="cuda", dtype=torch.int64)
    codes = torch.index_select(s["codes"].flatten(0, -2).double(), 0, at)
    byte = torch.index_select(s["scales"].flatten(0, -2).view(torch.uint8), 0, at)
    col = torch.arange(c["d"], device="cuda") // c["block"]
    return codes * torch.pow(2.0, byte.double() - 127)[:, col]
