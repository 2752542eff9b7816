"""Cases of the attention operators around the coded store: what is measured,
their plain forms in elementary torch operations, and their definition in 64 bits.

  rotate   queries and keys normed per head and turned by their positions, in
           one pass; for training with the gradients
  attend   attention over packed prompts of different lengths, grouped heads;
           for training with the gradients
  decode   attention of one new token per sequence over a paged store of 8-bit
           codes, with or without the rows' attention weights added up
  evict    rows of small accumulated weight dropped from a paged store

A store's row is all key-value heads of one token, E4M3 or int8 codes with one
power-of-two scale for each block of values (an E8M0 byte).
"""
import math

import torch

own = False  # True: run() calls the framework's operators

TOP = {"f8": 448.0, "i8": 127.0}
CODE = {"f8": torch.float8_e4m3fn, "i8": torch.int8}
NUM = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one step of serving: a new token of each of five sequences, far into them
        dict(name="rotate_5x32x128", op="rotate", n=5, hq=32, hk=8, width=128, turned=128,
             dtype="bf16", grad=False, far=100000),
        # a whole prompt
        dict(name="rotate_16384x32x128", op="rotate", n=16384, hq=32, hk=8, width=128, turned=128,
             dtype="bf16", grad=False, far=0),
        # a training step of a model with heads of 96, half of each turned
        dict(name="rotate_train_4099x12x96_f32", op="rotate", n=4099, hq=12, hk=4, width=96,
             turned=48, dtype="f32", grad=True, far=0),
        # short texts as an encoder of embeddings takes them: every token sees its whole text
        dict(name="attend_33x500x16x64_f16", op="attend", seqs=33, longest=500, hq=16, hk=16,
             width=64, dtype="f16", causal=False, grad=False, pad=0),
        # one long prompt: matrix rate
        dict(name="attend_1x16384x32x128", op="attend", seqs=1, longest=16384, hq=32, hk=8,
             width=128, dtype="bf16", causal=True, grad=False, pad=0),
        # a training step on packed texts of odd lengths, padded behind the last
        dict(name="attend_train_7x4000x32x128", op="attend", seqs=7, longest=4000, hq=32, hk=8,
             width=128, dtype="bf16", causal=True, grad=True, pad=37),
        # a few short sequences: latency
        dict(name="decode_3x300x16x96_i8", op="decode", seqs=3, longest=300, hq=16, hk=16, width=96,
             page=16, block=96, fmt="i8", dtype="f16", weights=False),
        # one sequence at full length: the card's bandwidth from a single row
        dict(name="decode_1x131072x32x128", op="decode", seqs=1, longest=131072, hq=32, hk=8,
             width=128, page=64, block=128, fmt="f8", dtype="bf16", weights=False),
        # a serving batch of ragged sequences
        dict(name="decode_64x8192x32x128", op="decode", seqs=64, longest=8192, hq=32, hk=8,
             width=128, page=16, block=128, fmt="f8", dtype="bf16", weights=False),
        # the same with the rows' weights added up, as eviction asks for
        dict(name="decode_16x4000x32x128_weights", op="decode", seqs=16, longest=4000, hq=32, hk=8,
             width=128, page=16, block=128, fmt="f8", dtype="bf16", weights=True),
        # a few sequences at their budget: latency
        dict(name="evict_3x700x4x64_i8", op="evict", seqs=3, longest=700, keep=256, recent=32, hk=4,
             width=64, page=16, block=64, fmt="i8"),
        # a batch cut to a quarter
        dict(name="evict_16x8192x8x128", op="evict", seqs=16, longest=8192, keep=2048, recent=256,
             hk=8, width=128, page=16, block=128, fmt="f8"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "attend", "attend", "decode", "decode", "evict"])
    width = rng.choice([64, 80, 96, 112, 128])
    hk, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 7])
    if op == "rotate":
        n = _log(rng, 1, 16384)
        return dict(op=op, n=n, hq=hk * group, hk=hk, width=width,
                    turned=rng.choice([width, width // 16 * 8]), dtype=rng.choice(list(NUM)),
                    grad=rng.random() < 0.5, far=rng.choice([0, 1000, 1000000]))
    if op == "attend":
        longest = _log(rng, 1, 3800)
        seqs = _log(rng, 1, max(1, min(48, 8000 // longest)))
        return dict(op=op, seqs=seqs, longest=longest, hq=hk * group, hk=hk, width=width,
                    dtype=rng.choice(["bf16", "f16"]), causal=rng.random() < 0.7,
                    grad=rng.random() < 0.5, pad=rng.choice([0, 5, 100]))
    page, fmt = rng.choice([1, 16, 24, 64]), rng.choice(["f8", "i8"])
    block = rng.choice([width, 64, 128])
    if op == "decode":
        longest = _log(rng, 1, 65536)
        seqs = _log(rng, 1, max(1, min(64, 262144 // longest)))
        return dict(op=op, seqs=seqs, longest=longest, hq=hk * group, hk=hk, width=width, page=page,
                    block=block, fmt=fmt, dtype=rng.choice(list(NUM)), weights=rng.random() < 0.5)
    longest = _log(rng, 1, 8192)
    keep = _log(rng, 1, longest)
    return dict(op=op, seqs=_log(rng, 1, 16), longest=longest, keep=keep,
                recent=rng.randint(0, keep), hk=hk, width=width, page=page, block=block, fmt=fmt)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _lengths(case):
    """Lengths of the ragged sequences, the longest among them and (of more than
    two) an empty one, whose order the seed gives."""
    n, most = case["seqs"], case["longest"]
    return [most] + [0] * (n > 2) + [int(most * (i * 0.6180339887 % 1.0))
                                     for i in range(1, n - (n > 2))]


def _rows_of(case):
    return sum(_lengths(case)) + case["pad"]


def _encoded(x, block, fmt):
    """Codes and scale bytes of the rows of x (fp32), a scale per `block` values."""
    n, d = x.shape
    nb = -(-d // block)
    p = torch.nn.functional.pad(x, (0, nb * block - d)).view(n, nb, block)
    a = p.abs().amax(2)
    m, e = torch.frexp(a)
    mt, et = math.frexp(TOP[fmt])
    e = torch.where(a > 0, (e - et + (m > mt)).clamp(-127, 127), 0)
    y = (p * torch.exp2(-e.float())[:, :, None]).clamp(-TOP[fmt], TOP[fmt])
    y = torch.round(y).to(torch.int8) if fmt == "i8" else y.to(torch.float8_e4m3fn)
    return y.view(n, nb * block)[:, :d], (e + 127).to(torch.uint8)


def _store(case, pages, g, spread):
    """A store of `pages` pages of rows as attention meets them: a few large
    columns, as keys have."""
    d, rows = case["hk"] * case["width"], pages * case["page"]
    codes = torch.empty(rows, d, device="cuda", dtype=CODE[case["fmt"]])
    scales = torch.empty(rows, -(-d // case["block"]), device="cuda", dtype=torch.uint8)
    wide = torch.where(torch.rand(1, d, device="cuda", generator=g) < 0.02, spread, 1.0)
    for at in range(0, rows, 65536):
        x = _randn(g, min(rows - at, 65536), d) * wide
        codes[at:at + len(x)], scales[at:at + len(x)] = _encoded(x, case["block"], case["fmt"])
    return (codes.view(pages, case["page"], d),
            scales.view(torch.float8_e8m0fnu).view(pages, case["page"], -1))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, op, s = case, case["op"], dict(case=case)
    if op == "rotate":
        # queries, keys and values in one row, as a fused projection leaves them
        n, hq, hk, w = c["n"], c["hq"], c["hk"], c["width"]
        wide = (_randn(g, n, (hq + 2 * hk) * w)
                * torch.exp(0.5 * _randn(g, n, 1))).to(NUM[c["dtype"]])
        s["q"] = wide[:, :hq * w].unflatten(1, (hq, w))
        s["k"] = wide[:, hq * w:(hq + hk) * w].unflatten(1, (hk, w))
        s["gq"], s["gk"] = (1 + 0.2 * _randn(g, 2, w)).to(NUM[c["dtype"]]).unbind(0)
        s["positions"] = torch.arange(n, device="cuda") if not c["far"] else \
            torch.randint(0, c["far"], (n,), device="cuda", generator=g)
        i = torch.arange(c["turned"] // 2, device="cuda", dtype=torch.float64)
        s["freqs"] = 10000.0 ** (-2 * i / c["turned"])
        if c["grad"]:
            s["dq"] = (0.01 * _randn(g, n, hq, w)).to(NUM[c["dtype"]])
            s["dk"] = (0.01 * _randn(g, n, hk, w)).to(NUM[c["dtype"]])
            for name in ("q", "k", "gq", "gk"):
                s[name].requires_grad_()
        return s
    lengths = torch.tensor(_lengths(c), device="cuda")
    lengths = lengths[torch.randperm(c["seqs"], device="cuda", generator=g)]
    if op == "attend":
        n, hq, hk, w = _rows_of(c), c["hq"], c["hk"], c["width"]
        for name, h, size in (("q", hq, 1.5), ("k", hk, 1.0), ("v", hk, 1.0)):
            s[name] = (size * _randn(g, n, h, w)).to(NUM[c["dtype"]])
            s[name].requires_grad_(c["grad"])
        if c["grad"]:
            s["do"] = (0.01 * _randn(g, n, hq, w)).to(NUM[c["dtype"]])
        s["starts"] = torch.cat([lengths.new_zeros(1), torch.cumsum(lengths, 0)]).int()
        return s
    # pages in the order in which they were freed; -1 behind a sequence's last
    used = -(-lengths // c["page"])
    most = -(-c["longest"] // c["page"])
    pages = int(used.sum()) + 7
    order = torch.randperm(pages, device="cuda", generator=g).int()
    at = torch.arange(most, device="cuda")
    first = torch.cumsum(used, 0) - used
    s["table"] = torch.where(at < used[:, None],
                             order[(first[:, None] + at).clamp(max=pages - 1)], -1)
    s["lengths"] = lengths.int()
    s["keys"], s["values"] = _store(c, pages, g, 4.0), _store(c, pages, g, 1.0)
    if op == "decode":
        s["q"] = (1.5 * _randn(g, c["seqs"], c["hq"], c["width"])).to(NUM[c["dtype"]])
    if op == "evict" or c["weights"]:  # what earlier tokens gave: a few rows hold most of it
        s["weights"] = torch.exp(2 * _randn(g, c["seqs"], most * c["page"]))
        s["weights"] *= torch.arange(most * c["page"], device="cuda") < lengths[:, None]
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import mini_means_amd as em
    c, op = s["case"], s["case"]["op"]
    if op == "rotate":
        y = em.norm_rotate(s["q"], s["k"], s["gq"], s["gk"], s["positions"], s["freqs"], eps=EPS)
        if not c["grad"]:
            return y
        return *(t.detach() for t in y), *torch.autograd.grad(
            y, (s["q"], s["k"], s["gq"], s["gk"]), (s["dq"], s["dk"]))
    if op == "attend":
        o = em.attend(s["q"], s["k"], s["v"], s["starts"], causal=c["causal"])
        if not c["grad"]:
            return o
        return o.detach(), *torch.autograd.grad(o, (s["q"], s["k"], s["v"]), s["do"])
    if op == "decode":
        o = em.cache_attend(s["q"], s["keys"], s["values"], s["table"], s["lengths"],
                            block=c["block"], weights=s.get("weights"))
        return (o, s["weights"]) if c["weights"] else o
    lengths, weights, kept = em.cache_evict((s["keys"], s["values"]), s["table"], s["lengths"],
                                            s["weights"], c["keep"], recent=c["recent"],
                                            block=c["block"])
    return *s["keys"], *s["values"], lengths, weights, kept


def _run_plain(s):
    with torch.no_grad():
        return globals()["_plain_" + s["case"]["op"]](s)


def _turn(y, cos, sin, half):
    a, b = y[..., :half], y[..., half:2 * half]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., 2 * half:]], -1)


def _plain_norm(x, gain, dy, cos, sin, half):
    """One side of rotate: its result and, given dy, the gradients."""
    t, x, g = x.dtype, x.float(), gain.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    y = _turn(x * r * g, cos, sin, half).to(t)
    if dy is None:
        return y, None, None
    u = _turn(dy.float(), cos, -sin, half)
    v = u * g
    dx = r * v - x * (r ** 3 * (v * x).mean(-1, keepdim=True))
    return y, dx.to(t), (u * x * r).sum((0, 1)).to(gain.dtype)


def _plain_rotate(s):
    turns = s["positions"].double()[:, None] * s["freqs"]
    cos, sin = torch.cos(turns).float()[:, None], torch.sin(turns).float()[:, None]
    half = s["freqs"].numel()
    q, dq, dgq = _plain_norm(s["q"], s["gq"], s.get("dq"), cos, sin, half)
    k, dk, dgk = _plain_norm(s["k"], s["gk"], s.get("dk"), cos, sin, half)
    return (q, k, dq, dk, dgq, dgk) if s["case"]["grad"] else (q, k)


def _plain_attend(s):
    """All sequences side by side, filled up to the longest; the heads of a group
    are rows of one product."""
    c, t = s["case"], s["q"].dtype
    hk, G, w, L = c["hk"], c["hq"] // c["hk"], c["width"], c["longest"]
    starts = s["starts"].long()
    at = torch.arange(L, device="cuda")
    live = at < (starts[1:] - starts[:-1])[:, None]
    rows = torch.where(live, starts[:-1, None] + at, 0)

    def side(x, heads):  # sequences x key-value heads x (group x places) x width
        x = torch.where(live[:, :, None, None], x[rows].float(), 0.0)
        return x.view(-1, L, hk, heads // hk, w).permute(0, 2, 3, 1, 4).reshape(
            -1, hk, heads // hk * L, w).contiguous()

    def back(y, heads):
        y = y.view(-1, hk, heads // hk, L, w).permute(0, 3, 1, 2, 4).reshape(-1, L, heads, w)
        out = torch.zeros(s["q"].shape[0], heads, w, device="cuda", dtype=t)
        out[rows[live]] = y[live].to(t)
        return out

    q, k, v = side(s["q"], c["hq"]), side(s["k"], hk), side(s["v"], hk)
    scale = w ** -0.5
    p = (q @ k.transpose(2, 3).contiguous()).mul_(scale)
    seen = live[:, None, None, None, :]
    if c["causal"]:
        seen = seen & (at <= at[:, None])
    p.view(-1, hk, G, L, L).masked_fill_(~seen, -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    p.div_(p.sum(-1, keepdim=True).clamp(min=1e-30))
    o = p @ v
    if not c["grad"]:
        return back(o, c["hq"])
    do = side(s["do"], c["hq"])
    dv = p.transpose(2, 3) @ do
    ds = (do @ v.transpose(2, 3).contiguous()).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq = (ds @ k).mul_(scale)
    dk = (ds.transpose(2, 3) @ q).mul_(scale)
    return back(o, c["hq"]), back(dq, c["hq"]), back(dk, hk), back(dv, hk)


def _places(s):
    """Row of the store of every place of every sequence, 0 behind their ends,
    and which places are in them."""
    page = s["case"]["page"]
    at = torch.arange(s["table"].shape[1] * page, device="cuda")
    live = at < s["lengths"][:, None]
    rows = s["table"].long()[:, at // page] * page + at % page
    return torch.where(live, rows, 0), live


def _plain_values(store, rows, live, c):
    """fp32 values of those rows, zeros where not live: sequences x key-value
    heads x places x width."""
    codes, scales = (t.flatten(0, 1).view(torch.uint8) for t in store)
    x = codes[rows].view(store[0].dtype).float()
    f = torch.exp2(scales[rows].float() - 127.0).repeat_interleave(c["block"], 2)
    x = torch.where(live[:, :, None], x * f[:, :, :x.shape[2]], 0.0)
    return x.unflatten(2, (c["hk"], c["width"])).transpose(1, 2).contiguous()


def _plain_decode(s):
    c = s["case"]
    rows, live = _places(s)
    k, v = _plain_values(s["keys"], rows, live, c), _plain_values(s["values"], rows, live, c)
    q = s["q"].float().unflatten(1, (c["hk"], -1)) * c["width"] ** -0.5
    p = (q @ k.transpose(2, 3).contiguous()).masked_fill_(~live[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p = (p - torch.where(top == -math.inf, 0.0, top)).exp()
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = (p @ v).flatten(1, 2).to(s["q"].dtype)
    if not c["weights"]:
        return o
    s["weights"] += p.sum((1, 2))
    return o, s["weights"]


def _plain_evict(s):
    c = s["case"]
    rows, live = _places(s)
    n = s["lengths"].long()[:, None]
    cap = rows.shape[1]
    at = torch.arange(cap, device="cuda").expand_as(rows)
    recent = at >= n - c["recent"]
    free = torch.where(live & ~recent, s["weights"], -math.inf)
    order = torch.sort(free, dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, at)
    keep = live & ((n <= c["keep"]) | recent | (rank < c["keep"] - c["recent"]))
    kept = torch.sort(torch.where(keep, at, cap), dim=1).values[:, :c["keep"]]
    kept = torch.nn.functional.pad(kept, (0, c["keep"] - kept.shape[1]), value=cap)
    fine = kept < cap
    there = kept.clamp(max=cap - 1)
    source = rows.gather(1, there)[fine]
    to = rows[:, :c["keep"]][fine[:, :cap]]
    for t in (*s["keys"], *s["values"]):
        flat = t.flatten(0, 1).view(torch.uint8)
        flat[to] = flat[source]
    weights = torch.zeros_like(s["weights"])
    m = min(c["keep"], cap)
    weights[:, :m] = torch.where(fine, s["weights"].gather(1, there), 0.0)[:, :m]
    kept = torch.where(fine, kept, -1).int()
    return *s["keys"], *s["values"], fine.sum(1).int(), weights, kept


# --------------------------------------------------------------------------
# the bytes and operations that a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    c, op = case, case["op"]
    if op == "rotate":  # x read, y written; with gradients dy read, dx written
        values = c["n"] * (c["hq"] + c["hk"]) * c["width"]
        return dict(bytes=values * SIZE[c["dtype"]] * (4 if c["grad"] else 2) + 8 * c["n"],
                    flops=values * (20 if c["grad"] else 7))
    lengths = _lengths(c)
    if op == "attend":
        pairs = sum(n * (n + 1) // 2 if c["causal"] else n * n for n in lengths)
        rows = _rows_of(c) * c["width"] * SIZE[c["dtype"]]
        once = 2 * c["hq"] + 2 * c["hk"]
        return dict(bytes=rows * (once * 2 if c["grad"] else once),
                    flops=pairs * c["hq"] * c["width"] * (14 if c["grad"] else 4))
    d = c["hk"] * c["width"]
    row = 2 * (d + -(-d // c["block"]))
    if op == "decode":
        total = sum(lengths)
        return dict(bytes=total * (row + (8 if c["weights"] else 0))
                    + 2 * c["seqs"] * c["hq"] * c["width"] * SIZE[c["dtype"]],
                    flops=4 * total * c["hq"] * c["width"])
    moved = sum(min(n, c["keep"]) for n in lengths)
    return dict(bytes=2 * moved * row + 4 * sum(lengths) + 8 * moved, flops=sum(lengths))


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def _softmax64(scores):
    if scores.shape[-1] == 0:
        return scores
    e = torch.exp(scores - scores.max(-1, keepdim=True).values)
    return e / e.sum(-1, keepdim=True)


def _exact_side(x, gain, dy, positions, freqs):
    """As complex numbers: a pair turned is its product with e^(i angle)."""
    x, gain = x.detach().double(), gain.detach().double()
    half = freqs.numel()
    angle = torch.outer(positions.double(), freqs)
    spin = torch.polar(torch.ones_like(angle), angle)[:, None, :]

    def turned(y, by):
        z = torch.complex(y[..., :half], y[..., half:2 * half]) * by
        return torch.cat([z.real, z.imag, y[..., 2 * half:]], -1)

    size = torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    y = turned(x / size * gain, spin)
    if dy is None:
        return y, None, None
    u = turned(dy.double(), spin.conj())
    inner = (u * gain * x).sum(-1, keepdim=True) / x.shape[-1]
    return y, u * gain / size - x * inner / size ** 3, (u * x / size).sum(0).sum(0)


def _exact_rows(case, s):
    """Row numbers in the store of each sequence's places."""
    page, table = case["page"], s["table"].cpu()
    return [torch.tensor([int(table[q, p // page]) * page + p % page for p in range(n)],
                         dtype=torch.int64).cuda() for q, n in enumerate(s["lengths"].tolist())]


def _exact_store(case, store, rows):
    codes, scales = (t.flatten(0, 1) for t in store)
    x = torch.index_select(codes.view(torch.uint8), 0, rows).view(codes.dtype).double()
    byte = torch.index_select(scales.view(torch.uint8), 0, rows).double()
    col = torch.arange(x.shape[1], device="cuda") // case["block"]
    return (x * torch.pow(2.0, byte[:, col] - 127)).view(len(rows), case["hk"], case["width"])


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "rotate":
        q, dq, dgq = _exact_side(s["q"], s["gq"], s.get("dq"), s["positions"], s["freqs"])
        k, dk, dgk = _exact_side(s["k"], s["gk"], s.get("dk"), s["positions"], s["freqs"])
        return (q, k, dq, dk, dgq, dgk) if c["grad"] else (q, k)
    group = c["hq"] // c["hk"] if "hq" in c else 0
    if op == "attend":
        q, k, v = (s[name].detach().double() for name in "qkv")
        o, dq, dk, dv = (torch.zeros_like(t) for t in (q, q, k, v))
        cuts = s["starts"].tolist()
        for a, b in zip(cuts[:-1], cuts[1:]):
            hidden = torch.ones(b - a, b - a, device="cuda", dtype=torch.bool).triu(1)
            for h in range(c["hq"]):
                z = q[a:b, h] @ k[a:b, h // group].T / math.sqrt(c["width"])
                if c["causal"]:
                    z[hidden] = -math.inf
                p = _softmax64(z)
                o[a:b, h] = p @ v[a:b, h // group]
                if c["grad"]:
                    do = s["do"][a:b, h].double()
                    dv[a:b, h // group] += p.T @ do
                    dp = do @ v[a:b, h // group].T
                    dz = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(c["width"])
                    dq[a:b, h] = dz @ k[a:b, h // group]
                    dk[a:b, h // group] += dz.T @ q[a:b, h]
        return (o, dq, dk, dv) if c["grad"] else o
    if op == "decode":
        o = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
        total = s["weights"].double() if c["weights"] else None
        for i, rows in enumerate(_exact_rows(c, s)):
            k, v = _exact_store(c, s["keys"], rows), _exact_store(c, s["values"], rows)
            for h in range(c["hq"]):
                p = _softmax64(k[:, h // group] @ s["q"][i, h].double() / math.sqrt(c["width"]))
                o[i, h] = p @ v[:, h // group]
                if c["weights"]:
                    total[i, :len(p)] += p
        return (o, total) if c["weights"] else o
    stores = [t.flatten(0, 1).view(torch.uint8) for t in (*s["keys"], *s["values"])]
    weights = torch.zeros_like(s["weights"])
    kept = torch.full((c["seqs"], c["keep"]), -1, device="cuda", dtype=torch.int32)
    lengths = s["lengths"].clone()
    for i, rows in enumerate(_exact_rows(c, s)):
        w = s["weights"][i, :len(rows)].tolist()
        places = list(range(len(w)))
        if len(w) > c["keep"]:
            old = places[:len(w) - c["recent"]]
            best = sorted(old, key=lambda p: -w[p])[:c["keep"] - c["recent"]]
            places = sorted(best) + places[len(w) - c["recent"]:]
        lengths[i] = len(places)
        there = torch.tensor(places, device="cuda", dtype=torch.int64)
        kept[i, :len(places)] = there.int()
        weights[i, :len(places)] = s["weights"][i, there]
        for t in stores:
            t[rows[:len(places)]] = t[rows[there]].clone()
    out = [t.view(o.dtype).view(o.shape) for t, o in zip(stores, (*s["keys"], *s["values"]))]
    out = [o if o.dtype == torch.int8 else o.double() for o in out]
    return *out, lengths, weights.double(), kept
