"""One attention layer served and trained around the coded store.

    python examples/token_attention.py

1. Prompts of different lengths are packed: projected with encoded weights
   (block_linear), queries and keys normed and turned (norm_rotate), attended
   (attend), and their keys and values written into paged stores (cache_write).
2. New tokens follow one per sequence: the same projection, the store written, and
   attention over the store (cache_attend), which adds up each row's weight.
3. Sequences over their budget drop the rows of least weight (cache_evict).
4. A training step: gradients through attend, norm_rotate and block_linear.

All data is synthetic (seeded).
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mini_means_amd as em  # noqa: E402


class Layer:
    """Weights of an attention layer, and its projections."""

    def __init__(self, d=512, hq=8, hk=2, width=64, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.d, self.hq, self.hk, self.width = d, hq, hk, width
        rows = (hq + 2 * hk) * width
        self.w_in = torch.randn(rows, d, device="cuda", generator=g).bfloat16() * d ** -0.5
        self.w_out = torch.randn(d, hq * width, device="cuda", generator=g).bfloat16() * d ** -0.5
        self.gain_q, self.gain_k = torch.ones(2, width, device="cuda").unbind(0)
        self.freqs = em.rotary_freqs(width)

    def parts(self, x, positions, w_in):
        """Queries, keys and values of the rows of x at their positions."""
        y = em.block_linear(x, w_in)
        q, k, v = y.unflatten(1, (-1, self.width)).split([self.hq, self.hk, self.hk], 1)
        return (*em.norm_rotate(q, k, self.gain_q, self.gain_k, positions, self.freqs), v)


class Cache:
    """Paged stores of keys and values, and who has which page."""

    def __init__(self, layer, seqs, pages_each, page=16):
        self.page = page
        self.keys, self.values = (em.cache_new((seqs * pages_each, page), layer.hk * layer.width,
                                               block=layer.width) for _ in range(2))
        order = torch.randperm(seqs * pages_each, generator=torch.Generator().manual_seed(2))
        self.table = order.int().view(seqs, pages_each).cuda()
        self.lengths = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.positions = torch.zeros(seqs, dtype=torch.int64, device="cuda")
        self.weights = torch.zeros(seqs, pages_each * page, device="cuda")
        self.block = layer.width

    def slots(self, seq, place):
        return self.table[seq, place // self.page].long() * self.page + place % self.page

    def write(self, k, v, seq, place):
        at = self.slots(seq, place)
        em.cache_write(k, at, *self.keys, block=self.block)
        em.cache_write(v, at, *self.values, block=self.block)


def prompt(layer, weights, cache, x, lengths):
    """The layer over packed prompts; their keys and values go to the stores."""
    n = torch.tensor(lengths, device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(lengths), device="cuda"), n)
    starts = torch.cat([n.new_zeros(1), n.cumsum(0)])
    place = torch.arange(len(x), device="cuda") - starts[seq]
    q, k, v = layer.parts(x, place, weights[0])
    cache.write(k, v, seq, place)
    cache.lengths += n.int()
    cache.positions += n
    o = em.attend(q, k, v, starts.int())
    return em.block_linear(o.flatten(1), weights[1]), (q, k, v, o)


def step(layer, weights, cache, x):
    """One new token per sequence."""
    q, k, v = layer.parts(x, cache.positions, weights[0])
    cache.write(k, v, torch.arange(len(x), device="cuda"), cache.lengths.long())
    cache.lengths += 1
    cache.positions += 1
    o = em.cache_attend(q, cache.keys, cache.values, cache.table, cache.lengths, block=cache.block,
                        weights=cache.weights)
    return em.block_linear(o.flatten(1), weights[1]), (q, o)


def trim(cache, keep, recent):
    """Sequences over `keep` rows drop the rows of least weight; the places that stay."""
    cache.lengths, cache.weights, kept = em.cache_evict(
        (cache.keys, cache.values), cache.table, cache.lengths, cache.weights, keep, recent=recent,
        block=cache.block)
    return kept


def train_step(layer, x, lengths, target):
    """Loss and gradients of the layer's weights."""
    n = torch.tensor(lengths, device="cuda")
    starts = torch.cat([n.new_zeros(1), n.cumsum(0)])
    place = torch.arange(len(x), device="cuda") - torch.repeat_interleave(starts[:-1], n)
    leaves = [t.detach().requires_grad_() for t in (layer.w_in, layer.w_out, layer.gain_q, layer.gain_k)]
    y = em.block_linear(x, leaves[0])
    q, k, v = y.unflatten(1, (-1, layer.width)).split([layer.hq, layer.hk, layer.hk], 1)
    q, k = em.norm_rotate(q, k, leaves[2], leaves[3], place, layer.freqs)
    o = em.attend(q, k, v, starts.int())
    loss = (em.block_linear(o.flatten(1), leaves[1]) - target).float().square().mean()
    return loss, torch.autograd.grad(loss, leaves)


def main(lengths=(70, 1, 33), steps=40, keep=64, recent=16):
    layer = Layer()
    weights = [em.block_encode(w, tiles=True) for w in (layer.w_in, layer.w_out)]
    cache = Cache(layer, len(lengths), 16)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(sum(lengths), layer.d, device="cuda", generator=g).bfloat16()
    y, _ = prompt(layer, weights, cache, x, lengths)
    kept = None
    for _ in range(steps):
        y, _ = step(layer, weights, cache, torch.randn(len(lengths), layer.d, device="cuda", generator=g).bfloat16())
        if int(cache.lengths.max()) >= keep + recent:
            kept = trim(cache, keep, recent)
    loss, grads = train_step(layer, x, lengths, torch.zeros_like(x))
    print(f"{len(lengths)} sequences at positions {cache.positions.tolist()}, {cache.lengths.tolist()} rows kept; "
          f"output {tuple(y.shape)}; loss {loss.item():.4f}, gradients {[round(t.float().norm().item(), 4) for t in grads]}")
    return dict(cache=cache, kept=kept, loss=loss, grads=grads, y=y)


if __name__ == "__main__":
    main()
