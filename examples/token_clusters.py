"""Clusters of a model's token embeddings, kept in 8-bit codes throughout.

    python examples/token_clusters.py

1. A projection from hidden states to embeddings is trained in FP8
   (block_linear with gradients).
2. Tokens arrive a few at a time: each step projects them with the encoded
   weights (block_linear with codes) and writes the embeddings into a paged store
   (cache_write).
3. The streaming loop clusters the stored embeddings, reading each batch back by
   slot (cache_read).
4. A new batch of sequences is read through its page table (cache_read_pages)
   and scored against all centroids with one 8-bit product (block_matmul); the
   labels are compared with the exact search (assign).

All data is synthetic (seeded).
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mini_means_amd as em  # noqa: E402


def hidden_states(n, d, g, kinds=64):
    """Hidden states around `kinds` directions, with a few large columns."""
    centers = torch.randn(kinds, d, generator=torch.Generator().manual_seed(3)).cuda()
    which = torch.randint(0, kinds, (n,), generator=g).cuda()
    x = centers[which] + 0.5 * torch.randn(n, d, generator=g).cuda()
    x[:, ::97] *= 8
    return x.to(torch.bfloat16)


def train_projection(d_in, d_out, steps, rows, g):
    """Fit w to a given linear map from its outputs; the losses."""
    target = torch.randn(d_out, d_in, generator=g).cuda() * d_in ** -0.5
    w = torch.zeros(d_out, d_in, device="cuda", requires_grad=True)
    rate, losses = 0.3, []
    for _ in range(steps):
        x = hidden_states(rows, d_in, g).float()
        x = x / x.norm(dim=1, keepdim=True) * d_in ** 0.5
        loss = (em.block_linear(x, w) - x @ target.t()).square().sum(1).mean() / 2
        grad, = torch.autograd.grad(loss, w)
        with torch.no_grad():
            w -= rate / d_in * 8 * grad
        losses.append(loss.item())
    return w.detach(), losses


def fill_store(w, tokens, per_step, page, g):
    """Serve `tokens` tokens, per_step at a time; the store and each slot's row."""
    d_out, d_in = w.shape
    weights = em.block_encode(w, tiles=True)
    pages = -(-tokens // page)
    codes, scales = em.cache_new((pages, page), d_out)
    order = torch.randperm(pages * page, generator=g)[:tokens].cuda()  # slots as they were freed
    for at in range(0, tokens, per_step):
        x = hidden_states(min(per_step, tokens - at), d_in, g)
        em.cache_write(em.block_linear(x, weights), order[at:at + len(x)], codes, scales)
    return codes, scales, order.int()


def cluster_store(codes, scales, slots, k, passes, seed=1234):
    """Cluster the rows that `slots` names with the streaming loop."""
    n, d = slots.numel(), codes.shape[-1]

    def rows(ids):
        return em.cache_read(codes, scales, slots[ids.long()], out_dtype=torch.bfloat16)

    start = rows(em.batch_rows(n, seed, -1, 0, k)).float()
    s = em.begin(n, start, passes, seed, dtype=torch.bfloat16)
    size = s.recipe["batch_size"]
    for e, count in enumerate(s.recipe["epoch_rows"]):
        ids = em.batch_rows(n, seed, e, 0, count)
        for at in range(0, count, size):
            s.accumulate(rows(ids[at:at + size]), labels=False)
            s.update()
        s.end_epoch()
    return s.finalize(), s


def label_sequences(codes, scales, table, starts, total, centroids):
    """Labels of ragged sequences by 8-bit scores, and by the exact search."""
    x = em.cache_read_pages(codes, scales, table, starts, total, out_dtype=torch.float32)
    scores = em.block_matmul(*em.block_encode(x), *em.block_encode(centroids),
                             out_dtype=torch.float32)
    labels = (scores - 0.5 * centroids.square().sum(1)).argmax(1)
    return labels, em.assign(x, centroids, with_dists=False)[0]


def main(d_in=1024, d_out=256, tokens=20_000, per_step=16, page=16, k=64, steps=40):
    g = torch.Generator().manual_seed(7)
    w, losses = train_projection(d_in, d_out, steps, 2048, g)
    codes, scales, slots = fill_store(w, tokens, per_step, page, g)
    centroids, stream = cluster_store(codes, scales, slots, k, 3.0)
    lengths = [0, 1, 5 * page + 3, 200, page]
    most = -(-max(lengths) // page)
    table = torch.randperm(codes.shape[0], generator=g)[:len(lengths) * most].int()
    starts = torch.tensor([0] + lengths).cumsum(0).int()
    labels, exact = label_sequences(codes, scales, table.view(len(lengths), most).cuda(),
                                    starts.cuda(), int(starts[-1]), centroids)
    agree = (labels == exact).float().mean().item()
    store = codes.numel() + scales.numel()
    print(f"projection loss {losses[0]:.2f} -> {losses[-1]:.3f}; {tokens} embeddings in "
          f"{store / 2 ** 20:.1f} MiB; mean squared distance {stream.stats['obj'][-1]:.3f}; "
          f"{agree:.1%} of the 8-bit labels are the exact search's")
    return dict(losses=losses, agree=agree, obj=stream.stats["obj"])


if __name__ == "__main__":
    main()
