"""Attention around the store: calls that the documentation allows, and what is refused."""
import numpy as np
import pytest

import attention_ref as ref
from test_gpu_attend import inputs
from test_gpu_attention_store import T, f64, gen, mm, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,heads", [(1, 2), (1, 1), (0, 2), (3, 1), (2, 2)])
def test_rows_and_heads_at_any_distance_where_there_is_one(mm, rows, heads, dtype):  # noqa: F811
    """torch calls a tensor contiguous whatever the distance of what there is one of: rows of a prompt of
    one token out of an odd buffer, a single head, a gradient like these."""
    import torch
    base = randn(gen(rows + heads), 8, 131 * 3).to(T(dtype))

    def view(i):
        return base[2:2 + rows, 131 * i:131 * i + 64 * heads].unflatten(1, (heads, 64))

    def apart(x):                  # the same values, heads 67 apart
        room = torch.zeros(x.shape[0], heads, 67, device="cuda", dtype=x.dtype)
        room[:, :, :64] = x
        return room[:, :, :64]

    def far(x):                    # rows 2^24 values apart, as a slice across a large buffer is
        return x.as_strided(x.shape, (1 << 24, 64, 1)) if x.shape[0] == 1 and x.is_contiguous() else x

    starts = torch.tensor([0, rows], device="cuda").int()
    plain = [view(i).clone(memory_format=torch.contiguous_format) for i in range(3)]
    do = randn(gen(9), rows, heads, 64).to(T(dtype))
    results = []
    for make, of in ((lambda x: x, plain), (lambda x: x, [view(i) for i in range(3)]), (apart, plain), (far, plain)):
        leaves = [make(x.detach()).requires_grad_() for x in of]
        o = mm.attend(*leaves, starts)
        results.append((o, *torch.autograd.grad(o, leaves, make(do))))
        with torch.no_grad():
            assert torch.equal(mm.attend(*leaves, starts), o)
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], r))


def test_the_same_starts_for_keys_of_a_longer_buffer(mm):  # noqa: F811
    """k_starts given, and the same tensor as starts: keys behind the last sequence are not read."""
    import torch
    q, k, v, _, starts, _ = inputs([30, 9], [30, 9], 2, 1, 64, "bf16", 4, 0, 0)
    pad = torch.full((7, 1, 64), float("nan"), device="cuda", dtype=k.dtype)
    got = mm.attend(q, torch.cat([k, pad]), torch.cat([v, pad]), starts, k_starts=starts)
    assert torch.equal(got, mm.attend(q, k, v, starts))
    with pytest.raises(mm.EmeansError, match="EINVAL"):
        mm.attend(q, torch.cat([k, pad]), torch.cat([v, pad]), starts)
