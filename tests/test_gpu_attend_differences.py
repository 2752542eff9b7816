"""Attention's gradients against differences of the definition in 64 bits."""
import pytest

import attention_ref as ref
from test_gpu_attend import inputs
from test_gpu_attention_store import f64, mm  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,sharp", [("bf16", 0.2), ("f16", 0.03)])
@pytest.mark.parametrize("causal,lq,lk,hq,hk,w", [(True, 90, 90, 2, 1, 64), (False, 70, 130, 4, 2, 128),
                                                  (True, 40, 150, 3, 3, 96), (True, 130, 33, 2, 1, 40)])
def test_gradients_against_differences_of_the_definition(mm, dtype, sharp, causal, lq, lk, hq, hk, w):  # noqa: F811
    import torch
    q, k, v, do, starts, k_starts = inputs([lq], [lk], hq, hk, w, dtype, lq + w, 0, 0)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    o = mm.attend(*leaves, starts, k_starts=None if lq == lk else k_starts, causal=causal)
    grads = [f64(g) for g in torch.autograd.grad(o, leaves, do)]
    for said, slope, off in ref.grad_slopes(*(f64(t) for t in (q, k, v, do)), grads, w ** -0.5, causal, dtype):
        assert off <= sharp * abs(slope)
        assert abs(said - slope) <= off, (said, slope, off)
