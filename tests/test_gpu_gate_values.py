"""Non-finite and extreme logits of the router's gate and its gradient."""
import math

import pytest
import torch

import ops_ref as ref
import permute_grouped_gemm_amd as pgg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _logits(T, E, seed, dtype="f32"):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=gen) * 1.5).to(ref.DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("E", [12, 100, 200, 400, 900, 1200])
def test_an_infinite_logit_makes_its_weights_nan(E, dtype):
    # exp(l - lse) with an infinite lse is no number, for the finite picks too: none
    # of them may look like a weight of 0
    l = _logits(4, E, E, dtype)
    l[1, 3] = math.inf
    l[2, 5] = math.nan
    l[3, 4] = l[3, 9] = math.inf
    for renorm in (False, True):
        ids, probs, lse = pgg.moe_gate(l.to(DEV), 4, renorm=renorm)
        assert probs[0].isfinite().all() and lse[0].isfinite()
        assert probs[1:].isnan().all() and lse[1:].isnan().all()
        grad = pgg.moe_gate_grad(l.to(DEV), lse, ids, torch.ones((4, 4), device=DEV), renorm=renorm)
        assert grad[0].isfinite().all()
        assert grad.gather(1, ids)[1:].isnan().all()
