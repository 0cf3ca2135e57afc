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


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("E,k", [(8, 2), (60, 8), (130, 8), (300, 4), (1100, 8)])
def test_gradients_of_rows_far_from_zero(E, k, dtype):
    # rows of the type's lowest or largest value, and rows with a large offset: the
    # softmax depends on differences of logits only, and so does its gradient's
    # error: exp of a rounded difference, E additions, a few products
    dt = ref.DTYPES[dtype]
    big = torch.finfo(dt).max
    l = _logits(8, E, 3 * E, dtype)
    l[0], l[1] = -big, big
    l[2] = -big
    l[2, E // 2] = -big * 0.75                         # one far above the others
    l[3] = 4096.0 + 4 * (torch.arange(E) % 3)
    l[4] = -8192.0 - 8 * (torch.arange(E) % 5)
    l[5, 3:] = -big                                    # three experts left
    gen = torch.Generator().manual_seed(E)
    gp, gl = torch.randn((8, k), generator=gen), torch.randn(8, generator=gen)
    ids, _, lse = pgg.moe_gate(l.to(DEV), k)
    ld = l.double()
    p = torch.softmax(ld, dim=1)
    d = torch.zeros((8, E), dtype=torch.float64).scatter(1, ids.cpu(), gp.double() * 2.5)
    far = (ld - ld.amax(dim=1, keepdim=True)).abs().clamp_max(128.0)   # beyond, exp is 0 either way
    for renorm in (False, True):
        chosen = torch.zeros((8, E), dtype=torch.bool).scatter(1, ids.cpu(), True)
        w = torch.softmax(ld.masked_fill(~chosen, -math.inf), dim=1) if renorm else p
        mean = (w * d).sum(dim=1, keepdim=True)
        size = w * (d.abs() + (w * d.abs()).sum(dim=1, keepdim=True)) + p * gl.double().abs()[:, None]
        want = w * (d - mean) + p * gl.double()[:, None]
        got = pgg.moe_gate_grad(l.to(DEV), lse, ids, gp.to(DEV), grad_lse=gl.to(DEV), renorm=renorm, scale=2.5)
        bound = size * (far.amax(dim=1, keepdim=True) + E + 32) * 2.0 ** -22
        ref.assert_within(got, want, ref.rounded(want, bound, dt), f"renorm {renorm}")


def test_a_nan_of_any_payload_is_a_gradient_like_others():
    # a product keeps a NaN's payload, so any bits can reach the kernel
    l = _logits(3, 20, 4)
    ids, _, lse = pgg.moe_gate(l.to(DEV), 3)
    for bits in (0x7FC00000, 0x7FC0DEAD, 0x7F80DEAD, 0x7FFFFFFF):
        gp = torch.ones((3, 3))
        gp.view(torch.int32)[1, 1] = bits
        for renorm in (False, True):
            grad = pgg.moe_gate_grad(l.to(DEV), lse, ids, gp.to(DEV), renorm=renorm)
            assert grad[[0, 2]].isfinite().all()
            assert grad[1].gather(0, ids[1]).isnan().all()
            if not renorm:
                assert grad[1].isnan().all()
