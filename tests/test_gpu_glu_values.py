"""The gated product's gradient at the ends of the gates' range."""
import pytest
import torch

import permute_grouped_gemm_amd as pgg

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [4, 700])
@pytest.mark.parametrize("D", [8, 600])
def test_slopes_of_gates_whose_square_overflows(dtype, rows, D):
    # far out the activation is its gate or 0 and its slope 1 or 0; dh is 2 and up 4,
    # so every result is exact (D 600: the reduction of few rows is split)
    gates = [2.0 ** 62, -2.0 ** 62, 2.0 ** 66, -2.0 ** 66, 2.0 ** 100, -2.0 ** 100, 2.0 ** 125, -2.0 ** 125]
    F = len(gates)
    g = torch.tensor(gates).expand(rows, F)
    gate_up = torch.cat([g, torch.full((rows, F), 4.0)], dim=1).to(dtype)
    gy, w = torch.zeros((rows, D)).to(dtype), torch.zeros((1, F, D)).to(dtype)
    gy[:, 1], w[:, :, 1] = 1.0, 2.0
    for act in ("silu", "gelu_tanh"):
        grad, h = pgg.moe_glu_grad(gy.to(DEV), w.to(DEV), gate_up.to(DEV), torch.tensor([rows], device=DEV), act=act)
        value = torch.where(g > 0, g, torch.zeros_like(g))
        assert torch.equal(grad[:, :F].float().cpu(), torch.where(g > 0, 8.0, 0.0).expand(rows, F))
        assert torch.equal(grad[:, F:].float().cpu(), 2 * value)
        assert torch.equal(h.float().cpu(), 4 * value)
