"""The gated product's gradient and its group tables at the group counts where
the threads that make them change (needs an MI355X)."""
import math

import pytest
import torch

import ops_ref as ref
import permute_grouped_gemm_amd as pgg

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("M", [3, 700, 4096, 4097])
@pytest.mark.parametrize("G", [257, 300, 1024, 1025, 2500])
def test_many_groups(G, M):
    gen = torch.Generator().manual_seed(G + M)
    D, F = 24, 8
    gl = torch.bincount(torch.randint(0, G, (M,), generator=gen), minlength=G)
    gy, gu = torch.randn((M, D), generator=gen).half(), torch.randn((M, 2 * F), generator=gen).half()
    w = (torch.randn((G, F, D), generator=gen) / math.sqrt(D)).half()
    args = [t.to(DEV) for t in (gy, w, gu, gl)]
    ws = torch.empty(pgg.glu_grad_workspace_size(*args), dtype=torch.uint8, device=DEV)
    grad, h = pgg.moe_glu_grad(*args, workspace=ws)
    wg, eg, wh, eh = ref.glu_grad(gy, w, gu, gl, "silu")
    ref.assert_within(grad, wg, eg, "grad")
    ref.assert_within(h, wh, eh, "h")
    assert pgg.read_device_error(ws) == (pgg.DEV_OK, 0)
    bad = gl.clone()
    bad[G - 1] -= M + 1
    pgg.moe_glu_grad(*args[:3], bad.to(DEV), workspace=ws)
    assert pgg.read_device_error(ws) == (pgg.DEV_GROUP_NEGATIVE, G - 1)


@pytest.mark.parametrize("G", [1, 63, 64, 65, 200])
def test_many_rows_in_a_few_groups(G):
    # tiles of 128 or 256 rows, whose table one wave makes up to 64 groups
    gen = torch.Generator().manual_seed(G)
    D, F, M = 24, 8, min(4000, 66 * G)
    gl = torch.bincount(torch.randint(0, G, (M,), generator=gen), minlength=G)
    for dtype in ("f32", "bf16"):
        dt = ref.DTYPES[dtype]
        gy, gu = torch.randn((M, D), generator=gen).to(dt), torch.randn((M, 2 * F), generator=gen).to(dt)
        w = (torch.randn((G, F, D), generator=gen) / math.sqrt(D)).to(dt)
        grad, h = pgg.moe_glu_grad(*[t.to(DEV) for t in (gy, w, gu, gl)])
        wg, eg, wh, eh = ref.glu_grad(gy, w, gu, gl, "silu")
        ref.assert_within(grad, wg, eg, "grad")
        ref.assert_within(h, wh, eh, "h")
