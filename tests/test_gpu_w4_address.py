"""Products with 4-bit weights of x that starts on no 16-byte boundary: the kernel and
so the bits of the same x on one, at every number of rows (needs an MI355X)."""
import pytest
import torch

import permute_grouped_gemm_amd as pgg
from test_gpu_w4 import DEV, _pack, _rows, _weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gs,zeros", [(32, True), (64, False), (128, True), (256, False)])
@pytest.mark.parametrize("counts", [[3, 2], [20, 30], [80, 65], [300, 0, 65]], ids=str)
def test_an_odd_start_gives_the_same_bits(counts, gs, zeros, dtype):
    M, gl = sum(counts), torch.tensor(counts, device=DEV)
    for K in (136, 1024, 3592, 1403):
        w = _pack(*_weights(len(counts), K, 200, gs, dtype, zeros, K), gs, False)
        x = _rows(M, K, dtype, 1).to(DEV)
        want = pgg.moe_fwd_w4(x, w, None, gl)
        for shift in (1, 2, 4):
            flat = torch.empty(x.numel() + shift, dtype=x.dtype, device=DEV)
            flat[shift:] = x.reshape(-1)
            assert torch.equal(pgg.moe_fwd_w4(flat[shift:].reshape(M, K), w, None, gl), want), (K, shift)


@pytest.mark.parametrize("row_idx_type", [0, 1])
def test_an_odd_start_with_an_index(row_idx_type):
    T, topk, K, gs = 150, 2, 520, 128
    w = _pack(*_weights(3, K, 140, gs, "bf16", True, 2), gs, True)
    eri = torch.randperm(T * topk, generator=torch.Generator().manual_seed(1)).to(DEV)
    gl = torch.tensor([170, 0, 130], device=DEV)
    x = _rows(T, K, "bf16", 1).to(DEV)
    x[7, 3] = float("inf")
    want = pgg.moe_glu_w4(x, w, eri, gl, topk, row_idx_type)
    flat = torch.empty(x.numel() + 3, dtype=x.dtype, device=DEV)
    flat[3:] = x.reshape(-1)
    got = pgg.moe_glu_w4(flat[3:].reshape(T, K), w, eri, gl, topk, row_idx_type)
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))
