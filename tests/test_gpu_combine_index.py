"""The combination's index of positions where it changes between searched and inverted:
the results of the same index by rows, and its errors (needs an MI355X)."""
import pytest
import torch

import permute_grouped_gemm_amd as pgg
from test_gpu_combine import DEV, _dev, _inputs, _run

pytestmark = pytest.mark.gpu


# around 8 entries to a thread (256 and 128 threads), 2^21 entries forward and 2^20 in
# the gradient, and 64 slots
SIZES = [(1448, 1, 2048), (1449, 1, 2048), (1023, 1, 2048), (1024, 1, 2048), (1025, 1, 2048), (1024, 1, 4096),
         (1025, 1, 4096), (1024, 2, 2048), (1025, 2, 2048), (512, 2, 4096), (725, 2, 4096), (32, 64, 2048),
         (31, 65, 2048), (2047, 1, 2047), (512, 1, 64), (513, 1, 64)]


@pytest.mark.parametrize("batch,topk,H", SIZES)
def test_positions_give_the_bits_of_rows(batch, topk, H):
    s = _inputs(batch, topk, H, "bf16", True, False, True, seed=batch)
    rows = {**s, "eri": torch.empty_like(s["eri"])}
    rows["eri"][s["eri"]] = torch.arange(batch * topk)
    for grad in (False, True):
        size = pgg.combine_grad_workspace_size if grad else pgg.combine_workspace_size
        ws = torch.full((size(_dev(s["permuted"]), _dev(s["probs"])),), 0xAB, dtype=torch.uint8, device=DEV)
        got = _run(s, 0, 0.7, 1e-5, grad, ws)
        assert pgg.read_device_error(ws) == (pgg.DEV_OK, 0)
        for a, b in zip(got, _run(rows, 1, 0.7, 1e-5, grad)):
            assert a is None and b is None or torch.equal(a, b)


@pytest.mark.parametrize("batch,topk,H", [(1024, 1, 4096), (1025, 1, 4096), (1448, 1, 2048), (1449, 1, 2048)])
def test_bad_positions_are_reported(batch, topk, H):
    s = _inputs(batch, topk, H, "bf16", True, False, True)
    M = batch * topk
    for bad, code in ((torch.where(s["eri"] == 3, M, s["eri"]), pgg.DEV_INDEX_RANGE),
                      (torch.where(s["eri"] == 3, -1, s["eri"]), pgg.DEV_INDEX_RANGE),
                      (torch.where(s["eri"] == 3, 4, s["eri"]), pgg.DEV_INDEX_DUP)):
        for grad in (False, True):
            size = pgg.combine_grad_workspace_size if grad else pgg.combine_workspace_size
            ws = torch.empty(size(_dev(s["permuted"]), _dev(s["probs"])), dtype=torch.uint8, device=DEV)
            _run({**s, "eri": bad}, 0, 1.0, 1e-6, grad, ws)
            assert pgg.read_device_error(ws)[0] == code, grad
