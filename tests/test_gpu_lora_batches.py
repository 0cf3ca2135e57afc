"""The adapters in batches of a few hundred to a few thousand tokens: tiles of
128 and 256 rows whose reduction is split, and the sums of the splits."""
import pytest
import torch

import ops_ref as ref
import permute_grouped_gemm_amd as pgg
from test_gpu_lora import _make, _run

pytestmark = pytest.mark.gpu
DEV = "cuda"

# tokens, K, N, adapters, rank.  Reductions of 512 and more split from 257 tokens
# on; columns at any address take the 128-row tiles, or from 2048 tokens a padded
# copy; from 262144 results on four columns of the sums go to a thread
SHAPES = [(257, 512, 264, 3, 8), (300, 1024, 264, 7, 16), (520, 2048, 512, 20, 12), (600, 1000, 99, 4, 16),
          (1030, 520, 256, 60, 16), (1030, 1031, 255, 9, 33), (2100, 600, 131, 5, 16), (2100, 515, 128, 60, 20),
          (128, 256, 2048, 9, 16), (700, 768, 520, 1, 64), (4100, 512, 64, 30, 8)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,K,N,P,R", SHAPES)
def test_split_batches(T, K, N, P, R, dtype):
    for order in ("runs", "mixed"):
        args = _make(T, K, N, P, R, dtype, T + K, order)
        # the partial products are there: the plan splits
        assert pgg.lora_workspace_size(*[t.to(DEV) for t in args]) >= 2 * 4 * T * N
        want, bound = ref.lora(*args)
        ref.assert_within(_run(*args), want, bound, order)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_split_batches_are_repeatable_and_keep_values_apart(dtype):
    x, w, a, b, ids, s = _make(1030, 520, 256, 6, 8, dtype, 3, "mixed")
    clean = _run(x, w, a, b, ids, s)
    assert torch.equal(clean, _run(x, w, a, b, ids, s))
    a2, b2, x2 = a.clone(), b.clone(), x.clone()
    a2[0, 3, 5] = b2[1, 2, 7] = float("nan")
    x2[512, 3] = float("inf")
    got = _run(x2, w, a2, b2, ids, s)
    touched = (ids == 0) | (ids == 1)
    touched[512] = True
    assert torch.equal(clean[~touched.to(DEV)], got[~touched.to(DEV)])
    alone = _run(x, w, torch.zeros_like(a), b, ids, s)
    assert torch.equal(alone, _run(x, w, a, b, torch.full_like(ids, -1), s))
