"""Products with 4-bit weights of rows that few experts have, at the averages where the
tile changes (needs an MI355X)."""
import pytest
import torch

from test_gpu_w4 import _check_fwd, _check_glu

pytestmark = pytest.mark.gpu
G = 16


def _counts(M, kind):
    """M rows on all experts, on two, on the last, or by popularity."""
    if kind == "alike":
        return [M // G + (g < M % G) for g in range(G)]
    if kind == "two":
        return [0] * 5 + [M // 2] + [0] * 6 + [M - M // 2] + [0] * 3
    if kind == "last":
        return [0] * (G - 1) + [M]
    p = [1.0 / (g + 1) ** 1.1 for g in range(G)]
    counts = [int(M * v / sum(p)) for v in p]
    counts[0] += M - sum(counts)
    return counts[::-1]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["alike", "two", "last", "popular"])
@pytest.mark.parametrize("M", [383, 384, 512, 513])
def test_fwd(M, kind, dtype):
    # 24 and 32 rows for each of 16 experts; 43 column blocks and one that is not full
    _check_fwd(_counts(M, kind), 136, 64 * 43 + 9, 64, dtype, True, seed=M)


@pytest.mark.parametrize("kind", ["alike", "two", "popular"])
@pytest.mark.parametrize("row_idx_type", [0, 1])
@pytest.mark.parametrize("M", [382, 384, 512])
def test_glu_with_an_index(M, row_idx_type, kind):
    _check_glu(_counts(M, kind), 100, 32 * 65 - 3, 32, "bf16", False, row_idx_type, 2, "silu", seed=M)


def test_workspace_of_either_tile():
    # what the query asks for is enough on both sides of the change
    for M in (383, 384):
        for odd in (0, 1):
            _check_fwd(_counts(M, "alike"), 131 + odd, 64 * 50, 128, "f16", False, seed=odd)
