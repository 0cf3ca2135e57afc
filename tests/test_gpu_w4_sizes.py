"""Products with 4-bit weights at sizes that divide the work differently: waves
side by side or along the reduction, the reduction over workgroups, tiles of 16,
32 and 64 rows, tables for few and many experts (needs an MI355X)."""
import pytest
import torch

import block_ref as ref
import ops_ref
import permute_grouped_gemm_amd as pgg
from test_gpu_w4 import DEV, _check_fwd, _check_glu, _pack, _rows, _weights

pytestmark = pytest.mark.gpu


# 64 experts; the column blocks (9, 19, 35, 53) end inside what stands side by side
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("blocks", [9, 19, 35, 53])
@pytest.mark.parametrize("rows", [2, 20])
def test_blocks_side_by_side(rows, blocks, dtype):
    counts = [rows, rows - 1, 0, rows + 3] * 16
    _check_fwd(counts, 72, 64 * blocks - 7, 32, dtype, True)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gs", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_reduction_over_workgroups(gs, zeros, dtype):
    _check_fwd([3, 0, 2], 3600, 130, gs, dtype, zeros)       # few rows
    _check_fwd([100, 7], 3592, 130, gs, dtype, zeros)        # 64-row tiles
    _check_glu([4, 4], 3640, 70, gs, dtype, zeros, 0, 2, "silu")
    _check_glu([150, 50], 2057, 150, gs, dtype, zeros, 1, 2, "gelu_tanh")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("counts", [[63, 64, 65], [1, 127, 128, 129], [0, 0, 200, 0], [192], [33] * 4 + [32]],
                         ids=lambda c: str(c)[:16])
def test_rows_around_the_tiles_edges(counts, dtype):
    _check_fwd(counts, 264, 300, 128, dtype, True)
    topk = 1 if sum(counts) % 2 else 2
    _check_glu(counts, 260, 150, 64, dtype, False, 0, topk, "silu")


@pytest.mark.parametrize("experts", [255, 300, 1500])
@pytest.mark.parametrize("indexed", [None, 0, 1])
def test_many_experts(experts, indexed):
    counts = [(i * 7) % 3 for i in range(experts)]
    counts[-1] += sum(counts) % 2      # rows of pairs
    _check_fwd(counts, 40, 33, 32, "bf16", True, indexed=indexed, topk=1 if indexed is None else 2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("row_idx_type", [0, 1])
@pytest.mark.parametrize("tokens", [12, 16, 17, 32, 33, 900])
def test_indexes_of_few_and_many_rows(tokens, row_idx_type, dtype):
    M = 4 * tokens
    counts = [M // 2, 0, M // 3, M - M // 2 - M // 3]
    _check_glu(counts, 136, 40, 64, dtype, True, row_idx_type, 4, "silu")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_sums_of_group_products_that_cancel(dtype):
    # rows of equal elements and codes of the zero point: every product is 0, as both
    # sums hold the same integers times one value
    G, K, N, gs = 2, 512, 70, 128
    codes = torch.full((G, K, N), 9, dtype=torch.uint8)
    scales, zeros = torch.ones((G, K // gs, N)), torch.full((G, K // gs, N), 9, dtype=torch.uint8)
    w = _pack(codes, scales.to(ops_ref.DTYPES[dtype]), zeros, gs, False)
    for rows in (3, 30, 200):
        x = torch.full((rows, K), 0.75, dtype=ops_ref.DTYPES[dtype], device=DEV)
        y = pgg.moe_fwd_w4(x, w, None, torch.tensor([rows, 0], device=DEV))
        assert torch.equal(y, torch.zeros_like(y))


def test_a_token_goes_to_one_expert_several_times():
    # every slot of every token at the same expert: the rows of x repeat inside a tile
    G, K, F, gs, T, topk = 3, 256, 50, 64, 70, 4
    w = _weights(G, K, 2 * F, gs, "bf16", True, 5)
    x = _rows(T, K, "bf16", 6)
    eri, gl = torch.arange(T * topk), torch.tensor([0, T * topk, 0])
    for kind in (0, 1):
        h = pgg.moe_glu_w4(x.to(DEV), _pack(*w, gs, True), eri.to(DEV), gl.to(DEV), topk, kind)
        want, bound = ref.w4_glu(x, *w, gs, gl, topk=topk, eri=eri, row_idx_type=kind)
        ops_ref.assert_within(h, want, bound, f"index {kind}")


# every end of a row inside and beside 8 elements, alone and behind whole tiles
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("counts", [[3, 2], [20, 30], [90, 75]], ids=str)
def test_every_end_of_a_row(counts, dtype):
    for K in list(range(1, 20)) + list(range(121, 138)) + [1027, 1030]:
        _check_fwd(counts, K, 33, 32 if K % 2 else 64, dtype, True, seed=K)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", [131, 260])
def test_nan_in_the_rows_beside(K, dtype):
    w = _pack(*_weights(1, K, 70, 64, dtype, True, 1), 64, False)
    for rows in (9, 40, 100):
        x, gl = _rows(rows, K, dtype, 2).to(DEV), torch.tensor([rows], device=DEV)
        want = pgg.moe_fwd_w4(x, w, None, gl)
        x[1::2] = float("nan")
        y = pgg.moe_fwd_w4(x, w, None, gl)
        assert bool(y[1::2].isnan().all())
        # (computed again with code - zero: other roundings of the same sum)
        assert torch.allclose(y[::2].float(), want[::2].float(), rtol=2.0 ** -7, atol=2.0 ** -9)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("K", [256, 200, 131])
@pytest.mark.parametrize("shift", [1, 4, 8])
def test_many_rows_at_any_address(shift, K, dtype):
    # x, and the result, that start 2, 8 and 16 bytes behind a boundary
    w = _weights(2, K, 96, 64, dtype, True, 7)
    x, gl = _rows(300, K, dtype, 8), torch.tensor([180, 120])
    flat = torch.empty(x.numel() + shift, dtype=x.dtype, device=DEV)
    flat[shift:] = x.to(DEV).reshape(-1)
    out = torch.empty(300 * 96 + shift, dtype=x.dtype, device=DEV)[shift:].reshape(300, 96)
    y = pgg.moe_fwd_w4(flat[shift:].reshape(300, K), _pack(*w, 64, False), None, gl.to(DEV), out=out)
    want, bound = ref.w4_fwd(x, *w, 64, gl)
    ops_ref.assert_within(y, want, bound)
