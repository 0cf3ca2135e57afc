"""Products with 4-bit weights where a wrong element, scale or zero point cannot hide
behind the rounding: whole numbers, single weights, and the bound of the additions as
the kernels chain them.  What a mistake would do is tried on the 64-bit form, on the CPU."""
import pytest
import torch

import block_ref as ref
import ops_ref
import permute_grouped_gemm_amd as pgg
from test_gpu_w4 import DEV, _pack, _rows, _weights

# experts' rows: the tiles of 16, 32 and 64 rows, with experts left out
COUNTS = [[1], [3, 0, 2], [20, 0, 20], [150, 0, 50], [0, 0, 0, 0, 0, 0, 100, 0]]
LENGTHS = [160, 1403, 3600, 7168]
KINDS = [(32, True), (64, False), (64, True), (128, True), (256, False), (1024, True)]


def _whole(counts, K, gs, dtype, zeros, N=70):
    """Whole numbers times powers of two of each group and column: every sum is a
    multiple of 1/4 below K * 15 * 2 * 8 < 2^22, so exact in fp32 in any order."""
    gen = torch.Generator().manual_seed(K + gs)
    G, S, T = len(counts), -(-K // gs), ops_ref.DTYPES[dtype]
    codes = torch.randint(0, 16, (G, K, N), generator=gen, dtype=torch.uint8)
    scales = (2.0 ** torch.randint(-2, 4, (G, S, N), generator=gen)).to(T)
    z = torch.randint(0, 16, (G, S, N), generator=gen, dtype=torch.uint8) if zeros else None
    x = torch.tensor([-2, -1, 1, 2])[torch.randint(0, 4, (sum(counts), K), generator=gen)].to(T)
    return x, codes, scales, z


def _run(x, codes, scales, z, gs, gl):
    return pgg.moe_fwd_w4(x.to(DEV), _pack(codes, scales, z, gs, False), None, gl.to(DEV)).cpu()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_whole_numbers(counts, K, dtype):
    gl = torch.tensor(counts)
    for gs, zeros in KINDS:
        s = _whole(counts, K, gs, dtype, zeros)
        want, _ = ref.w4_product(*s, gs, gl)
        assert torch.equal(_run(*s, gs, gl), want.to(s[0].dtype)), (gs, zeros)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_one_weight_to_a_column(counts, K, dtype):
    # a power of two, so that the result is an element of x as it stands, all its bits
    gen = torch.Generator().manual_seed(K)
    G, N, T = len(counts), 200, ops_ref.DTYPES[dtype]
    at = torch.randint(0, K, (G, N), generator=gen)
    at[:, :9] = torch.tensor([0, 1, 31, 32, 127, 128, K - 9, K - 2, K - 1])
    shift = torch.randint(0, 4, (G, 1, N), generator=gen)
    codes = torch.zeros((G, K, N), dtype=torch.uint8).scatter(1, at[:, None], (1 << shift).to(torch.uint8))
    x = torch.randn((sum(counts), K), generator=gen).to(T)
    gl = torch.tensor(counts)
    g = torch.repeat_interleave(torch.arange(G), gl)
    for gs in (32, 64, 128, 512):
        S = -(-K // gs)
        scales = (2.0 ** -(3 + torch.arange(S) % 3).float())[None, :, None].expand(G, S, N).to(T).contiguous()
        y = _run(x, codes, scales, torch.zeros((G, S, N), dtype=torch.uint8), gs, gl)
        factor = 2.0 ** (shift[:, 0] - 3 - at // gs % 3).double()
        want = torch.gather(x, 1, at[g]).double() * factor[g]
        assert torch.equal(y, want.to(T)), gs


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 40])
def test_small_fp32_x(rows):
    # all 24 bits down to 2^-90; under that what lies below 2^-133 is cut off
    K, scale = 128, 2.0 ** 60
    w = _pack(torch.eye(K, dtype=torch.uint8)[None], torch.full((1, 1, K), scale),
              torch.zeros((1, 1, K), dtype=torch.uint8), 128, False)
    for e in (90, 112, 124, 132):
        x = (torch.randn((rows, K), generator=torch.Generator().manual_seed(e), dtype=torch.float64) * 2.0 ** -e).float()
        y = pgg.moe_fwd_w4(x.to(DEV), w, None, torch.tensor([rows], device=DEV)).cpu().double()
        cut = torch.where(x.abs() < 2.0 ** -110, 2.0 ** -133, 0.0).double() * scale
        assert bool(((y - x.double() * scale).abs() <= cut).all()), e


def _chained(x, codes, scales, z, gs, gl):
    """w4_fwd with the bound of the chain that the kernels add in: a group's products
    (fp32 x in three parts), the groups of a wave, and 16 for waves, splits and the
    zero point's product."""
    y, err = ref.w4_product(x, codes, scales, z, gs, gl)
    K, inside = x.shape[1], min(gs, 128)
    depth = (3 if x.dtype == torch.float32 else 1) * inside + -(-K // inside) + 16
    return y, ops_ref.rounded(y, err * (ops_ref.gamma(depth) / ops_ref.gamma(K)), x.dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", [3600, 7168])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_long_reductions(counts, K, dtype):
    gl = torch.tensor(counts)
    for gs, zeros in KINDS[:4]:
        s = (_rows(sum(counts), K, dtype, K + 1), *_weights(len(counts), K, 64, gs, dtype, zeros, K))
        want, bound = _chained(*s, gs, gl)
        ops_ref.assert_within(_run(*s, gs, gl), want, bound, f"groups of {gs}")


def _mistakes(x, codes, scales, z):
    """The same inputs with one mistake each."""
    short = x.clone()
    short[:, -1] = 0
    yield "the last element left out", (short, codes, scales, z)
    if scales.shape[1] > 1:
        shifted = scales.clone()
        shifted[:, -1] = scales[:, -2]
        yield "the last group with its neighbour's scale", (x, codes, shifted, z)
    if z is not None and z.shape[1] > 1:
        shifted = z.clone()
        shifted[:, -1] = z[:, -2]
        yield "the last group with its neighbour's zero point", (x, codes, scales, shifted)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("counts", COUNTS[1:3], ids=str)
def test_mistakes_show(counts, K, dtype):
    gl = torch.tensor(counts)
    for gs, zeros in KINDS:
        s = _whole(counts, K, gs, dtype, zeros)
        want = ref.w4_product(*s, gs, gl)[0].to(s[0].dtype)
        for what, bad in _mistakes(*s):
            assert not torch.equal(ref.w4_product(*bad, gs, gl)[0].to(want.dtype), want), (what, gs)
    if K < 3600:
        return
    for gs, zeros in KINDS[:4]:
        s = (_rows(sum(counts), K, dtype, K + 1), *_weights(len(counts), K, 64, gs, dtype, zeros, K))
        want, bound = _chained(*s, gs, gl)
        for what, bad in _mistakes(*s):
            off = (ref.w4_product(*bad, gs, gl)[0] - want).abs() - ops_ref.U[s[0].dtype] * want.abs()
            assert bool((off > bound).any()), (what, gs)
