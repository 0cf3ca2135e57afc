"""Products with 4-bit weights against their 64-bit forms."""
import math

import pytest
import torch

import block_ref as ref
import ops_ref
import permute_grouped_gemm_amd as pgg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _weights(G, K, N, gs, dtype, zeros, seed):
    gen = torch.Generator().manual_seed(seed)
    S = -(-K // gs)
    codes = torch.randint(0, 16, (G, K, N), generator=gen, dtype=torch.uint8)
    scales = ((0.5 + torch.rand((G, S, N), generator=gen)) / math.sqrt(K) / 4).to(ops_ref.DTYPES[dtype])
    z = torch.randint(0, 16, (G, S, N), generator=gen, dtype=torch.uint8) if zeros else None
    return codes, scales, z


def _pack(codes, scales, z, gs, gated):
    return pgg.w4_pack(codes.to(DEV), scales.to(DEV), gs, zeros=None if z is None else z.to(DEV), gated=gated)


def _rows(T, K, dtype, seed):
    return torch.randn((T, K), generator=torch.Generator().manual_seed(seed)).to(ops_ref.DTYPES[dtype])


def _routing(counts, topk, row_idx_type, seed):
    M = sum(counts)
    eri = torch.randperm(M, generator=torch.Generator().manual_seed(seed))
    return eri, torch.tensor(counts)


def _ws(*args):
    size = pgg.w4_workspace_size(*args)
    return torch.full((size,), 0xAB, dtype=torch.uint8, device=DEV)


def _check_fwd(counts, K, N, gs, dtype, zeros, indexed=None, topk=1, seed=0):
    G, M = len(counts), sum(counts)
    w = _weights(G, K, N, gs, dtype, zeros, seed)
    x = _rows(M // topk, K, dtype, seed + 1)
    eri, gl = _routing(counts, topk, indexed, seed)
    kw = {} if indexed is None else dict(topk=topk, eri=eri, row_idx_type=indexed)
    args = (x.to(DEV), _pack(*w, gs, False), None if indexed is None else eri.to(DEV), gl.to(DEV), topk, indexed or 0)
    ws = _ws(*args)
    y = pgg.moe_fwd_w4(*args, workspace=ws)
    torch.cuda.synchronize()
    assert pgg.read_device_error(ws) == (pgg.DEV_OK, 0)
    want, bound = ref.w4_fwd(x, *w, gs, gl, **kw)
    assert y.dtype == x.dtype
    ops_ref.assert_within(y, want, bound, "y")


def _check_glu(counts, K, F, gs, dtype, zeros, indexed, topk, act, seed=0):
    G, M = len(counts), sum(counts)
    w = _weights(G, K, 2 * F, gs, dtype, zeros, seed)
    x = _rows(M // topk, K, dtype, seed + 1)
    eri, gl = _routing(counts, topk, indexed, seed)
    args = (x.to(DEV), _pack(*w, gs, True), eri.to(DEV), gl.to(DEV), topk, indexed)
    ws = _ws(*args)
    h = pgg.moe_glu_w4(*args, act=act, workspace=ws)
    torch.cuda.synchronize()
    assert pgg.read_device_error(ws) == (pgg.DEV_OK, 0)
    want, bound = ref.w4_glu(x, *w, gs, gl, name=act, topk=topk, eri=eri, row_idx_type=indexed)
    ops_ref.assert_within(h, want, bound, "h")


# one row; odd reductions and columns around the tiles' edges; groups that end
# inside a tile; empty experts in front, between and behind; many rows
SHAPES = [([1], 32, 1), ([1], 1, 5), ([1], 7168, 64), ([3], 130, 67), ([16], 128, 64), ([17, 0, 1], 200, 130),
          ([0, 33, 0, 0, 5, 0], 257, 63), ([64, 1], 384, 192), ([5] * 40, 96, 40), ([100, 31], 640, 96),
          ([130, 0, 70], 1000, 200), ([2] * 300, 64, 33), ([600], 512, 128), ([255, 257], 333, 129)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("counts,K,N", SHAPES, ids=lambda v: str(v)[:20])
def test_fwd(counts, K, N, dtype):
    for gs, zeros in ((32, True), (64, False), (128, True), (256, False)):
        _check_fwd(counts, K, N, gs, dtype, zeros, seed=K + gs)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("counts,K,F,topk", [([2], 64, 16, 2), ([8, 0, 8], 128, 33, 4), ([30, 1, 0, 17], 300, 50, 2),
                                             ([90, 110], 257, 64, 5), ([3] * 40, 136, 7, 3), ([1000, 24], 160, 96, 8),
                                             ([2500, 0, 2500], 96, 40, 1), ([5] * 280, 64, 20, 7)],
                         ids=lambda v: str(v)[:20])
def test_glu(counts, K, F, topk, dtype):
    for n, (gs, zeros, act) in enumerate(((32, False, "silu"), (64, True, "gelu_tanh"), (128, False, "silu"))):
        _check_glu(counts, K, F, gs, dtype, zeros, n % 2, topk, act, seed=K + n)


@pytest.mark.parametrize("indexed,topk", [(0, 1), (1, 1), (0, 3), (1, 3)])
def test_fwd_with_an_index(indexed, topk):
    _check_fwd([12, 0, 30, 3], 200, 70, 64, "bf16", True, indexed, topk)
    _check_fwd([3000, 1500, 600], 64, 70, 32, "f16", False, indexed, topk)


def test_codes_are_exact():
    # whole numbers throughout: every sum is exact in fp32, so is the result
    for dtype, std in (("f32", 8), ("f16", 2), ("bf16", 1)):
        G, K, N, gs = 2, 160, 70, 32
        gen = torch.Generator().manual_seed(1)
        codes = torch.randint(0, 16, (G, K, N), generator=gen, dtype=torch.uint8)
        z = torch.randint(0, 16, (G, 5, N), generator=gen, dtype=torch.uint8)
        scales = torch.ones((G, 5, N), dtype=ops_ref.DTYPES[dtype])
        x = torch.randint(-std, std + 1, (40, K), generator=gen).to(ops_ref.DTYPES[dtype])
        gl = torch.tensor([21, 19])
        y = pgg.moe_fwd_w4(x.to(DEV), _pack(codes, scales, z, gs, False), None, gl.to(DEV))
        want, _ = ref.w4_product(x, codes, scales, z, gs, gl)
        assert torch.equal(y.cpu(), want.to(y.dtype))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [3, 40, 300])
def test_infinities_and_nan_stay_in_their_rows(dtype, rows):
    K, N, gs = 288, 70, 32
    codes, scales, z = _weights(1, K, N, gs, dtype, True, 3)
    codes[:, :, 5] = 15
    z[:, :, 5] = 3
    x = _rows(rows, K, dtype, 4)
    x[0, 7], x[1, K - 1], x[2, 200] = math.inf, -math.inf, math.nan
    gl = torch.tensor([rows])
    y = pgg.moe_fwd_w4(x.to(DEV), _pack(codes, scales, z, gs, False), None, gl.to(DEV)).cpu()
    want, bound = ref.w4_fwd(x, codes, scales, z, gs, gl)     # an infinity times a weight of 0 is NaN
    assert torch.equal(y[:3].isnan(), want[:3].isnan()) and torch.equal(y[:2].double().nan_to_num(0.0, 1.0, -1.0),
                                                                        want[:2].nan_to_num(0.0, 1.0, -1.0))
    assert y[0, 5] == math.inf and y[1, 5] == -math.inf and bool(y[2].isnan().all())
    ops_ref.assert_within(y[3:], want[3:], bound[3:])


def test_large_and_small_values():
    K, N = 128, 64
    for dtype, big in (("f16", 6e4), ("bf16", 1e30), ("f32", 1e30)):
        codes, scales, z = _weights(1, K, N, 128, dtype, True, 3)
        scales = scales * 2.0 ** -8
        x = _rows(20, K, dtype, 4)
        x[0] = torch.where(x[0] > 0, big, -big)
        x[1] *= 2.0 ** -10
        gl = torch.tensor([20])
        y = pgg.moe_fwd_w4(x.to(DEV), _pack(codes, scales, z, 128, False), None, gl.to(DEV))
        want, bound = ref.w4_fwd(x, codes, scales, z, 128, gl)
        ops_ref.assert_within(y, want, bound)


def test_bits_above_the_code_are_ignored():
    codes, scales, z = _weights(1, 64, 32, 32, "bf16", True, 5)
    x, gl = _rows(4, 64, "bf16", 6).to(DEV), torch.tensor([4], device=DEV)
    a = pgg.moe_fwd_w4(x, _pack(codes, scales, z, 32, False), None, gl)
    b = pgg.moe_fwd_w4(x, _pack(codes | 0x50, scales, z | 0xA0, 32, False), None, gl)
    assert torch.equal(a, b)


def test_repeated_calls_give_the_same_bits():
    codes, scales, z = _weights(4, 1024, 200, 128, "bf16", True, 5)
    w = _pack(codes, scales, z, 128, True)
    eri, gl = _routing([5, 60, 0, 31], 3, 0, 1)
    x = _rows(32, 1024, "bf16", 6).to(DEV)
    args = (x, w, eri.to(DEV), gl.to(DEV), 3)
    first = pgg.moe_glu_w4(*args)
    for _ in range(5):
        assert torch.equal(pgg.moe_glu_w4(*args, workspace=_ws(*args)), first)


def test_unaligned_tensors():
    # data that starts on no 16-byte boundary
    for dtype in ("bf16", "f32"):
        codes, scales, z = _weights(2, 256, 96, 64, dtype, True, 7)
        x = _rows(50, 256, dtype, 8)
        flat = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)
        flat[1:] = x.to(DEV).reshape(-1)
        gl = torch.tensor([20, 30])
        store = torch.empty(50 * 96 + 3, dtype=x.dtype, device=DEV)
        out = store[3:].reshape(50, 96)
        y = pgg.moe_fwd_w4(flat[1:].reshape(50, 256), _pack(codes, scales, z, 64, False), None, gl.to(DEV), out=out)
        want, bound = ref.w4_fwd(x, codes, scales, z, 64, gl)
        ops_ref.assert_within(y, want, bound)


def test_nothing_is_written_beside_the_result():
    codes, scales, z = _weights(3, 130, 67, 32, "bf16", False, 7)
    x, gl = _rows(37, 130, "bf16", 8).to(DEV), torch.tensor([20, 0, 17], device=DEV)
    store = torch.full((39, 67), 7.0, dtype=torch.bfloat16, device=DEV)
    y = pgg.moe_fwd_w4(x, _pack(codes, scales, z, 32, False), None, gl, out=store[1:38])
    assert bool((store[0] == 7).all()) and bool((store[38] == 7).all())
    assert torch.equal(y, pgg.moe_fwd_w4(x, _pack(codes, scales, z, 32, False), None, gl))


def test_bad_tables_are_reported():
    codes, scales, z = _weights(2, 64, 32, 32, "bf16", False, 9)
    w = _pack(codes, scales, z, 32, False)
    for M in (30, 6000):
        x = _rows(M, 64, "bf16", 1).to(DEV)
        eri = torch.arange(M, device=DEV)
        half = M // 2
        for counts, index, code in (([half, half - 1], eri, pgg.DEV_GROUP_SUM), ([-1, M + 1], eri, pgg.DEV_GROUP_NEGATIVE),
                                    ([half, half], torch.where(eri == 4, M, eri), pgg.DEV_INDEX_RANGE),
                                    ([half, half], torch.where(eri == 4, 7, eri), pgg.DEV_INDEX_DUP),
                                    ([1 << 40, 3], eri, pgg.DEV_GROUP_SUM)):
            for kind in (None, 0, 1):
                if kind is None and index is not eri:
                    continue
                gl = torch.tensor(counts, device=DEV)
                args = (x, w, None if kind is None else index, gl, 1, kind or 0)
                ws = _ws(*args)
                pgg.moe_fwd_w4(*args, workspace=ws)
                assert pgg.read_device_error(ws)[0] == code, (counts, kind)


def test_refusals():
    codes, scales, z = (None if t is None else t.to(DEV) for t in _weights(2, 64, 32, 32, "bf16", True, 9))
    for bad in (dict(codes=codes.int()), dict(codes=codes[0]), dict(codes=codes.cpu()), dict(scales=scales[:, :1]),
                dict(scales=scales.double()), dict(zeros=z[:1]), dict(zeros=z.int()), dict(group_size=48),
                dict(codes=codes.transpose(1, 2))):
        kw = {**dict(codes=codes, scales=scales, group_size=32, zeros=z), **bad}
        with pytest.raises(pgg.PggError):
            pgg.w4_pack(**kw)
    w, g = pgg.w4_pack(codes, scales, 32, zeros=z), pgg.w4_pack(codes, scales, 32, gated=True)
    x, gl = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV), torch.tensor([3, 1], device=DEV)
    assert w.shape == (2, 64, 32) and w.group_size == 32 and not w.gated and g.gated and w.dtype == torch.bfloat16
    eri = torch.arange(4, device=DEV)
    for call in (lambda: pgg.moe_fwd_w4(x, g, None, gl), lambda: pgg.moe_glu_w4(x, w, None, gl),
                 lambda: pgg.moe_fwd_w4(x.half(), w, None, gl), lambda: pgg.moe_fwd_w4(x[:, :32].contiguous(), w, None, gl),
                 lambda: pgg.moe_fwd_w4(x, w, None, gl, 2), lambda: pgg.moe_fwd_w4(x, w, eri[:3], gl),
                 lambda: pgg.moe_fwd_w4(x, w, eri.int(), gl), lambda: pgg.moe_fwd_w4(x, w, None, gl[:1]),
                 lambda: pgg.moe_fwd_w4(x, codes, None, gl), lambda: pgg.moe_glu_w4(x, g, None, gl, act="relu"),
                 lambda: pgg.moe_fwd_w4(x, w, None, gl, out=torch.zeros((4, 31), device=DEV).bfloat16()),
                 lambda: pgg.moe_fwd_w4(x, w, None, gl, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises(pgg.PggError):
            call()
