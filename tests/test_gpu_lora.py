"""The shared projection with low-rank adapters against its 64-bit form."""
import math

import pytest
import torch

import ops_ref as ref
import permute_grouped_gemm_amd as pgg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _make(T, K, N, P, R, dtype, seed, order="runs"):
    gen = torch.Generator().manual_seed(seed)
    dt = ref.DTYPES[dtype]
    x = torch.randn((T, K), generator=gen).to(dt)
    w = (torch.randn((K, N), generator=gen) / math.sqrt(K)).to(dt)
    a = (torch.randn((P, R, K), generator=gen) / math.sqrt(K)).to(dt)
    b = torch.randn((P, R, N), generator=gen).to(dt)
    ids = torch.randint(-1, P, (T,), generator=gen)
    if order == "runs":
        ids = ids[torch.arange(T) // 37 * 37 % T]
    scales = 0.5 + torch.rand(P, generator=gen)
    return x, w, a, b, ids, scales


def _run(*args):
    args = [t.to(DEV) for t in args]
    ws = torch.empty(pgg.lora_workspace_size(*args), dtype=torch.uint8, device=DEV)
    y = pgg.lora_fwd(*args, workspace=ws)
    torch.cuda.synchronize()
    assert pgg.read_device_error(ws) == (pgg.DEV_OK, 0)
    return y


# tokens, K, N, adapters, rank: single tokens; a few; the boundaries of the
# tiles (32, 64, 128, 256); odd sizes; ranks that do not fill a step
SHAPES = [(1, 1, 1, 1, 1), (1, 2048, 264, 4, 8), (2, 67, 33, 3, 5), (16, 520, 300, 20, 16), (33, 256, 129, 2, 17),
          (64, 1000, 70, 70, 3), (65, 129, 257, 5, 33), (130, 72, 136, 1, 64), (300, 264, 520, 7, 12), (257, 99, 101, 3, 40),
          (600, 67, 35, 4, 9), (600, 72, 35, 4, 16), (520, 67, 40, 3, 70), (90, 67, 64, 3, 8), (1100, 128, 64, 6, 16),
          (2100, 67, 35, 4, 9), (100, 264, 520, 5, 12), (128, 67, 35, 9, 16), (129, 67, 35, 9, 16), (256, 520, 136, 30, 33),
          (2100, 264, 40, 60, 16), (2060, 67, 35, 40, 20), (2055, 130, 72, 50, 40), (300, 72, 40, 3, 500)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,K,N,P,R", SHAPES)
def test_lora(T, K, N, P, R, dtype):
    for order in ("runs", "mixed"):
        args = _make(T, K, N, P, R, dtype, T + K, order)
        y = _run(*args)
        want, bound = ref.lora(*args)
        assert y.dtype == args[0].dtype
        ref.assert_within(y, want, bound, order)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_lora_large_tiles(dtype):
    # enough 256 x 256 tiles for the direct-to-LDS kernel, rows and columns that end inside one
    args = _make(2300, 72, 5000, 9, 16, dtype, 5)
    y = _run(*args)
    want, bound = ref.lora(*args)
    ref.assert_within(y, want, bound)


@pytest.mark.parametrize("T", [20, 200, 2300])
def test_no_adapter_is_the_projection_alone(T):
    x, w, a, b, ids, s = _make(T, 136, 5000 if T > 2000 else 264, 3, 8, "bf16", 3)
    plain = _run(x, w, a, b, torch.full_like(ids, -1), s)
    zero = _run(x, w, torch.zeros_like(a), b, ids, s)
    assert torch.equal(plain, zero)
    far = _run(x, w, a, b, torch.full_like(ids, -(1 << 62)), s)
    assert torch.equal(plain, far)


@pytest.mark.parametrize("T", [20, 200, 2300])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_values_of_one_adapter_stay_in_its_tokens(T, dtype):
    x, w, a, b, ids, s = _make(T, 136, 5000 if T > 2000 else 264, 5, 8, dtype, 4, "mixed")
    clean = _run(x, w, a, b, ids, s)
    a2, b2, s2, x2 = a.clone(), b.clone(), s.clone(), x.clone()
    a2[0, 3, 5] = math.nan
    b2[1, 2, 7] = math.inf
    s2[2] = math.nan
    x2[T // 2, 3] = math.inf
    got = _run(x2, w, a2, b2, ids, s2)
    touched = (ids >= 0) & (ids <= 2)
    touched[T // 2] = True
    assert torch.equal(clean[~touched.to(DEV)], got[~touched.to(DEV)])
    assert not got[(ids == 0).to(DEV)].isfinite().any()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_inner_products_beyond_the_range_of_fp16(dtype):
    # z of about 2e5 against b of about 6e-5: fp16 could not hold z
    x, w, a, b, ids, s = _make(40, 64, 48, 2, 4, dtype, 6)
    x, b = x * 8, (b.float() * 2.0 ** -14).to(b.dtype)
    s = s * 2.0 ** 15
    y = _run(x, w, a, b, ids, s)
    want, bound = ref.lora(x, w, a, b, ids, s)
    ref.assert_within(y, want, bound)


@pytest.mark.parametrize("T", [20, 300])
def test_inner_products_beyond_the_largest_bf16(T):
    # z = 2^64 * 255 * 2^56 * scale lies between bf16's largest value and fp32's
    x, w = torch.full((T, 8), 0.0).bfloat16(), torch.zeros((8, 16)).bfloat16()
    x[:, 0] = 2.0 ** 64
    a, b = torch.zeros((1, 4, 8)).bfloat16(), torch.full((1, 4, 16), 2.0 ** -100).bfloat16()
    a[0, 1, 0] = 255 * 2.0 ** 56
    args = (x, w, a, b, torch.zeros(T, dtype=torch.int64), torch.tensor([1.0037]))
    want, bound = ref.lora(*args)
    assert torch.isfinite(want).all()
    ref.assert_within(_run(*args), want, bound)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,K,N", [(8, 256, 128), (100, 128, 264), (300, 128, 264), (600, 72, 40)])
def test_operands_at_any_address(T, K, N, dtype):
    def moved(t):
        out = torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)[1:1 + t.numel()].view(t.shape)
        return out.copy_(t)
    args = _make(T, K, N, 5, 8, dtype, 12)
    out = moved(torch.zeros((T, N), dtype=args[0].dtype))
    pgg.lora_fwd(*[moved(t) for t in args], out=out)
    want, bound = ref.lora(*args)
    ref.assert_within(out, want, bound)


def test_token_rows_do_not_depend_on_the_batch_order():
    x, w, a, b, ids, s = _make(200, 136, 264, 5, 8, "bf16", 4, "mixed")
    y = _run(x, w, a, b, ids, s)
    order = torch.randperm(200, generator=torch.Generator().manual_seed(1))
    assert torch.equal(_run(x[order].contiguous(), w, a, b, ids[order].contiguous(), s), y[order.to(DEV)])


@pytest.mark.parametrize("T", [10, 300])
def test_an_id_past_the_adapters_sets_the_error_word(T):
    x, w, a, b, ids, s = [t.to(DEV) for t in _make(T, 64, 40, 3, 4, "f16", 2)]
    ws = torch.empty(pgg.lora_workspace_size(x, w, a, b, ids, s), dtype=torch.uint8, device=DEV)
    ids[7], ids[9] = 3, 1 << 50
    pgg.lora_fwd(x, w, a, b, ids, s, workspace=ws)
    assert pgg.read_device_error(ws) == (pgg.DEV_ADAPTER_RANGE, 7)
    ids[7] = ids[9] = 2
    pgg.lora_fwd(x, w, a, b, ids, s, workspace=ws)
    assert pgg.read_device_error(ws) == (pgg.DEV_OK, 0)


def test_lora_captures_into_a_graph_and_follows_its_stream():
    for T in (4, 300):
        args = [t.to(DEV) for t in _make(T, 256, 264, 5, 16, "bf16", 9)]
        ws = torch.empty(pgg.lora_workspace_size(*args), dtype=torch.uint8, device=DEV)
        y = pgg.lora_fwd(*args, workspace=ws)
        want = y.clone()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        again = pgg.lora_fwd(*args, stream=side)
        side.synchronize()
        assert torch.equal(again, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pgg.lora_fwd(*args, out=y, workspace=ws)
        for _ in range(3):
            y.fill_(math.nan)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)


def test_adapter_gradients_through_the_grouped_products():
    # tokens in adapter order make the adapters experts: dz = dy·Bᵀ is moe_dx, dB and
    # dA are moe_dw; fp32, so each product is off by gamma times its magnitudes
    T, K, N, P, R = 60, 48, 40, 3, 4
    x, w, a, b, _, s = _make(T, K, N, P, R, "f32", 7)
    counts = torch.tensor([25, 0, 35])
    ids = torch.repeat_interleave(torch.arange(P), counts)
    dy = torch.randn((T, N), generator=torch.Generator().manual_seed(8))
    eri, gl = torch.arange(T).to(DEV), counts.to(DEV)
    sc = s[ids][:, None]
    dz = pgg.moe_dx((dy * sc).to(DEV), b.to(DEV), eri, gl, T, 1)
    z = pgg.moe_fwd(x.to(DEV), a.transpose(1, 2).contiguous().to(DEV), eri, gl, 1)
    db = pgg.moe_dw(z, (dy * sc).to(DEV), eri, gl, 1)
    da = pgg.moe_dw(dz, x.to(DEV), eri, gl, 1)
    xd, ad, bd, dyd = x.double(), a.double(), b.double(), dy.double() * sc.double()
    for p in range(P):
        at = ids == p
        wz, wdz = xd[at] @ ad[p].t(), dyd[at] @ bd[p].t()
        ez = ref.gamma(K) * (xd[at].abs() @ ad[p].abs().t())
        edz = ref.gamma(N) * (dyd[at].abs() @ bd[p].abs().t()) + 2.0 ** -23 * (dyd[at].abs() @ bd[p].abs().t())
        ref.assert_within(db[p], wz.t() @ dyd[at], (ez.t() + (ref.gamma(T) + 2.0 ** -23) * wz.abs().t()) @ dyd[at].abs()
                          + 1e-30, "dB")
        ref.assert_within(da[p], wdz.t() @ xd[at], (edz.t() + ref.gamma(T) * wdz.abs().t()) @ xd[at].abs() + 1e-30, "dA")


def test_lora_refusals():
    x, w, a, b, ids, s = [t.to(DEV) for t in _make(8, 32, 16, 3, 4, "bf16", 1)]
    for call in (lambda: pgg.lora_fwd(x, w.half(), a, b, ids, s), lambda: pgg.lora_fwd(x, w[:31], a, b, ids, s),
                 lambda: pgg.lora_fwd(x, w, a[:, :, :31].contiguous(), b, ids, s),
                 lambda: pgg.lora_fwd(x, w, a, b[:2].contiguous(), ids, s),
                 lambda: pgg.lora_fwd(x, w, a, b[:, :3].contiguous(), ids, s),
                 lambda: pgg.lora_fwd(x, w, a, b, ids.int(), s), lambda: pgg.lora_fwd(x, w, a, b, ids[:7], s),
                 lambda: pgg.lora_fwd(x, w, a, b, ids, s.half()), lambda: pgg.lora_fwd(x, w, a, b, ids, s.cpu()),
                 lambda: pgg.lora_fwd(x.t(), w, a, b, ids, s), lambda: pgg.lora_fwd(x[:0], w, a, b, ids[:0], s),
                 lambda: pgg.lora_fwd(x, w, a, b, ids, s, out=torch.empty((8, 16), device=DEV))):
        with pytest.raises(pgg.PggError) as e:
            call()
        assert e.value.status == pgg.ERR_INVALID_ARG
    with pytest.raises(pgg.PggError) as e:
        pgg.lora_fwd(x, w, a, b, ids, s, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.status == pgg.ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(pgg.PggError) as e:
        pgg.lora_fwd(x, w, a.new_zeros((1, 1025, 32)), b.new_zeros((1, 1025, 16)), ids.clamp_max(0), s[:1])
    assert e.value.status == pgg.ERR_UNSUPPORTED
