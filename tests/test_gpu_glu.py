"""The experts' gated product and its gradient against their 64-bit forms."""
import math

import pytest
import torch

import ops_ref as ref
import permute_grouped_gemm_amd as pgg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _routing(batch, topk, G, seed, row_idx_type, skew=0.0, empty=0):
    gen = torch.Generator().manual_seed(seed)
    usable = torch.randperm(G, generator=gen)[:G - empty]
    w = torch.zeros(G)
    w[usable] = (torch.arange(1, G - empty + 1).float()) ** -skew
    ids = torch.stack([torch.multinomial(w, topk, generator=gen) for _ in range(batch)]).reshape(-1)
    eri = torch.sort(ids, stable=True).indices
    if row_idx_type == 1:
        back = torch.empty_like(eri)
        back[eri] = torch.arange(eri.numel())
        eri = back
    return eri, torch.bincount(ids, minlength=G)


def _make(batch, topk, G, K, F, dtype, seed, row_idx_type=0, skew=0.0, empty=0):
    eri, gl = _routing(batch, topk, G, seed, row_idx_type, skew, empty)
    gen = torch.Generator().manual_seed(seed + 1)
    dt = ref.DTYPES[dtype]
    x = torch.randn((batch, K), generator=gen).to(dt)
    w = (torch.randn((G, K, 2 * F), generator=gen) * 1.5 / math.sqrt(K)).to(dt)
    return x, w, eri, gl


def _run(x, w, eri, gl, topk, row_idx_type, act, save=True):
    args = [t.to(DEV) for t in (x, w, eri, gl)]
    ws = torch.empty(pgg.glu_workspace_size(*args, topk, row_idx_type), dtype=torch.uint8, device=DEV)
    got = pgg.moe_glu(*args, topk, row_idx_type, act=act, save_gate_up=save, workspace=ws)
    torch.cuda.synchronize()
    assert pgg.read_device_error(ws) == (pgg.DEV_OK, 0)
    return got


# batch, topk, experts, K, F: one token; odd sizes whose rows start anywhere;
# few rows (with the reduction split and not) and many rows per expert; tiles
# that end inside K, F and the expert's rows
GLU = [(1, 1, 1, 1, 1), (1, 2, 4, 64, 32), (5, 2, 3, 33, 7), (16, 8, 16, 2048, 128), (17, 3, 5, 1000, 72),
       (64, 2, 4, 256, 64), (100, 4, 6, 520, 200), (257, 2, 3, 129, 65), (400, 2, 2, 328, 136),
       (300, 1, 1, 200, 264), (200, 1, 1, 40, 24), (520, 1, 2, 64, 8), (260, 1, 1, 136, 520),
       (600, 1, 1, 67, 35), (600, 1, 1, 72, 35), (600, 1, 1, 67, 40), (90, 1, 1, 67, 40),
       (8, 2, 256, 40, 8), (8, 2, 257, 40, 8), (512, 8, 100, 16, 8), (513, 8, 100, 24, 7),
       (60, 4, 5, 520, 200), (100, 2, 5, 67, 40), (1200, 8, 300, 24, 8), (41, 2, 2, 1024, 136)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("batch,topk,G,K,F", GLU)
def test_glu(batch, topk, G, K, F, dtype):
    for row_idx_type, act in ((0, "silu"), (1, "gelu_tanh")):
        x, w, eri, gl = _make(batch, topk, G, K, F, dtype, K + F, row_idx_type, skew=1.0, empty=min(1, G - topk))
        h, gu = _run(x, w, eri, gl, topk, row_idx_type, act)
        wh, eh, wy, ey = ref.glu(x, w, eri, gl, topk, row_idx_type, act)
        assert h.dtype == gu.dtype == x.dtype
        ref.assert_within(h, wh, eh, f"h {act}")
        ref.assert_within(gu, wy, ey, f"gate_up {act}")
        assert torch.equal(_run(x, w, eri, gl, topk, row_idx_type, act, save=False), h)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("batch,topk,G,K,F", [(16, 4, 8, 1024, 96), (300, 2, 2, 192, 160), (200, 2, 3, 67, 35)])
def test_glu_products_are_exact_on_whole_numbers(batch, topk, G, K, F, dtype):
    # values of -2..2 over K with |sum| at most 4 K < 2^11: gate_up is exact where it
    # fits the type, so every operand element is where it belongs
    K = min(K, 60) if dtype != "f32" else K
    gen = torch.Generator().manual_seed(3)
    eri, gl = _routing(batch, topk, G, 4, 0, 1.0)
    dt = ref.DTYPES[dtype]
    x = torch.randint(-2, 3, (batch, K), generator=gen).to(dt)
    w = torch.randint(-2, 3, (G, K, 2 * F), generator=gen).to(dt)
    _, gu = _run(x, w, eri, gl, topk, 0, "silu")
    want = ref.glu(x, w, eri, gl, topk, 0, "silu")[2].to(dt)
    assert torch.equal(gu.cpu(), want)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_values_of_one_expert_stay_in_its_rows(dtype):
    # infinities and NaN in an expert's weights, and in a token's row, reach only
    # the rows that read them
    x, w, eri, gl = _make(90, 2, 3, 136, 72, dtype, 8)
    clean = _run(x, w, eri, gl, 2, 0, "silu")
    ends = gl.cumsum(0)
    w2, x2 = w.clone(), x.clone()
    w2[1, 5, 3] = math.inf
    w2[1, 7, 90] = math.nan
    x2[13, 2] = math.nan
    got = _run(x2, w2, eri, gl, 2, 0, "silu")
    touched = torch.zeros(180, dtype=torch.bool)
    touched[int(ends[0]):int(ends[1])] = True
    touched |= ref.positions(eri, 0) // 2 == 13
    for u, v in zip(clean, got):
        assert torch.equal(u[~touched.to(DEV)], v[~touched.to(DEV)])


def test_extreme_gates():
    # act at the ends of its range: large negative gates give 0, large positive ones the gate
    K, F = 32, 32
    x = torch.ones((4, K))
    w = torch.zeros((1, K, 2 * F))
    w[0, 0, :F] = torch.tensor([-1e4, 1e4, -200.0, 200.0] * (F // 4))
    w[0, 0, F:] = 2.0
    eri, gl = torch.arange(4), torch.tensor([4])
    for act in ("silu", "gelu_tanh"):
        h, _ = _run(x, w, eri, gl, 1, 0, act)
        want = torch.tensor([0.0, 2e4, 0.0, 400.0] * (F // 4)).expand(4, F)
        assert torch.equal(h.cpu().abs(), want)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("batch,topk,G,D,F", [(1, 1, 1, 1, 1), (1, 2, 4, 64, 32), (5, 2, 3, 33, 7), (40, 2, 5, 200, 136),
                                              (333, 2, 7, 203, 141), (300, 1, 1, 264, 200), (257, 2, 2, 520, 264),
                                              (600, 2, 3, 192, 320), (200, 1, 1, 40, 24), (520, 1, 2, 64, 8),
                                              (600, 1, 1, 67, 35), (1100, 1, 2, 135, 130), (8, 2, 256, 40, 8),
                                              (8, 2, 257, 300, 8), (125, 2, 5, 203, 35), (120, 2, 5, 520, 264),
                                              (1800, 8, 300, 40, 8)])
def test_glu_grad(batch, topk, G, D, F, dtype):
    _, gl = _routing(batch, topk, G, D + F, 0, 1.0, min(1, G - topk))
    gen = torch.Generator().manual_seed(D)
    dt, M = ref.DTYPES[dtype], batch * topk
    gy = torch.randn((M, D), generator=gen).to(dt)
    w = (torch.randn((G, F, D), generator=gen) / math.sqrt(D)).to(dt)
    gu = (torch.randn((M, 2 * F), generator=gen) * 1.5).to(dt)
    for act in ("silu", "gelu_tanh"):
        args = [t.to(DEV) for t in (gy, w, gu, gl)]
        ws = torch.empty(pgg.glu_grad_workspace_size(*args), dtype=torch.uint8, device=DEV)
        grad, h = pgg.moe_glu_grad(*args, act=act, workspace=ws)
        torch.cuda.synchronize()
        assert pgg.read_device_error(ws) == (pgg.DEV_OK, 0)
        wg, eg, wh, eh = ref.glu_grad(gy, w, gu, gl, act)
        ref.assert_within(grad, wg, eg, f"grad_gate_up {act}")
        ref.assert_within(h, wh, eh, f"h {act}")
        only, none = pgg.moe_glu_grad(*args, act=act, want_h=False)
        assert none is None and torch.equal(only, grad)


def test_glu_grad_against_differences():
    # loss = sum(gy * (h W2)); central differences over gate_up of the 64-bit
    # forward, error step^2 / 6 times the third derivative (below 8 times the
    # coefficient), and the loss's rounding over the step
    gen = torch.Generator().manual_seed(4)
    G, D, F, gl = 2, 24, 8, torch.tensor([3, 2])
    gy, w = torch.randn((5, D), generator=gen), torch.randn((G, F, D), generator=gen) / math.sqrt(D)
    gu = torch.randn((5, 2 * F), generator=gen)
    for act in ("silu", "gelu_tanh"):
        grad, _ = pgg.moe_glu_grad(gy.to(DEV), w.to(DEV), gu.to(DEV), gl.to(DEV), act=act)
        owner = torch.tensor([0, 0, 0, 1, 1])
        dh = torch.stack([w[owner[i]].double() @ gy[i].double() for i in range(5)])

        def loss(v):
            return (ref.act(act, v[:, :F])[0] * v[:, F:] * dh).sum()

        step, bound = 1e-4, rounded_bound(gy, w, gu, gl, act)
        for i in range(5):
            for f in range(2 * F):
                hi, lo = gu.double(), gu.double()
                hi[i, f] += step
                lo[i, f] -= step
                diff = (loss(hi) - loss(lo)) / (2 * step)
                coef = float(dh.abs().max() * gu.abs().max())
                assert abs(float(grad[i, f]) - float(diff)) <= 8 * coef * step ** 2 + 1e-12 / step + float(bound[i, f])


def rounded_bound(gy, w, gu, gl, act):
    return ref.glu_grad(gy, w, gu, gl, act)[1]


def _moved(t):
    """The same values at an address one element past an aligned one."""
    big = torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)
    out = big[1:1 + t.numel()].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("batch,topk,G,K,F", [(16, 4, 8, 128, 64), (60, 4, 5, 128, 64), (300, 2, 2, 128, 64),
                                              (600, 1, 1, 72, 40)])
def test_operands_at_any_address(batch, topk, G, K, F, dtype):
    x, w, eri, gl = _make(batch, topk, G, K, F, dtype, 31)
    wh, eh, wy, ey = ref.glu(x, w, eri, gl, topk, 0, "silu")
    M = batch * topk
    h, gu = _moved(torch.zeros((M, F), dtype=x.dtype)), _moved(torch.zeros((M, 2 * F), dtype=x.dtype))
    pgg.moe_glu(_moved(x), _moved(w), eri.to(DEV), gl.to(DEV), topk, out=h, gate_up=gu)
    ref.assert_within(h, wh, eh, "h")
    ref.assert_within(gu, wy, ey, "gate_up")
    w2 = w[:, :, :F].transpose(1, 2).contiguous()          # [G, F, K]
    gy, gu = x.repeat_interleave(topk, 0).contiguous(), gu.cpu()
    out = _moved(torch.zeros((M, 2 * F), dtype=x.dtype))
    grad, hh = pgg.moe_glu_grad(_moved(gy), _moved(w2), _moved(gu), gl.to(DEV), out=out)
    wg, eg, wh, eh = ref.glu_grad(gy, w2, gu, gl, "silu")
    ref.assert_within(grad, wg, eg, "grad")
    ref.assert_within(hh, wh, eh, "h")


@pytest.mark.parametrize("row_idx_type", [0, 1])
@pytest.mark.parametrize("batch,G", [(20, 4), (80, 4), (20, 300), (700, 4)])
def test_wrong_routing_sets_the_error_word(batch, G, row_idx_type):
    # few rows with few and many groups, and many rows
    x, w, eri, gl = _make(batch, 2, G, 64, 32, "bf16", 6, row_idx_type)
    args = [t.to(DEV) for t in (x, w)]
    one = torch.zeros_like(gl)
    one[1] = 1
    for bad_eri, bad_gl, code in ((eri, gl + one, pgg.DEV_GROUP_SUM), (eri, gl - 100000 * one, pgg.DEV_GROUP_NEGATIVE),
                                  (eri, gl + (1 << 40) * one, pgg.DEV_GROUP_SUM),
                                  (eri.clone().index_fill_(0, torch.tensor([5]), 2 * batch), gl, pgg.DEV_INDEX_RANGE),
                                  (eri.clone().index_fill_(0, torch.tensor([5]), -1), gl, pgg.DEV_INDEX_RANGE),
                                  (eri.clone().index_fill_(0, torch.tensor([5, 6]), 7), gl, pgg.DEV_INDEX_DUP),
                                  (eri, gl, pgg.DEV_OK)):
        ws = torch.empty(pgg.glu_workspace_size(*args, eri.to(DEV), gl.to(DEV), 2, row_idx_type), dtype=torch.uint8,
                         device=DEV)
        pgg.moe_glu(*args, bad_eri.to(DEV), bad_gl.to(DEV), 2, row_idx_type, workspace=ws)
        assert pgg.read_device_error(ws)[0] == code


@pytest.mark.parametrize("M,G", [(40, 4), (200, 4), (40, 300), (700, 4)])
def test_wrong_counts_set_the_gradients_error_word(M, G):
    gl = torch.zeros(G, dtype=torch.int64)
    gl[1], gl[3] = M // 2, M - M // 2
    gy, gu = torch.zeros((M, 16), device=DEV), torch.zeros((M, 16), device=DEV)
    w2 = torch.zeros((G, 8, 16), device=DEV)
    ws = torch.empty(pgg.glu_grad_workspace_size(gy, w2, gu, gl.to(DEV)), dtype=torch.uint8, device=DEV)
    for at, by, want in ((1, 4, (pgg.DEV_GROUP_SUM, M + 4)), (3, -M, (pgg.DEV_GROUP_NEGATIVE, 3)), (0, 0, (pgg.DEV_OK, 0))):
        bad = gl.clone()
        bad[at] += by
        pgg.moe_glu_grad(gy, w2, gu, bad.to(DEV), workspace=ws)
        assert pgg.read_device_error(ws) == want


def test_glu_captures_into_a_graph():
    for shape in ((16, 4, 8, 1024, 96), (300, 2, 2, 192, 160)):
        batch, topk = shape[:2]
        x, w, eri, gl = [t.to(DEV) for t in _make(*shape, "bf16", 12)]
        ws = torch.empty(pgg.glu_workspace_size(x, w, eri, gl, topk), dtype=torch.uint8, device=DEV)
        h, gu = pgg.moe_glu(x, w, eri, gl, topk, save_gate_up=True, workspace=ws)
        want, want_gu = h.clone(), gu.clone()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            pgg.moe_glu(x, w, eri, gl, topk, out=h, gate_up=gu, workspace=ws)
        for _ in range(3):
            h.fill_(math.nan)
            gu.fill_(math.nan)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(h, want) and torch.equal(gu, want_gu)


def test_glu_grad_captures_into_a_graph():
    gen = torch.Generator().manual_seed(9)
    for M, G, D, F in ((40, 8, 200, 48), (700, 2, 192, 160), (600, 1, 67, 35)):
        gl = torch.full((G,), M // G)
        gy, w, gu = torch.randn((M, D), generator=gen), torch.randn((G, F, D), generator=gen), torch.randn((M, 2 * F), generator=gen)
        gy, w, gu, gl = [t.to(DEV) for t in (gy.half(), (w * 0.05).half(), gu.half(), gl)]
        ws = torch.empty(pgg.glu_grad_workspace_size(gy, w, gu, gl), dtype=torch.uint8, device=DEV)
        out, h = pgg.moe_glu_grad(gy, w, gu, gl, workspace=ws)
        want, want_h = out.clone(), h.clone()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            pgg.moe_glu_grad(gy, w, gu, gl, out=out, h=h, workspace=ws)
        for _ in range(3):
            out.fill_(math.nan)
            h.fill_(math.nan)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(h, want_h)


def test_glu_refusals():
    x, w, eri, gl = [t.to(DEV) for t in _make(8, 2, 4, 32, 16, "bf16", 1)]
    short = torch.empty(64, dtype=torch.uint8, device=DEV)
    for call in (lambda: pgg.moe_glu(x, w[:, :, :31].contiguous(), eri, gl, 2), lambda: pgg.moe_glu(x, w.half(), eri, gl, 2),
                 lambda: pgg.moe_glu(x, w, eri[:-1], gl, 2), lambda: pgg.moe_glu(x, w, eri, gl[:-1], 2),
                 lambda: pgg.moe_glu(x.t(), w, eri, gl, 2), lambda: pgg.moe_glu(x, w, eri.int(), gl, 2),
                 lambda: pgg.moe_glu(x, w, eri, gl, 2, 2), lambda: pgg.moe_glu(x, w, eri, gl, 2, act="relu"),
                 lambda: pgg.moe_glu(x, w, eri, gl, 2, out=torch.empty((16, 16), device=DEV)),
                 lambda: pgg.moe_glu(x, w, eri.cpu(), gl, 2), lambda: pgg.moe_glu(x[:, :31].contiguous(), w, eri, gl, 2)):
        with pytest.raises(pgg.PggError) as e:
            call()
        assert e.value.status == pgg.ERR_INVALID_ARG
    with pytest.raises(pgg.PggError) as e:
        pgg.moe_glu(x, w, eri, gl, 2, workspace=short)
    assert e.value.status == pgg.ERR_WORKSPACE_TOO_SMALL
    big = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    with pytest.raises(pgg.PggError) as e:
        pgg.moe_glu(x, w, eri, gl, 2, workspace=big[8:])
    assert e.value.status == pgg.ERR_MISALIGNED
    gy, w2, gu = x.new_zeros((16, 24)), w.new_zeros((4, 16, 24)), x.new_zeros((16, 32))
    for call in (lambda: pgg.moe_glu_grad(gy, w2[:, :, :23].contiguous(), gu, gl), lambda: pgg.moe_glu_grad(gy, w2.half(), gu, gl),
                 lambda: pgg.moe_glu_grad(gy, w2, gu[:, :31].contiguous(), gl), lambda: pgg.moe_glu_grad(gy, w2, gu, gl[:3]),
                 lambda: pgg.moe_glu_grad(gy, w2, gu.float(), gl), lambda: pgg.moe_glu_grad(gy, w2, gu, gl, act="tanh"),
                 lambda: pgg.moe_glu_grad(gy, w2, gu, gl, h=torch.empty(3, device=DEV))):
        with pytest.raises(pgg.PggError) as e:
            call()
        assert e.value.status == pgg.ERR_INVALID_ARG
