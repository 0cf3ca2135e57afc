"""Operands and results of more than 2^31 elements: sampled rows and columns at
their ends against the 64-bit forms (needs an MI355X's memory)."""
import math

import pytest
import torch

import ops_ref as ref
import permute_grouped_gemm_amd as pgg

pytestmark = pytest.mark.gpu
DEV = "cuda"
LIMIT = 1 << 31


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def _fill(std, *shape):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, std)


def _ends(n, k=3):
    """A few indices at both ends of range(n)."""
    return sorted({*range(min(k, n)), n // 2, *range(max(0, n - k), n)})


def _check_glu(x, w, gl, h, gu, rows, cols):
    """Rows (neighbours in one group are not needed) and columns of moe_glu over x in order."""
    F = w.shape[2] // 2
    group = torch.searchsorted(gl.cumsum(0), torch.tensor(rows, device=DEV), right=True).tolist()
    both = cols + [F + c for c in cols]
    for r, g in zip(rows, group):
        wg = w[g][:, both].cpu()[None]
        wh, eh, wy, ey = ref.glu(x[r:r + 1].cpu(), wg, torch.zeros(1, dtype=torch.int64), torch.tensor([1]), 1, 0, "silu")
        ref.assert_within(h[r:r + 1][:, cols], wh, eh, f"h row {r}")
        if gu is not None:
            ref.assert_within(gu[r:r + 1][:, both], wy, ey, f"gate_up row {r}")


# batch, experts, K, F and which operand is large: weights (few and many rows per
# expert, aligned and not), the products, x
GLU = [(40, 70, 4096, 4096, "w"), (40, 70, 4097, 4095, "w"), (400, 5, 16384, 14336, "w"), (400, 5, 16385, 14335, "w"),
       (70000, 2, 64, 16384, "gate_up"), (70000, 2, 67, 16385, "gate_up"), (140000, 1, 16384, 8, "x"),
       (140000, 1, 16385, 7, "x")]


@pytest.mark.parametrize("batch,G,K,F,large", GLU)
def test_glu(batch, G, K, F, large):
    x, w = _fill(1.0, batch, K), _fill(1.5 / math.sqrt(K), G, K, 2 * F)
    gl = torch.zeros(G, dtype=torch.int64, device=DEV)
    gl[0], gl[G - 1] = batch // 3, 0
    gl[G - 1] += batch - batch // 3
    if G == 1:
        gl[0] = batch
    assert {"w": w.numel(), "gate_up": batch * 2 * F, "x": x.numel()}[large] > LIMIT
    eri = torch.arange(batch, device=DEV)
    h, gu = pgg.moe_glu(x, w, eri, gl, 1, save_gate_up=True)
    torch.cuda.synchronize()
    _check_glu(x, w, gl, h, gu, _ends(batch), _ends(F))


@pytest.mark.parametrize("M,G,D,F,large", [(40, 70, 8192, 4096, "w"), (40, 70, 8193, 4095, "w"), (700, 3, 28672, 28672, "w"),
                                           (700, 3, 28673, 28671, "w"), (70000, 2, 64, 16384, "gate_up"),
                                           (70000, 2, 67, 16385, "gate_up"), (140000, 1, 16384, 8, "grad_y"),
                                           (140000, 1, 16385, 7, "grad_y")])
def test_glu_grad(M, G, D, F, large):
    gy, w, gu = _fill(1.0, M, D), _fill(1.0 / math.sqrt(D), G, F, D), _fill(1.5, M, 2 * F)
    gl = torch.zeros(G, dtype=torch.int64, device=DEV)
    gl[G - 1] = M - M // 3 if G > 1 else M
    if G > 1:
        gl[0] = M // 3
    assert {"w": w.numel(), "gate_up": gu.numel(), "grad_y": gy.numel()}[large] > LIMIT
    grad, h = pgg.moe_glu_grad(gy, w, gu, gl)
    torch.cuda.synchronize()
    cols, rows = _ends(F), _ends(M)
    both = cols + [F + c for c in cols]
    group = torch.searchsorted(gl.cumsum(0), torch.tensor(rows, device=DEV), right=True).tolist()
    for r, g in zip(rows, group):
        wg, eg, wh, eh = ref.glu_grad(gy[r:r + 1].cpu(), w[g][cols].cpu()[None], gu[r:r + 1][:, both].cpu(),
                                      torch.tensor([1]), "silu")
        ref.assert_within(grad[r:r + 1][:, both], wg, eg, f"grad row {r}")
        ref.assert_within(h[r:r + 1][:, cols], wh, eh, f"h row {r}")


@pytest.mark.parametrize("T,K,N,P,R,large", [
    (5, 65536, 32832, 3, 8, "w"), (300, 65536, 32832, 3, 8, "w"), (5, 65537, 32831, 3, 8, "w"), (140000, 16384, 16, 4, 8, "x"),
    (140000, 16385, 15, 4, 8, "x"), (70000, 64, 32768, 4, 8, "y"), (70000, 65, 32767, 4, 8, "y"),
    (5, 524416, 16, 64, 64, "a"), (300, 524416, 16, 64, 64, "a"), (2500, 524416, 16, 64, 64, "a"), (5, 16, 524416, 64, 64, "b"),
    (300, 16, 524416, 64, 64, "b")])
def test_lora(T, K, N, P, R, large):
    x, w = _fill(1.0, T, K), _fill(1.0 / math.sqrt(K), K, N)
    a, b = _fill(1.0 / math.sqrt(K), P, R, K), _fill(0.3, P, R, N)
    ids = torch.arange(T, device=DEV) * P // T
    ids[1::7] = -1
    scales = torch.linspace(0.5, 1.5, P, device=DEV)
    assert {"w": w.numel(), "x": x.numel(), "y": T * N, "a": a.numel(), "b": b.numel()}[large] > LIMIT
    y = pgg.lora_fwd(x, w, a, b, ids, scales)
    torch.cuda.synchronize()
    rows, cols = _ends(T), _ends(N)
    wc = w[:, cols].cpu()
    for r in rows:
        p = max(0, int(ids[r]))
        want, bound = ref.lora(x[r:r + 1].cpu(), wc, a[p:p + 1].cpu(), b[p:p + 1][:, :, cols].cpu(),
                               torch.tensor([0 if int(ids[r]) >= 0 else -1]), scales[p:p + 1].cpu())
        ref.assert_within(y[r:r + 1][:, cols], want, bound, f"row {r}")


def test_gate():
    T, E, k = 270000, 8192, 4
    l = _fill(1.5, T, E)
    assert l.numel() > LIMIT
    ids, probs, lse = pgg.moe_gate(l, k)
    gp, gl = torch.randn((T, k), device=DEV), torch.randn(T, device=DEV)
    grad = pgg.moe_gate_grad(l, lse, ids, gp, grad_lse=gl)
    torch.cuda.synchronize()
    rows = _ends(T)
    lc = l[rows].cpu()
    want, p, ep, s, es = ref.gate(lc, k)
    assert torch.equal(ids[rows].cpu(), want)
    ref.assert_within(probs[rows], p, ep, "probs")
    ref.assert_within(lse[rows], s, es, "lse")
    wg, eg = ref.gate_grad(lc, ids[rows], gp[rows], gl[rows])
    ref.assert_within(grad[rows], wg, ref.rounded(wg, eg, l.dtype), "grad")
