"""Plain 64-bit forms of the gate, the gated products and the adapters, with
the bounds that a 32-bit evaluation rounded once keeps, for the GPU tests.

All on the CPU in float64, row by row or expert by expert.  A bound follows
the error of each step: a sum of n products in fp32 is off by at most
GAMMA(n) = 2 (n + 8) 2^-24 times the sum of their magnitudes (2: the matrix
units may truncate where they align), a final rounding by U[dtype] times the
value, and below the normal range by TINY[dtype].
"""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def gamma(n):
    return 2.0 * (n + 8) * 2.0 ** -24


def rounded(value, err, dtype):
    """Bound on |stored - value| when the unrounded value is off by err."""
    return err + U[dtype] * (value.abs() + err) + TINY[dtype]


def assert_within(got, want, bound, what=""):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (got.shape, want.shape)
    ok = (got - want).abs() <= bound
    ok |= (got == want) | (got.isnan() & want.isnan())
    if not bool(ok.all()):
        i = tuple(int(v) for v in (~ok).nonzero()[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} outside, first at {i}: "
                             f"{got[i].item()} for {want[i].item()} (bound {bound[i].item()})")


# ---------------------------------------------------------------- gate

def gate(logits, topk, bias=None, renorm=False, scale=1.0):
    """(ids, probs, bound on probs, lse, bound on lse)."""
    l = logits.cpu().double()
    T, E = l.shape
    key = logits.cpu().float() if bias is None else logits.cpu().float() + bias.cpu()
    ids = torch.empty((T, topk), dtype=torch.int64)
    for t in range(T):
        k = [(math.inf, True) if math.isnan(v) else (v, False) for v in key[t].tolist()]
        ids[t] = torch.tensor(sorted(range(E), key=lambda e: (not k[e][1], -k[e][0], e))[:topk])
    over = l.gather(1, ids) if renorm else l
    top = over.amax(dim=1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    total = torch.exp(over - top).sum(dim=1, keepdim=True)
    e = torch.exp(l.gather(1, ids) - top)
    probs = torch.where(total == 0, e, e / total) * scale
    # exp of a rounded difference, n additions, a division, a product
    rel = ((l.gather(1, ids) - top).abs().nan_to_num(0.0, posinf=0.0, neginf=0.0) + over.shape[1] + 16) * 2.0 ** -23
    lse = torch.logsumexp(l, dim=1)
    return ids, probs, probs.abs() * rel + 2.0 ** -126, lse, (E + 16 + lse.abs().nan_to_num(0.0, 0.0, 0.0)) * 2.0 ** -23


def gate_grad(logits, ids, grad_probs, grad_lse=None, renorm=False, scale=1.0):
    """(grad_logits, bound before the final rounding)."""
    l = logits.cpu().double()
    ids = ids.cpu()
    T, E = l.shape
    p = torch.softmax(l, dim=1).nan_to_num(0.0)
    chosen = torch.zeros_like(l, dtype=torch.bool).scatter(1, ids, True)
    w = torch.softmax(l.masked_fill(~chosen, -math.inf), dim=1).nan_to_num(0.0) if renorm else p
    d = torch.zeros_like(l).scatter(1, ids, grad_probs.cpu().double() * scale)
    mean = (w * d).sum(dim=1, keepdim=True)
    g = w * (d - mean)
    size = w * (d.abs() + (w * d.abs()).sum(dim=1, keepdim=True))
    if grad_lse is not None:
        g = g + p * grad_lse.cpu().double()[:, None]
        size = size + p * grad_lse.cpu().double().abs()[:, None]
    lse = torch.logsumexp(l, dim=1, keepdim=True).nan_to_num(0.0, 0.0, 0.0)
    spread = (l.abs().nan_to_num(0.0, 0.0, 0.0).amax(dim=1, keepdim=True) + lse.abs()) * 2
    return g, size * (spread + E + 32) * 2.0 ** -22


# ---------------------------------------------------------------- gated products

def act(name, g):
    """(value, slope) of the activation."""
    if name == "silu":
        s, du = torch.sigmoid(g), torch.ones_like(g)
    else:
        c = math.sqrt(2.0 / math.pi)
        s = torch.sigmoid(2.0 * c * (g + 0.044715 * g ** 3))
        du = 2.0 * c * (1.0 + 3.0 * 0.044715 * g ** 2)
    return g * s, s + g * s * (1.0 - s) * du


SLOPE = 1.2        # above |act'| of both activations
CURVE = 1.2        # above |act''| of both
ACT_ULP = 32.0 * 2.0 ** -24   # relative error of the activations in fp32, per 1 + |argument|


def positions(eri, row_idx_type):
    eri = eri.cpu()
    if row_idx_type == 0:
        return eri
    p = torch.empty_like(eri)
    p[eri] = torch.arange(eri.numel())
    return p


def glu(x, weight, eri, group_list, topk, row_idx_type, name):
    """(h, bound, gate_up, bound), bounds after the rounding to x's dtype."""
    dtype, K = x.dtype, x.shape[1]
    src = x.cpu().double()[positions(eri, row_idx_type) // topk]
    M, C = src.shape[0], weight.shape[2]
    y, size = torch.zeros((M, C), dtype=torch.float64), torch.zeros((M, C), dtype=torch.float64)
    row = 0
    for g, n in enumerate(group_list.tolist()):
        if n:
            w = weight[g].cpu().double()
            y[row:row + n], size[row:row + n] = src[row:row + n] @ w, src[row:row + n].abs() @ w.abs()
        row += n
    err = gamma(K) * size
    F = C // 2
    gate, up, eg, eu = y[:, :F], y[:, F:], err[:, :F], err[:, F:]
    a, _ = act(name, gate)
    h = a * up
    ea = SLOPE * eg + ACT_ULP * (1 + gate.abs()) * a.abs()
    eh = ea * (up.abs() + eu) + a.abs() * eu + 2.0 ** -23 * h.abs()
    return h, rounded(h, eh, dtype), y, rounded(y, err, dtype)


def glu_grad(grad_y, weight, gate_up, group_list, name):
    """(grad_gate_up, bound, h, bound)."""
    dtype, D = grad_y.dtype, grad_y.shape[1]
    gy, F = grad_y.cpu().double(), weight.shape[1]
    M = gy.shape[0]
    dh, size = torch.zeros((M, F), dtype=torch.float64), torch.zeros((M, F), dtype=torch.float64)
    row = 0
    for g, n in enumerate(group_list.tolist()):
        if n:
            w = weight[g].cpu().double().t().contiguous()
            dh[row:row + n], size[row:row + n] = gy[row:row + n] @ w, gy[row:row + n].abs() @ w.abs()
        row += n
    ed = gamma(D) * size
    gate, up = gate_up[:, :F].cpu().double(), gate_up[:, F:].cpu().double()
    a, s = act(name, gate)
    ea = ACT_ULP * (1 + gate.abs()) * a.abs()
    es = ACT_ULP * (1 + gate.abs()) ** 3 * (s.abs() + 1.0)
    gg, gu = dh * up * s, dh * a
    egg = up.abs() * (ed * (s.abs() + es) + dh.abs() * es) + 2.0 ** -22 * gg.abs()
    egu = ed * (a.abs() + ea) + dh.abs() * ea + 2.0 ** -23 * gu.abs()
    h = a * up
    return (torch.cat([gg, gu], dim=1), rounded(torch.cat([gg, gu], dim=1), torch.cat([egg, egu], dim=1), dtype),
            h, rounded(h, ea * up.abs() + 2.0 ** -23 * h.abs(), dtype))


# ---------------------------------------------------------------- adapters

def lora(x, weight, a, b, ids, scales):
    """(y, bound after the rounding to x's dtype)."""
    dtype, (T, K), R = x.dtype, x.shape, a.shape[1]
    xd, w = x.cpu().double(), weight.cpu().double()
    y, err = xd @ w, gamma(K) * (xd.abs() @ w.abs())
    for t, p in enumerate(ids.tolist()):
        if p < 0:
            continue
        ad, bd, s = a[p].cpu().double(), b[p].cpu().double(), float(scales[p])
        z, ez = s * (ad @ xd[t]), abs(s) * gamma(K) * (ad.abs() @ xd[t].abs())
        y[t] += z @ bd
        # z as two bf16 parts is off by 2^-16 of itself; then a sum of R products
        err[t] += (ez + z.abs() * 2.0 ** -16) @ bd.abs() + gamma(R) * (z.abs() @ bd.abs())
    return y, rounded(y, err + 2.0 ** -23 * y.abs(), dtype)
