"""Plain 64-bit forms of the grouped gate, the 4-bit products and the
combination with the residual stream, with the bounds that a 32-bit evaluation
rounded once keeps, for the GPU tests.

A sum of n fp32 terms added in a tree or in runs is off by at most GAMMA(depth)
times the sum of the magnitudes, depth being the longest chain of additions
(ops_ref.gamma doubles it, and adds 8 for the products and conversions).
"""
import math

import torch

from ops_ref import ACT_ULP, SLOPE, act, gamma, positions, rounded


# ---------------------------------------------------------------- gate

def gate_grouped(logits, topk, score="sigmoid", groups=1, topk_groups=None, bias=None, renorm=True, scale=1.0):
    """(ids, probs, bound on probs)."""
    topk_groups = groups if topk_groups is None else topk_groups
    l = logits.cpu().double()
    T, E = l.shape
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, dim=1)
    key = s if bias is None else s + bias.cpu().double()
    each = E // groups
    ids = torch.empty((T, topk), dtype=torch.int64)
    for t in range(T):
        # (-inf for an excluded expert; NaN above everything)
        k = [-math.inf if l[t, e] == -math.inf else math.inf if math.isnan(v) else v
             for e, v in enumerate(key[t].tolist())]
        total = []
        for g in range(groups):
            best = sorted(k[g * each:(g + 1) * each], reverse=True)[:2]
            total.append(best[0] + (best[1] if len(best) > 1 and best[1] != -math.inf else 0.0))
        kept = set(sorted(range(groups), key=lambda g: (-total[g], g))[:topk_groups])
        ids[t] = torch.tensor(sorted((e for e in range(E) if e // each in kept), key=lambda e: (-k[e], e))[:topk])
    w, rel = _weights(l, ids, score, renorm)
    probs = w * scale
    return ids, probs, probs.abs() * rel + 2.0 ** -126


def _weights(l, ids, score, renorm):
    """Weights before the scale and a bound on their relative error: exp of a
    rounded difference, n additions, a division, products."""
    picked = l.gather(1, ids)
    if score == "sigmoid" and not renorm:
        return torch.sigmoid(picked), 16 * 2.0 ** -23
    logs = torch.nn.functional.logsigmoid(picked) if score == "sigmoid" else picked
    over = logs if renorm else l
    top = over.amax(dim=1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    total = torch.exp(over - top).sum(dim=1, keepdim=True)
    e = torch.exp(logs - top)
    spread = (logs - top).abs().nan_to_num(0.0, posinf=0.0, neginf=0.0) + over.shape[1] + 24
    return torch.where(total == 0, e, e / total), spread * 2.0 ** -23


def gate_grouped_grad(logits, ids, grad_probs, score="sigmoid", renorm=True, scale=1.0):
    """(grad_logits, bound before the final rounding)."""
    l, ids = logits.cpu().double(), ids.cpu()
    w, rel = _weights(l, ids, score, renorm)
    rel = torch.as_tensor(rel, dtype=torch.float64).expand(w.shape).amax(dim=1, keepdim=True)
    d = grad_probs.cpu().double() * scale
    mean, size = (d * w).sum(dim=1, keepdim=True), (d * w).abs().sum(dim=1, keepdim=True)
    zero = torch.zeros_like(l)
    if score == "softmax" and not renorm:
        p = torch.softmax(l, dim=1).nan_to_num(0.0)
        at = zero.scatter(1, ids, d)
        spread = l.abs().nan_to_num(0.0, 0.0, 0.0).amax(dim=1, keepdim=True) * 2 * 2.0 ** -23
        return p * (at - mean), p * (at.abs() + size) * (4 * rel + 2 * spread)
    rest = torch.sigmoid(-l.gather(1, ids)) if score == "sigmoid" else 1.0
    if renorm:
        g, b = w * rest * (d - mean), w * rest * (d.abs() + size)
    else:
        g = w * rest * d
        b = g.abs()
    return zero.scatter(1, ids, g), zero.scatter(1, ids, b * (4 * rel + 32 * 2.0 ** -23))


# ---------------------------------------------------------------- 4-bit weights

def w4_weights(codes, scales, zeros, group_size):
    """W and the magnitude that its parts have, float64 [G, K, N]."""
    K = codes.shape[1]
    wide = lambda t: t.cpu().double().repeat_interleave(group_size, dim=1)[:, :K]  # noqa: E731
    z = 8.0 if zeros is None else wide(zeros)
    q, s = codes.cpu().double(), wide(scales)
    return (q - z) * s, (q + z) * s.abs()


def w4_product(x, codes, scales, zeros, group_size, group_list, topk=1, eri=None, row_idx_type=0):
    """(y, error before the rounding): codes and zero points are exact, so all that
    is off are the fp32 sums of code x and zero x over the reduction."""
    w, size = w4_weights(codes, scales, zeros, group_size)
    src = x.cpu().double()
    if eri is not None:
        src = src[positions(eri, row_idx_type) // topk]
    y = torch.zeros((src.shape[0], w.shape[2]), dtype=torch.float64)
    err = torch.zeros_like(y)
    row = 0
    for g, n in enumerate(group_list.tolist()):
        if n:
            y[row:row + n] = src[row:row + n] @ w[g]
            err[row:row + n] = src[row:row + n].abs() @ size[g]
        row += n
    return y, gamma(x.shape[1]) * err


def w4_fwd(x, *weights, **kw):
    y, err = w4_product(x, *weights, **kw)
    return y, rounded(y, err, x.dtype)


def w4_glu(x, *weights, name="silu", **kw):
    y, err = w4_product(x, *weights, **kw)
    (gate, up), (eg, eu) = y.chunk(2, dim=1), err.chunk(2, dim=1)
    a, _ = act(name, gate)
    h = a * up
    ea = SLOPE * eg + ACT_ULP * (1 + gate.abs()) * a.abs()
    return h, rounded(h, ea * (up.abs() + eu) + a.abs() * eu + 2.0 ** -23 * h.abs(), x.dtype)


# ---------------------------------------------------------------- combination

ROW = gamma(64)   # sums over a row: 32 elements to a thread, 6 steps in a wave, 16 waves


class Near:
    """A float64 tensor with a bound on the error of its fp32 evaluation."""

    def __init__(self, v, e=None):
        self.v, self.e = v, torch.zeros_like(v) if e is None else e

    def __mul__(self, o):
        o = o if isinstance(o, Near) else Near(torch.as_tensor(o, dtype=torch.float64))
        v = self.v * o.v
        return Near(v, self.v.abs() * o.e + self.e * (o.v.abs() + o.e) + 2.0 ** -23 * v.abs())

    def __add__(self, o):
        v = self.v + o.v
        return Near(v, self.e + o.e + 2.0 ** -23 * (self.v.abs() + o.v.abs()))

    def __neg__(self):
        return Near(-self.v, self.e)

    def sum(self, dim, depth, keepdim=True):
        return Near(self.v.sum(dim=dim, keepdim=keepdim),
                    self.e.sum(dim=dim, keepdim=keepdim) + depth * self.v.abs().sum(dim=dim, keepdim=keepdim))

    def rsqrt(self):
        v = self.v.rsqrt()
        return Near(v, v * (0.5 * (self.e / self.v) * (1 + self.e / self.v) + 8 * 2.0 ** -23))


def _norm(x, eps):
    """1 / sqrt(mean(x^2) + eps), one to a row."""
    ms = (x * x).sum(1, ROW) * (1.0 / x.v.shape[1])
    return (ms + Near(torch.full_like(ms.v, float(torch.tensor(eps, dtype=torch.float32))))).rsqrt()


def slots(eri, batch, topk, row_idx_type):
    """Expanded row of every slot [batch, topk]."""
    eri = eri.cpu()
    if row_idx_type == 0:
        back = torch.empty_like(eri)
        back[eri] = torch.arange(eri.numel())
        eri = back
    return eri.reshape(batch, topk)


def combine(permuted, eri, probs, residual, row_idx_type=0, post=None, gate=None, alpha=1.0, nxt=None, eps=1e-6,
            grad_out=None, grad_normed=None):
    """{name: Near} of the results or, with grad_out, of the gradients (before rounding)."""
    batch, topk = probs.shape
    wide = lambda t: Near(t.cpu().double())  # noqa: E731
    at = slots(eri, batch, topk, row_idx_type)
    y, p = Near(permuted.cpu().double()[at]), Near(probs.cpu().double()[:, :, None])
    c = (y * p).sum(1, gamma(topk), keepdim=False)
    alpha = float(torch.tensor(alpha, dtype=torch.float32))
    g = Near(torch.ones((batch, 1), dtype=torch.float64)) if gate is None else Near(gate.cpu().double()[:, None])
    r = _norm(c, eps) if post is not None else Near(torch.ones((batch, 1), dtype=torch.float64))
    w = wide(post) if post is not None else Near(torch.ones(c.v.shape[1], dtype=torch.float64))
    out = wide(residual) * alpha + g * (c * r * w)
    q = _norm(out, eps) if nxt is not None else None
    if grad_out is None:
        res = {"out": out}
        if nxt is not None:
            res["normed"] = out * (q * wide(nxt))
        return res
    H = c.v.shape[1]
    go, res = wide(grad_out), {}
    if nxt is not None:
        gn = wide(grad_normed)
        u = gn * wide(nxt)
        res["next"] = (gn * (out * q)).sum(0, gamma(64), keepdim=False)
        go = go + q * u + -(out * (q * q * q * ((u * out).sum(1, ROW) * (1.0 / H))))
    res["residual"] = go * alpha
    s = (go * w * c).sum(1, ROW)
    if gate is not None:
        res["gate"] = Near((r * s).v[:, 0], (r * s).e[:, 0])
    if post is not None:
        res["post"] = (g * go * (c * r)).sum(0, gamma(64), keepdim=False)
        gc = g * r * (go * w) + -(c * (g * (r * r * r) * (s * (1.0 / H))))
    else:
        gc = g * go
    wide_gc = Near(gc.v[:, None, :], gc.e[:, None, :])
    res["probs"] = (wide_gc * y).sum(2, ROW, keepdim=False)
    slot = p * wide_gc
    flat = at.reshape(-1)
    v, e = torch.empty((batch * topk, H), dtype=torch.float64), torch.empty((batch * topk, H), dtype=torch.float64)
    v[flat], e[flat] = slot.v.reshape(-1, H), slot.e.reshape(-1, H)
    res["permuted"] = Near(v, e)
    return res
