"""A mixture-of-experts block from the residual stream to the residual stream.

Training: router over experts in groups -> routing tables -> the experts' gated
product -> their second matrix -> weighted sum, norm, residual stream and the
norm in front of the next block, and the gradients of all of it.  Serving: the
same block with the experts' weights in 4 bits.

    python examples/moe_block.py            # needs an MI355X and the built library

Both are checked against the same block in 64-bit torch, the training step with
autograd.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import permute_grouped_gemm_amd as pgg  # noqa: E402

EPS = 1e-6


class MoeBlock:
    """Weights and, between forward and backward, what the gradients need."""

    def __init__(self, hidden, ffn, experts, topk, groups, topk_groups, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
        make = lambda *s: (rand(*s) * s[-2] ** -0.5).to(dtype)  # noqa: E731
        self.experts, self.topk = experts, topk
        self.gate = dict(score="sigmoid", groups=groups, topk_groups=topk_groups, scale=1.5)
        self.bias = rand(experts) * 0.1                  # balances the choice, not trained by gradients
        self.router = make(hidden, experts)
        self.w_in = make(experts, hidden, 2 * ffn)       # gate columns, then up columns
        self.w_out = make(experts, ffn, hidden)
        self.post = (1 + 0.1 * rand(hidden)).to(dtype)   # norm behind the experts
        self.next = (1 + 0.1 * rand(hidden)).to(dtype)   # norm in front of the next block

    def _route(self, x):
        logits = x @ self.router
        ids, probs = pgg.moe_gate_grouped(logits, self.topk, bias=self.bias, **self.gate)
        counts, gather, scatter, _ = pgg.moe_routing(ids, self.experts)
        return logits, ids, probs, counts, gather, scatter

    def _combine(self, y, scatter, probs, residual):
        return pgg.moe_combine(y, scatter, probs, residual, row_idx_type=1, post_weight=self.post,
                               next_weight=self.next, eps=EPS)

    def forward(self, x, residual):
        """(residual stream, its norm) [tokens, hidden] from the normed x and the residual stream."""
        logits, ids, probs, counts, gather, scatter = self._route(x)
        h, gate_up = pgg.moe_glu(x, self.w_in, gather, counts, self.topk, save_gate_up=True)
        rows = torch.arange(h.shape[0], device=x.device)         # h is in expert order already
        y = pgg.moe_fwd(h, self.w_out, rows, counts, 1).to(x.dtype)
        self.saved = (x, residual, logits, ids, probs, counts, gather, scatter, gate_up, rows, y)
        return self._combine(y, scatter, probs, residual)

    def backward(self, grad, grad_normed):
        """Gradients of x, residual, router, w_in, w_out, post and next."""
        x, residual, logits, ids, probs, counts, gather, scatter, gate_up, rows, y = self.saved
        grad_y, grad_probs, grad_residual, _, grad_post, grad_next = pgg.moe_combine_grad(
            grad, y, scatter, probs, residual, grad_normed=grad_normed, row_idx_type=1, post_weight=self.post,
            next_weight=self.next, eps=EPS)
        grad_gate_up, h = pgg.moe_glu_grad(grad_y, self.w_out, gate_up, counts)
        grad_w_out = pgg.moe_dw(h, grad_y, rows, counts, 1)
        grad_w_in = pgg.moe_dw(x, grad_gate_up, gather, counts, self.topk)
        grad_x = pgg.moe_dx(grad_gate_up, self.w_in, gather, counts, x.shape[0], self.topk)
        grad_logits = pgg.moe_gate_grouped_grad(logits, ids, grad_probs, score=self.gate["score"],
                                                scale=self.gate["scale"])
        grad_x += grad_logits.float() @ self.router.float().t()
        return grad_x, grad_residual, x.float().t() @ grad_logits.float(), grad_w_in, grad_w_out, grad_post, grad_next

    def quantize(self, group_size):
        """The experts' weights in 4 bits, laid out for serve()."""
        self.in4 = _quantize(self.w_in, group_size)
        self.out4 = _quantize(self.w_out, group_size)
        self.served = (pgg.w4_pack(self.in4[0], self.in4[1], group_size, zeros=self.in4[2], gated=True),
                       pgg.w4_pack(self.out4[0], self.out4[1], group_size, zeros=self.out4[2]))

    def serve(self, x, residual):
        """As forward, with the weights in 4 bits."""
        _, ids, probs, counts, gather, scatter = self._route(x)
        h = pgg.moe_glu_w4(x, self.served[0], gather, counts, self.topk)
        y = pgg.moe_fwd_w4(h, self.served[1], None, counts)      # h is in expert order already
        return (ids,) + self._combine(y, scatter, probs, residual)


def _quantize(w, group_size):
    """(codes, scales, zero points) of [G, K, N] weights, by the groups' ranges."""
    G, K, N = w.shape
    pad = -K % group_size
    grouped = torch.nn.functional.pad(w.float(), (0, 0, 0, pad)).reshape(G, -1, group_size, N)
    lo, hi = grouped.amin(dim=2).clamp_max(0), grouped.amax(dim=2).clamp_min(0)
    scales = ((hi - lo) / 15).clamp_min(1e-8).to(w.dtype)
    zeros = (-lo / scales.float()).round().clamp(0, 15)
    codes = (grouped / scales.float()[:, :, None] + zeros[:, :, None]).round().clamp(0, 15)
    return codes.reshape(G, -1, N)[:, :K].to(torch.uint8).contiguous(), scales, zeros.to(torch.uint8)


def _wide(quantized, group_size):
    """The weights that (codes, scales, zero points) stand for, float64."""
    codes, scales, zeros = (t.double() for t in quantized)
    wide = lambda t: t.repeat_interleave(group_size, dim=1)[:, :codes.shape[1]]  # noqa: E731
    return (codes - wide(zeros)) * wide(scales)


def exact(block, x, residual, ids, w_in, w_out, router, post, nxt):
    """(residual stream, its norm) in the inputs' float64 (ids: the experts chosen)."""
    s = torch.sigmoid(x @ router).gather(1, ids)
    probs = block.gate["scale"] * s / s.sum(dim=1, keepdim=True)
    c = torch.zeros_like(x)
    for e in range(block.experts):
        token, slot = (ids == e).nonzero(as_tuple=True)
        gate, up = (x[token] @ w_in[e]).chunk(2, dim=1)
        y = (torch.nn.functional.silu(gate) * up) @ w_out[e]
        c = c.index_add(0, token, y * probs[token, slot][:, None])
    norm = lambda v: v / (v.pow(2).mean(dim=1, keepdim=True) + EPS).sqrt()  # noqa: E731
    out = residual + norm(c) * post
    return out, norm(out) * nxt


def main(tokens=512, hidden=256, ffn=192, experts=16, topk=4, groups=4, topk_groups=2, group_size=64):
    """Runs both steps; returns {name: normwise relative error}."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda: torch.randn((tokens, hidden), generator=gen, device="cuda")  # noqa: E731
    block = MoeBlock(hidden, ffn, experts, topk, groups, topk_groups)
    x, residual, grad, grad_normed = (rand().bfloat16() for _ in range(4))
    results = block.forward(x, residual)
    grads = block.backward(grad, grad_normed)
    leaves = [t.double().requires_grad_() for t in (x, residual, block.router, block.w_in, block.w_out, block.post,
                                                    block.next)]
    wx, wr, router, w_in, w_out, post, nxt = leaves
    want = exact(block, wx, wr, block.saved[3], w_in, w_out, router, post, nxt)
    want_grads = torch.autograd.grad(want, leaves, (grad.double(), grad_normed.double()))
    errors = {}
    names = ("stream", "normed", "grad x", "grad residual", "grad router", "grad w_in", "grad w_out", "grad post",
             "grad next")
    for name, g, w in zip(names, results + grads, want + want_grads):
        w = w.detach()
        errors[name] = float(g.double().sub(w).norm() / w.norm())

    block.quantize(group_size)
    ids, stream, normed = block.serve(x, residual)
    want = exact(block, x.double(), residual.double(), ids, _wide(block.in4, group_size),
                 _wide(block.out4, group_size), block.router.double(), block.post.double(), block.next.double())
    for name, g, w in zip(("served stream", "served normed"), (stream, normed), want):
        errors[name] = float(g.double().sub(w).norm() / w.norm())
    return errors


if __name__ == "__main__":
    for name, error in main().items():
        print(f"{name:14s} normwise relative error {error:.2e}")
