"""One training step and one serving step of a mixture-of-experts layer.

Training: router -> gate -> routing tables -> the experts' gated product ->
their second matrix -> weighted sum, and the gradients of all of it.  Serving:
a projection that all requests share, with each request's low-rank adapter
beside it, in front of the layer.

    python examples/moe_layer.py            # needs an MI355X and the built library

Every product but the router's own small matrix runs in the library.  The step
is checked against the same layer in 64-bit torch with autograd.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import permute_grouped_gemm_amd as pgg  # noqa: E402


class MoeLayer:
    """Weights and, between forward and backward, what the gradients need."""

    def __init__(self, hidden, ffn, experts, topk, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        make = lambda *s: (torch.randn(s, generator=gen, device=device) * s[-2] ** -0.5).to(dtype)  # noqa: E731
        self.topk, self.experts = topk, experts
        self.router = make(hidden, experts)
        self.w_in = make(experts, hidden, 2 * ffn)      # gate columns, then up columns
        self.w_out = make(experts, ffn, hidden)

    def forward(self, x):
        """float32 [tokens, hidden] for x [tokens, hidden]."""
        tokens = x.shape[0]
        logits = x @ self.router
        ids, probs, lse = pgg.moe_gate(logits, self.topk, renorm=True)
        counts, eri, _, _ = pgg.moe_routing(ids, self.experts, scatter=False)
        h, gate_up = pgg.moe_glu(x, self.w_in, eri, counts, self.topk, save_gate_up=True)
        rows = torch.arange(tokens * self.topk, device=x.device)     # h is in expert order already
        y = pgg.moe_fwd(h, self.w_out, rows, counts, 1)
        self.saved = (x, logits, ids, probs, lse, counts, eri, gate_up, rows, y)
        return pgg.moe_unpermute(y, eri, tokens, self.topk, 0, probs)

    def backward(self, grad):
        """Gradients of x, router, w_in and w_out for grad [tokens, hidden] float32."""
        x, logits, ids, probs, lse, counts, eri, gate_up, rows, y = self.saved
        tokens = x.shape[0]
        grad_y, grad_probs = pgg.moe_unpermute_grad(grad, eri, tokens, self.topk, 0, y, probs)
        grad_y = grad_y.to(x.dtype)
        grad_gate_up, h = pgg.moe_glu_grad(grad_y, self.w_out, gate_up, counts)
        grad_w_out = pgg.moe_dw(h, grad_y, rows, counts, 1)
        grad_w_in = pgg.moe_dw(x, grad_gate_up, eri, counts, self.topk)
        grad_x = pgg.moe_dx(grad_gate_up, self.w_in, eri, counts, tokens, self.topk)
        grad_logits = pgg.moe_gate_grad(logits, lse, ids, grad_probs, renorm=True)
        grad_x += grad_logits.float() @ self.router.float().t()
        return grad_x, x.float().t() @ grad_logits.float(), grad_w_in, grad_w_out


def exact(layer, x, ids, grad):
    """Output and gradients of the layer in float64 (ids: the experts chosen)."""
    x, router, w_in, w_out = (t.detach().double().requires_grad_() for t in (x, layer.router, layer.w_in, layer.w_out))
    logits = x @ router
    probs = torch.softmax(logits.gather(1, ids), dim=1)
    out = torch.zeros_like(x)
    for e in range(layer.experts):
        token, slot = (ids == e).nonzero(as_tuple=True)
        gate, up = (x[token] @ w_in[e]).chunk(2, dim=1)
        y = (torch.nn.functional.silu(gate) * up) @ w_out[e]
        out = out.index_add(0, token, y * probs[token, slot][:, None])
    return out, torch.autograd.grad(out, (x, router, w_in, w_out), grad.double())


def main(tokens=512, hidden=256, ffn=192, experts=16, topk=4, adapters=5, rank=8):
    """Runs both steps; returns {name: normwise relative error}."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    layer = MoeLayer(hidden, ffn, experts, topk)

    # serving: the requests' projection, then the layer
    a, b = (rand(adapters, rank, hidden) * hidden ** -0.5).bfloat16(), (rand(adapters, rank, hidden) * 0.2).bfloat16()
    scales = torch.full((adapters,), 2.0, device=dev)
    owner = torch.arange(tokens, device=dev) // 37 % (adapters + 1) - 1      # -1: a request without an adapter
    proj, tok = (rand(hidden, hidden) * hidden ** -0.5).bfloat16(), rand(tokens, hidden).bfloat16()
    x = pgg.lora_fwd(tok, proj, a, b, owner, scales)
    want = tok.double() @ proj.double()
    for p in range(adapters):
        at = owner == p
        want[at] += 2.0 * (tok[at].double() @ a[p].double().t().contiguous()) @ b[p].double()
    errors = {"adapters": x.double().sub(want).norm() / want.norm()}

    # training
    grad = rand(tokens, hidden)
    out = layer.forward(x)
    grads = layer.backward(grad)
    want, want_grads = exact(layer, x, layer.saved[2], grad)
    want = want.detach()
    errors["output"] = out.double().sub(want).norm() / want.norm()
    for name, g, w in zip(("grad x", "grad router", "grad w_in", "grad w_out"), grads, want_grads):
        errors[name] = g.double().sub(w).norm() / w.norm()
    return {k: float(v) for k, v in errors.items()}


if __name__ == "__main__":
    for name, error in main().items():
        print(f"{name:12s} normwise relative error {error:.2e}")
