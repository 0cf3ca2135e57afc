"""Cases for timing and checking the router's gate, the experts' gated
products and the low-rank adapters, each beside its plain form.

``listed()`` and ``draw(rng)`` give cases, ``prepare(case, seed)`` the inputs
on the GPU, ``run(state)`` one pass: the framework's operators where ``own``
is true, otherwise the same formulas in elementary torch operations on 32-bit
values, rounded once at the end.  ``exact(case, seed)`` evaluates the
definitions in 64 bits, and ``work(case)`` counts the bytes and operations
that a pass cannot do without.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
KINDS = ("gate", "gate_grad", "glu", "glu_grad", "lora")


def listed():
    return [
        # the router of one decode step: 16 tokens, weights summing to one; launch latency is all of it
        dict(name="gate decode", op="gate", dtype="bf16", tokens=16, experts=16, topk=8, renorm=True,
             scale=1.0, bias=False, masked=False),
        # the router of a large training batch, with a balancing bias, banned experts (-inf) and padding rows
        dict(name="gate train", op="gate", dtype="f32", tokens=13824, experts=60, topk=8, renorm=False,
             scale=2.5, bias=True, masked=True),
        # its backward on a middling batch: weights that sum to one, no term for the log-sum-exp
        dict(name="gate grad mid", op="gate_grad", dtype="f16", tokens=2048, experts=16, topk=8, renorm=True,
             scale=1.0, bias=False, masked=False, lse_grad=False),
        # its backward on a large batch with the log-sum-exp penalty's gradient
        dict(name="gate grad train", op="gate_grad", dtype="f32", tokens=13824, experts=60, topk=8,
             renorm=False, scale=2.5, bias=False, masked=True, lse_grad=True),
        # a tiny fp32 layer: every launch is short
        dict(name="glu tiny", op="glu", dtype="f32", batch=64, topk=2, groups=4, empty=1, k=256, f=64,
             skew=0.0, row_idx_type=0, act="silu", save=True),
        # one decode step: the weights of the used experts are read once for 128 rows
        dict(name="glu decode", op="glu", dtype="bf16", batch=16, topk=8, groups=16, empty=4, k=7168, f=2048,
             skew=0.0, row_idx_type=0, act="silu", save=False),
        # a training or prefill batch over experts of very different popularity
        dict(name="glu mid", op="glu", dtype="bf16", batch=2048, topk=8, groups=16, empty=0, k=7168, f=2048,
             skew=1.1, row_idx_type=1, act="silu", save=True),
        # the backward at odd sizes: no row starts on a 16-byte boundary, experts hold about ten rows
        dict(name="glu grad odd", op="glu_grad", dtype="bf16", batch=333, topk=2, groups=64, empty=5, d=2039,
             f=1403, skew=1.1, act="gelu_tanh"),
        # the backward of a large fp16 training batch
        dict(name="glu grad large", op="glu_grad", dtype="f16", batch=13824, topk=8, groups=60, empty=0, d=7168,
             f=2048, skew=0.0, act="silu"),
        # one token of one request on a small projection
        dict(name="lora one token", op="lora", dtype="bf16", tokens=1, k=2048, n=1408, adapters=16, rank=8,
             none=0.0, run=1),
        # a decode step of 16 requests, nearly each with an adapter of its own
        dict(name="lora decode", op="lora", dtype="bf16", tokens=16, k=7168, n=4096, adapters=60, rank=16,
             none=0.1, run=1),
        # prefill of many requests of a few hundred tokens each
        dict(name="lora prefill", op="lora", dtype="f16", tokens=13824, k=7168, n=2048, adapters=60, rank=16,
             none=0.1, run=300),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row length: half of them a multiple of 64 or 8, the others as they come."""
    v = _spread(rng, lo, hi)
    m = rng.choice((64, 8, 1, 1))
    return max(lo, v // m * m)


def draw(rng):
    op = rng.choice(KINDS)
    dtype = rng.choice(("bf16", "f16", "bf16", "f16", "f32"))
    if op in ("gate", "gate_grad"):
        experts = _spread(rng, 4, 512)
        c = dict(op=op, dtype=dtype, tokens=_spread(rng, 1, 13824), experts=experts,
                 topk=rng.randint(1, min(8, experts)), renorm=rng.random() < 0.5, scale=rng.choice((1.0, 2.5)),
                 bias=op == "gate" and rng.random() < 0.5, masked=rng.random() < 0.5)
        if op == "gate_grad":
            c["lse_grad"] = rng.random() < 0.5
        return c
    most = 2e11 if dtype == "f32" else 1.5e12
    while True:
        if op == "lora":
            c = dict(op=op, dtype=dtype, tokens=_spread(rng, 1, 13824), k=_width(rng, 64, 7168),
                     n=_width(rng, 64, 7168), adapters=_spread(rng, 1, 64), rank=rng.choice((1, 4, 8, 12, 16, 32, 64)),
                     none=rng.choice((0.0, 0.1, 0.5)), run=_spread(rng, 1, 2048))
        else:
            groups = _spread(rng, 1, 64)
            empty = rng.randint(0, groups // 4)
            c = dict(op=op, dtype=dtype, batch=_spread(rng, 1, 4096), topk=rng.randint(1, min(8, groups - empty)),
                     groups=groups, empty=empty, f=_width(rng, 32, 4096), skew=rng.choice((0.0, 1.1)),
                     act=rng.choice(("silu", "silu", "gelu_tanh")))
            if op == "glu":
                c.update(k=_width(rng, 64, 7168), row_idx_type=rng.randint(0, 1), save=rng.random() < 0.5)
            else:
                c["d"] = _width(rng, 64, 7168)
        w = work(c)
        if w["flops"] <= most and w["bytes"] <= 3e9:
            return c


def work(case):
    s = SIZES[case["dtype"]]
    op = case["op"]
    if op in ("gate", "gate_grad"):
        t, e, k = case["tokens"], case["experts"], case["topk"]
        if op == "gate":   # logits read; ids, weights and the log-sum-exp written
            return {"bytes": t * e * s + t * k * 12 + t * 4 + (4 * e if case["bias"] else 0), "flops": 4.0 * t * e}
        return {"bytes": 2 * t * e * s + t * k * 12 + t * (8 if case["lse_grad"] else 4), "flops": 4.0 * t * e}
    if op == "lora":
        t, k, n, r = case["tokens"], case["k"], case["n"], case["rank"]
        used = min(case["adapters"], t)
        return {"bytes": s * (t * k + k * n + t * n + used * r * (k + n)) + 8 * t + 4 * case["adapters"],
                "flops": 2.0 * t * k * n + 2.0 * t * r * (k + n)}
    m, f = case["batch"] * case["topk"], case["f"]
    used = min(case["groups"] - case["empty"], m)
    if op == "glu":
        k = case["k"]
        return {"bytes": s * (case["batch"] * k + used * k * 2 * f + m * f * (3 if case["save"] else 1)) + 8 * m
                + 8 * case["groups"], "flops": 4.0 * m * k * f}
    d = case["d"]
    return {"bytes": s * (m * d + used * f * d + 5 * m * f) + 8 * case["groups"], "flops": 2.0 * m * d * f}


# ---------------------------------------------------------------- inputs

def _routing(case, gen, dev):
    """Distinct experts for every token, drawn by popularity: the routing index
    of the case's encoding, the rows per expert, and the largest of them."""
    batch, topk, groups = case["batch"], case["topk"], case["groups"]
    usable = groups - case["empty"]
    order = torch.randperm(groups, generator=gen, device=dev)
    weight = torch.full((groups,), float("-inf"), device=dev)
    weight[order[:usable]] = -case["skew"] * torch.arange(1, usable + 1, device=dev).log()
    noise = -torch.empty((batch, groups), device=dev).exponential_(generator=gen).clamp_min(1e-30).log()
    ids = (weight + noise).topk(topk, dim=1).indices.reshape(-1)
    eri = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=groups)
    if case.get("row_idx_type", 0) == 1:
        back = torch.empty_like(eri)
        back[eri] = torch.arange(eri.numel(), device=dev)
        eri = back
    return eri, counts, int(counts.max())


def _values(gen, dev, dtype, std, *shape):
    out = torch.empty(shape, dtype=dtype, device=dev)
    if out.numel() <= 1 << 28:
        return out.copy_(torch.randn(shape, generator=gen, device=dev) * std)
    for part in out:   # large weights: a slice at a time
        part.copy_(torch.randn(part.shape, generator=gen, device=dev) * std)
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(1000003 * int(seed) + 17)
    dtype = DTYPES[case["dtype"]]
    op = case["op"]
    s = {"case": case}
    if op in ("gate", "gate_grad"):
        t, e, k = case["tokens"], case["experts"], case["topk"]
        logits = torch.randn((t, e), generator=gen, device=dev) * 1.5
        if case["masked"]:
            banned = torch.rand((t, e), generator=gen, device=dev) < 0.1
            banned[torch.rand((t,), generator=gen, device=dev) < 0.01] = True   # padding rows: nothing left
            logits = logits.masked_fill(banned, float("-inf"))
        s["logits"] = logits.to(dtype)
        s["bias"] = torch.randn((e,), generator=gen, device=dev) * 0.1 if case["bias"] else None
        if op == "gate_grad":
            l = s["logits"].float()
            s["ids"] = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k].contiguous()
            s["lse"] = torch.logsumexp(l, dim=1)
            s["grad_probs"] = torch.randn((t, k), generator=gen, device=dev)
            s["grad_lse"] = torch.randn((t,), generator=gen, device=dev) * 0.1 if case["lse_grad"] else None
        return s
    if op == "lora":
        t, k, n, p, r = case["tokens"], case["k"], case["n"], case["adapters"], case["rank"]
        s["x"] = _values(gen, dev, dtype, 1.0, t, k)
        s["weight"] = _values(gen, dev, dtype, 0.02, k, n)
        s["a"] = _values(gen, dev, dtype, 0.02, p, r, k)
        s["b"] = _values(gen, dev, dtype, 0.05, p, r, n)
        s["scales"] = 0.5 + torch.rand((p,), generator=gen, device=dev) * 1.5
        # requests one after another, each of about `run` tokens and of one adapter or none
        request = torch.arange(t, device=dev) // case["run"]
        pick = torch.randint(0, p, (t,), generator=gen, device=dev)
        pick[torch.rand((t,), generator=gen, device=dev) < case["none"]] = -1
        s["ids"] = pick[request]
        return s
    s["eri"], s["group_list"], s["cap"] = _routing(case, gen, dev)
    m, f, g = case["batch"] * case["topk"], case["f"], case["groups"]
    if op == "glu":
        s["x"] = _values(gen, dev, dtype, 1.0, case["batch"], case["k"])
        s["weight"] = _values(gen, dev, dtype, 0.02, g, case["k"], 2 * f)
    else:
        s["grad_y"] = _values(gen, dev, dtype, 1.0, m, case["d"])
        s["weight"] = _values(gen, dev, dtype, 0.02, g, f, case["d"])
        s["gate_up"] = _values(gen, dev, dtype, 1.5, m, 2 * f)
    return s


# ---------------------------------------------------------------- the framework's operators

def _run_own(s):
    import permute_grouped_gemm_amd as pgg

    c = s["case"]
    op = c["op"]
    if op == "gate":
        return pgg.moe_gate(s["logits"], c["topk"], bias=s["bias"], renorm=c["renorm"], scale=c["scale"])
    if op == "gate_grad":
        return pgg.moe_gate_grad(s["logits"], s["lse"], s["ids"], s["grad_probs"], grad_lse=s["grad_lse"],
                                 renorm=c["renorm"], scale=c["scale"])
    if op == "glu":
        args = (s["x"], s["weight"], s["eri"], s["group_list"], c["topk"], c["row_idx_type"])
        if "workspace" not in s:
            s["workspace"] = torch.empty(pgg.glu_workspace_size(*args), dtype=torch.uint8, device="cuda")
        return pgg.moe_glu(*args, act=c["act"], save_gate_up=c["save"], workspace=s["workspace"])
    if op == "glu_grad":
        args = (s["grad_y"], s["weight"], s["gate_up"], s["group_list"])
        if "workspace" not in s:
            s["workspace"] = torch.empty(pgg.glu_grad_workspace_size(*args), dtype=torch.uint8, device="cuda")
        return pgg.moe_glu_grad(*args, act=c["act"], workspace=s["workspace"])
    args = (s["x"], s["weight"], s["a"], s["b"], s["ids"], s["scales"])
    if "workspace" not in s:
        s["workspace"] = torch.empty(pgg.lora_workspace_size(*args), dtype=torch.uint8, device="cuda")
    return pgg.lora_fwd(*args, workspace=s["workspace"])


# ---------------------------------------------------------------- the plain forms

def _softmax(l):
    """Softmax and log-sum-exp of the rows; a row of -inf gives zeros and -inf."""
    top = l.amax(dim=1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    e = torch.exp(l - top)
    total = e.sum(dim=1, keepdim=True)
    return torch.where(total > 0, e / total, e), (top + total.log()).squeeze(1)


def _gate(s):
    c = s["case"]
    l = s["logits"].float()
    key = l if s["bias"] is None else l + s["bias"]
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["topk"]]
    p, lse = _softmax(l)
    w = _softmax(l.gather(1, ids))[0] if c["renorm"] else p.gather(1, ids)
    return ids, w * c["scale"], lse


def _gate_grad(s):
    c = s["case"]
    l, dw = s["logits"].float(), s["grad_probs"] * c["scale"]
    p = torch.exp(l - s["lse"].clamp_min(torch.finfo(torch.float32).min)[:, None])
    if c["renorm"]:
        w = _softmax(l.gather(1, s["ids"]))[0]
        grad = torch.zeros_like(l).scatter(1, s["ids"], w * (dw - (dw * w).sum(dim=1, keepdim=True)))
    else:
        d = torch.zeros_like(l).scatter(1, s["ids"], dw)
        grad = p * (d - (d * p).sum(dim=1, keepdim=True))
    if s["grad_lse"] is not None:
        grad = grad + s["grad_lse"][:, None] * p
    return grad.to(s["logits"].dtype)


def _by_expert(s, rows, weight):
    """rows[i] times the weight of the row's expert: rows padded to the fullest
    expert, one batched product."""
    counts = s["group_list"]
    ends = counts.cumsum(0)
    place = torch.arange(s["cap"], device=rows.device)
    at = (ends - counts)[:, None] + torch.minimum(place, (counts - 1).clamp_min(0)[:, None])
    y = torch.bmm(rows[at.clamp_max(rows.shape[0] - 1)].float(), weight.float())
    i = torch.arange(rows.shape[0], device=rows.device)
    g = torch.searchsorted(ends, i, right=True)
    return y.reshape(-1, y.shape[2])[g * s["cap"] + i - (ends - counts)[g]]


def _act(case, g):
    """The activation and its derivative."""
    if case["act"] == "silu":
        q = 1 / (1 + torch.exp(-g))
        return g * q, q * (1 + g * (1 - q))
    c0, c1 = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(c0 * (g + c1 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c0 * (1 + 3 * c1 * g * g)


def _position(s):
    """Original position of every expanded row."""
    if s["case"]["row_idx_type"] == 0:
        return s["eri"]
    p = torch.empty_like(s["eri"])
    p[s["eri"]] = torch.arange(p.numel(), device=p.device)
    return p


def _glu(s):
    c = s["case"]
    y = _by_expert(s, s["x"][_position(s) // c["topk"]], s["weight"])
    gate, up = y[:, :c["f"]], y[:, c["f"]:]
    h = (_act(c, gate)[0] * up).to(s["x"].dtype)
    return (h, y.to(s["x"].dtype)) if c["save"] else h


def _glu_grad(s):
    c = s["case"]
    dh = _by_expert(s, s["grad_y"], s["weight"].transpose(1, 2))
    gate, up = s["gate_up"][:, :c["f"]].float(), s["gate_up"][:, c["f"]:].float()
    a, da = _act(c, gate)
    return torch.cat([dh * up * da, dh * a], dim=1).to(s["grad_y"].dtype), (a * up).to(s["grad_y"].dtype)


def _lora(s):
    x = s["x"].float()
    p, r = s["a"].shape[:2]
    mine = (s["ids"][:, None] == torch.arange(p, device=x.device)) * s["scales"]
    z = (x @ s["a"].reshape(p * r, -1).float().t()).reshape(-1, p, r) * mine[:, :, None]
    return (x @ s["weight"].float() + z.reshape(-1, p * r) @ s["b"].reshape(p * r, -1).float()).to(s["x"].dtype)


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "gate":
        return _gate(state)
    if op == "gate_grad":
        return _gate_grad(state)
    if op == "glu":
        return _glu(state)
    return _glu_grad(state) if op == "glu_grad" else _lora(state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_act(name, g):
    if name == "silu":
        q = torch.sigmoid(g)
        return g * q, q + g * q * (1 - q)
    u = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    du = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
    return g * torch.sigmoid(2 * u), torch.sigmoid(2 * u) + g * 2 * du * torch.sigmoid(2 * u) * torch.sigmoid(-2 * u)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("gate", "gate_grad"):
        l = s["logits"].double()
        lse = torch.logsumexp(l, dim=1)
        p = torch.softmax(l, dim=1).nan_to_num(0.0)
        if op == "gate":
            key = s["logits"].float() if s["bias"] is None else s["logits"].float() + s["bias"]
            # experts by (key, index): an expert's place is the number of experts before it
            place = torch.empty(key.shape, dtype=torch.int64, device=key.device)
            index = torch.arange(key.shape[1], device=key.device)
            for e in range(key.shape[1]):
                mine = key[:, e:e + 1]
                place[:, e] = ((key > mine) | ((key == mine) & (index < e))).sum(dim=1)
            ids = place.argsort(dim=1)[:, :case["topk"]]
            w = p.gather(1, ids)
            if case["renorm"]:
                w = torch.softmax(l.gather(1, ids), dim=1).nan_to_num(0.0)
            return ids, w * case["scale"], lse
        chosen = torch.zeros_like(l, dtype=torch.bool).scatter(1, s["ids"], True)
        dw = torch.zeros_like(l).scatter(1, s["ids"], s["grad_probs"].double()) * case["scale"]
        w = torch.softmax(l.masked_fill(~chosen, float("-inf")), dim=1).nan_to_num(0.0) if case["renorm"] else p
        grad = w * (dw - (w * dw).sum(dim=1, keepdim=True))
        if s["grad_lse"] is not None:
            grad = grad + p * s["grad_lse"].double()[:, None]
        return grad
    if op == "lora":
        y = s["x"].double() @ s["weight"].double()
        for q in range(case["adapters"]):
            at = (s["ids"] == q).nonzero().squeeze(1)
            if at.numel():
                z = s["x"][at].double() @ s["a"][q].double().t().contiguous()
                y[at] += s["scales"][q].double() * (z @ s["b"][q].double())
        return y
    f = case["f"]
    counts = s["group_list"].tolist()
    if op == "glu":
        position = _position(s) // case["topk"]
        y = torch.empty((position.numel(), 2 * f), dtype=torch.float64, device="cuda")
        row = 0
        for g, n in enumerate(counts):
            if n:
                y[row:row + n] = s["x"][position[row:row + n]].double() @ s["weight"][g].double()
                row += n
        h = _exact_act(case["act"], y[:, :f])[0] * y[:, f:]
        return (h, y) if case["save"] else h
    grad = torch.empty((sum(counts), 2 * f), dtype=torch.float64, device="cuda")
    h = torch.empty((sum(counts), f), dtype=torch.float64, device="cuda")
    row = 0
    for g, n in enumerate(counts):
        if n:
            dh = s["grad_y"][row:row + n].double() @ s["weight"][g].double().t().contiguous()
            gate, up = s["gate_up"][row:row + n, :f].double(), s["gate_up"][row:row + n, f:].double()
            a, da = _exact_act(case["act"], gate)
            grad[row:row + n, :f], grad[row:row + n, f:], h[row:row + n] = dh * up * da, dh * a, a * up
            row += n
    return grad, h
