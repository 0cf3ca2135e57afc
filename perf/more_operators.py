"""Cases for timing and checking the grouped gate, the experts' products with
4-bit weights and the combination of the experts' rows with the residual
stream, each beside its plain form.

``listed()`` and ``draw(rng)`` give cases, ``prepare(case, seed)`` the inputs
on the GPU, ``run(state)`` one pass: the framework's operators where ``own``
is true, otherwise the same formulas in elementary torch operations on 32-bit
values (the gate's choice on 64-bit ones), rounded once at the end.
``exact(case, seed)`` evaluates the definitions in 64 bits, and ``work(case)``
counts the bytes and operations that a pass cannot do without.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
KINDS = ("gate", "gate_grad", "glu_w4", "fwd_w4", "combine", "combine_grad")
EPS = 1e-6


def listed():
    return [
        # the router of one decode step, experts in groups: the launch and the picks are all of it
        dict(name="gate decode", op="gate", dtype="bf16", tokens=16, experts=256, topk=8, groups=8, topk_groups=4,
             score="sigmoid", bias=True, renorm=True, scale=2.5, masked=False),
        # the router of a large training batch, with banned experts (-inf) and padding rows
        dict(name="gate train", op="gate", dtype="f32", tokens=13824, experts=256, topk=8, groups=8, topk_groups=4,
             score="sigmoid", bias=True, renorm=True, scale=2.5, masked=True),
        # the backward of a middling batch: softmax scores as they are, groups that fill no vector
        dict(name="gate grad mid", op="gate_grad", dtype="f16", tokens=2048, experts=60, topk=6, groups=4,
             topk_groups=2, score="softmax", bias=False, renorm=False, scale=1.0, masked=False),
        # the backward of the large training batch
        dict(name="gate grad train", op="gate_grad", dtype="bf16", tokens=13824, experts=256, topk=8, groups=8,
             topk_groups=4, score="sigmoid", bias=True, renorm=True, scale=2.5, masked=True),
        # one token through one small matrix: latency
        dict(name="w4 one token", op="fwd_w4", dtype="bf16", batch=1, topk=1, groups=1, empty=0, k=2048, n=1408,
             skew=0.0, group_size=32, zeros=True),
        # first products of a decode step: the used experts' weights are read once for 128 rows
        dict(name="w4 glu decode", op="glu_w4", dtype="bf16", batch=16, topk=8, groups=16, empty=4, k=7168, n=4096,
             skew=0.0, row_idx_type=0, act="silu", group_size=128, zeros=False),
        # second products at odd sizes: rows that start on no 16-byte boundary, a last group that is not full
        dict(name="w4 odd", op="fwd_w4", dtype="f16", batch=333, topk=2, groups=64, empty=5, k=1403, n=2039,
             skew=1.1, group_size=64, zeros=True),
        # a prefill batch over experts of very different popularity
        dict(name="w4 glu prefill", op="glu_w4", dtype="bf16", batch=2048, topk=8, groups=16, empty=0, k=7168, n=4096,
             skew=1.1, row_idx_type=1, act="silu", group_size=128, zeros=True),
        # the end of a decode step's block
        dict(name="combine decode", op="combine", dtype="bf16", batch=16, topk=8, h=7168, row_idx_type=1, post=True,
             gate=False, next=True, alpha=1.0),
        # the end of a large training batch's block
        dict(name="combine train", op="combine", dtype="f16", batch=13824, topk=8, h=7168, row_idx_type=1, post=True,
             gate=True, next=True, alpha=0.5),
        # its backward at odd sizes, in fp32, from the other form of the routing index
        dict(name="combine grad odd", op="combine_grad", dtype="f32", batch=333, topk=2, h=2039, row_idx_type=0,
             post=True, gate=True, next=True, alpha=0.7),
        # the backward of the large training batch
        dict(name="combine grad train", op="combine_grad", dtype="bf16", batch=13824, topk=8, h=7168, row_idx_type=1,
             post=True, gate=True, next=True, alpha=1.0),
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
        groups = rng.choice((1, 2, 3, 4, 8, 8, 16))
        each = _spread(rng, 2, 512 // groups)
        chosen = rng.randint(1, groups)
        return dict(op=op, dtype=dtype, tokens=_spread(rng, 1, 13824), experts=groups * each,
                    topk=rng.randint(1, min(8, chosen * each)), groups=groups, topk_groups=chosen,
                    score=rng.choice(("sigmoid", "softmax")), bias=rng.random() < 0.5, renorm=rng.random() < 0.5,
                    scale=rng.choice((1.0, 2.5)), masked=rng.random() < 0.5)
    while True:
        if op in ("combine", "combine_grad"):
            c = dict(op=op, dtype=dtype, batch=_spread(rng, 1, 13824), topk=rng.randint(1, 8), h=_width(rng, 64, 8192),
                     row_idx_type=rng.randint(0, 1), post=rng.random() < 0.7, gate=rng.random() < 0.5,
                     next=rng.random() < 0.7, alpha=rng.choice((1.0, 0.7)))
            if work(c)["bytes"] <= 3e9:
                return c
            continue
        groups = _spread(rng, 1, 64)
        empty = rng.randint(0, groups // 4)
        c = dict(op=op, dtype=dtype, batch=_spread(rng, 1, 2048), topk=rng.randint(1, min(8, groups - empty)),
                 groups=groups, empty=empty, k=_width(rng, 64, 7168), n=_width(rng, 64, 7168),
                 skew=rng.choice((0.0, 1.1)), group_size=rng.choice((32, 64, 128, 128, 256)), zeros=rng.random() < 0.5)
        if op == "glu_w4":
            c.update(n=c["n"] // 2 * 2, row_idx_type=rng.randint(0, 1), act=rng.choice(("silu", "silu", "gelu_tanh")))
        if work(c)["flops"] <= (1e11 if dtype == "f32" else 9e11) and groups * c["k"] * c["n"] <= 1.2e9:
            return c


def work(case):
    s = SIZES[case["dtype"]]
    op = case["op"]
    if op in ("gate", "gate_grad"):
        t, e, k = case["tokens"], case["experts"], case["topk"]
        if op == "gate":   # logits read; ids and weights written
            return {"bytes": t * e * s + t * k * 12 + (4 * e if case["bias"] else 0), "flops": 4.0 * t * e}
        # the picks' logits read (of softmax scores the whole row), the gradient's row written
        read = t * e * s if case["score"] == "softmax" and not case["renorm"] else t * k * s
        return {"bytes": read + t * e * s + t * k * 12, "flops": 8.0 * t * k}
    if op in ("combine", "combine_grad"):
        b, m, h = case["batch"], case["batch"] * case["topk"], case["h"]
        vectors = s * h * (case["post"] + case["next"])
        if op == "combine":
            return {"bytes": s * h * (m + 2 * b + (b if case["next"] else 0)) + 12 * m + (4 * b if case["gate"] else 0)
                    + vectors, "flops": 2.0 * m * h + 8.0 * b * h}
        return {"bytes": s * h * (2 * m + 3 * b + (b if case["next"] else 0)) + 16 * m + (8 * b if case["gate"] else 0)
                + vectors + 4 * h * (case["post"] + case["next"]), "flops": 5.0 * m * h + 20.0 * b * h}
    m, k, n = case["batch"] * case["topk"], case["k"], case["n"]
    used = min(case["groups"] - case["empty"], m)
    rows = -(-k // case["group_size"])
    weights = used * (k * n / 2 + rows * n * (s + (1 if case["zeros"] else 0)))
    if op == "glu_w4":
        return {"bytes": weights + s * (case["batch"] * k + m * n // 2) + 8 * m + 8 * case["groups"],
                "flops": 2.0 * m * k * n}
    return {"bytes": weights + s * m * (k + n) + 8 * case["groups"], "flops": 2.0 * m * k * n}


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
    for part in out.chunk(8):   # large ones: a slice at a time
        part.copy_(torch.randn(part.shape, generator=gen, device=dev) * std)
    return out


def _choose(logits, bias, case):
    """The gate's experts [T, topk]: keys in 64 bits, the groups' two largest
    added, larger first and equal ones by lower index."""
    l = logits.double()
    live = l != float("-inf")
    if case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        top = l.amax(dim=1, keepdim=True)
        e = torch.exp(l - torch.where(top == float("-inf"), 0.0, top))
        s = e / e.sum(dim=1, keepdim=True)
    key = (s if bias is None else s + bias.double()).masked_fill(~live, float("-inf"))
    groups = case["groups"]
    if groups > 1:
        best = torch.sort(key.reshape(key.shape[0], groups, -1), dim=2, descending=True).values
        score = best[:, :, 0]
        if best.shape[2] > 1:   # an excluded expert adds nothing to its group
            score = score + torch.where(best[:, :, 1] == float("-inf"), 0.0, best[:, :, 1])
        chosen = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        allowed = torch.zeros_like(score, dtype=torch.bool).scatter(1, chosen, True)
        allowed = allowed.repeat_interleave(key.shape[1] // groups, dim=1)
    else:
        allowed = torch.ones_like(live)
    # experts of other groups come behind the excluded ones of the chosen groups
    key = key.clamp_min(-1e300).masked_fill(~allowed, float("-inf"))
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, :case["topk"]].contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(1000003 * int(seed) + 29)
    dtype = DTYPES[case["dtype"]]
    op = case["op"]
    s = {"case": case}
    if op in ("gate", "gate_grad"):
        t, e = case["tokens"], case["experts"]
        logits = torch.randn((t, e), generator=gen, device=dev) * 1.5
        if case["masked"]:
            banned = torch.rand((t, e), generator=gen, device=dev) < 0.1
            banned[torch.rand((t,), generator=gen, device=dev) < 0.01] = True   # padding rows: nothing left
            logits = logits.masked_fill(banned, float("-inf"))
        s["logits"] = logits.to(dtype)
        spread = 0.1 if case["score"] == "sigmoid" else 0.3 / e
        s["bias"] = torch.randn((e,), generator=gen, device=dev) * spread if case["bias"] else None
        if op == "gate_grad":
            s["ids"] = _choose(s["logits"], s["bias"], case)
            s["grad_probs"] = torch.randn((t, case["topk"]), generator=gen, device=dev)
        return s
    if op in ("combine", "combine_grad"):
        b, k, h = case["batch"], case["topk"], case["h"]
        s["rows"] = torch.randperm(b * k, generator=gen, device=dev)
        s["permuted"] = _values(gen, dev, dtype, 0.5, b * k, h)
        s["probs"] = torch.softmax(torch.randn((b, k), generator=gen, device=dev), dim=1)
        s["residual"] = _values(gen, dev, dtype, 1.0, b, h)
        s["post"] = (1 + 0.1 * torch.randn((h,), generator=gen, device=dev)).to(dtype) if case["post"] else None
        s["next"] = (1 + 0.1 * torch.randn((h,), generator=gen, device=dev)).to(dtype) if case["next"] else None
        s["gate"] = torch.rand((b,), generator=gen, device=dev) * 2 if case["gate"] else None
        if op == "combine_grad":
            s["grad_out"] = _values(gen, dev, dtype, 1.0, b, h)
            s["grad_normed"] = _values(gen, dev, dtype, 1.0, b, h) if case["next"] else None
        return s
    g, k, n = case["groups"], case["k"], case["n"]
    eri, s["group_list"], s["cap"] = _routing(case, gen, dev)
    if op == "glu_w4":
        s["x"], s["eri"] = _values(gen, dev, dtype, 1.0, case["batch"], k), eri
    else:   # the second product: its rows are in expert order already
        s["x"] = _values(gen, dev, dtype, 1.0, case["batch"] * case["topk"], k)
    rows = -(-k // case["group_size"])
    s["codes"] = torch.randint(0, 16, (g, k, n), generator=gen, device=dev, dtype=torch.uint8)
    s["scales"] = ((0.5 + torch.rand((g, rows, n), generator=gen, device=dev)) * 0.25 / math.sqrt(k)).to(dtype)
    s["zeros"] = (torch.randint(5, 12, (g, rows, n), generator=gen, device=dev, dtype=torch.uint8)
                  if case["zeros"] else None)
    return s


# ---------------------------------------------------------------- the framework's operators

def _run_own(s):
    import permute_grouped_gemm_amd as pgg

    c = s["case"]
    op = c["op"]
    if op == "gate":
        return pgg.moe_gate_grouped(s["logits"], c["topk"], score=c["score"], groups=c["groups"],
                                    topk_groups=c["topk_groups"], bias=s["bias"], renorm=c["renorm"], scale=c["scale"])
    if op == "gate_grad":
        return pgg.moe_gate_grouped_grad(s["logits"], s["ids"], s["grad_probs"], score=c["score"], renorm=c["renorm"],
                                         scale=c["scale"])
    if op in ("glu_w4", "fwd_w4"):
        if "weight" not in s:   # laid out once, as the program loads its weights
            s["weight"] = pgg.w4_pack(s["codes"], s["scales"], c["group_size"], zeros=s["zeros"],
                                      gated=op == "glu_w4")
        if op == "glu_w4":
            args, call = (s["x"], s["weight"], s["eri"], s["group_list"], c["topk"], c["row_idx_type"]), pgg.moe_glu_w4
            extra = {"act": c["act"]}
        else:
            args, call, extra = (s["x"], s["weight"], None, s["group_list"]), pgg.moe_fwd_w4, {}
        if "workspace" not in s:
            s["workspace"] = torch.empty(pgg.w4_workspace_size(*args), dtype=torch.uint8, device="cuda")
        return call(*args, workspace=s["workspace"], **extra)
    kind = dict(row_idx_type=c["row_idx_type"], post_weight=s["post"], gate=s["gate"], residual_scale=c["alpha"],
                next_weight=s["next"], eps=EPS)
    if "workspace" not in s:
        size = pgg.combine_workspace_size if op == "combine" else pgg.combine_grad_workspace_size
        s["workspace"] = torch.empty(size(s["permuted"], s["probs"], row_idx_type=c["row_idx_type"]),
                                     dtype=torch.uint8, device="cuda")
    if op == "combine":
        return pgg.moe_combine(s["permuted"], s["rows"], s["probs"], s["residual"], workspace=s["workspace"], **kind)
    grads = pgg.moe_combine_grad(s["grad_out"], s["permuted"], s["rows"], s["probs"], s["residual"],
                                 grad_normed=s["grad_normed"], workspace=s["workspace"], **kind)
    return tuple(g for g in grads if g is not None)


# ---------------------------------------------------------------- the plain forms

def _scores(s):
    """Weights of the chosen experts before the scale (32 bits), and the chosen
    experts' share that the sigmoid leaves, 1 - s."""
    c = s["case"]
    l = s["logits"].float()
    p = l.gather(1, s["ids"])
    if c["score"] == "sigmoid":
        rest = 1 / (1 + torch.exp(p))
        if not c["renorm"]:
            return 1 / (1 + torch.exp(-p)), rest
        p = p.clamp_max(0) - torch.log1p(torch.exp(-p.abs()))   # the scores' logarithms
    else:
        rest = None
        if not c["renorm"]:
            top = l.amax(dim=1, keepdim=True)
            top = torch.where(top == float("-inf"), 0.0, top)
            total = torch.exp(l - top).sum(dim=1, keepdim=True)
            return torch.where(total > 0, torch.exp(p - top) / total, 0.0), rest
    top = p.amax(dim=1, keepdim=True)
    e = torch.exp(p - torch.where(top == float("-inf"), 0.0, top))
    total = e.sum(dim=1, keepdim=True)
    return torch.where(total > 0, e / total, 0.0), rest


def _gate(s):
    ids = _choose(s["logits"], s["bias"], s["case"])
    return ids, _scores({**s, "ids": ids})[0] * s["case"]["scale"]


def _gate_grad(s):
    c = s["case"]
    l, d = s["logits"].float(), s["grad_probs"] * c["scale"]
    w, rest = _scores(s)
    if c["score"] == "softmax" and not c["renorm"]:
        top = l.amax(dim=1, keepdim=True)
        e = torch.exp(l - torch.where(top == float("-inf"), 0.0, top))
        total = e.sum(dim=1, keepdim=True)
        p = torch.where(total > 0, e / total, 0.0)
        at = torch.zeros_like(l).scatter(1, s["ids"], d)
        return (p * (at - (d * w).sum(dim=1, keepdim=True))).to(s["logits"].dtype)
    if c["renorm"]:
        d = d - (d * w).sum(dim=1, keepdim=True)
    grad = d * w if rest is None else d * w * rest
    return torch.zeros_like(l).scatter(1, s["ids"], grad).to(s["logits"].dtype)


def _by_expert(s, rows, weight):
    """rows[i] times the weight of the row's expert: rows padded to the fullest
    expert, one batched product."""
    counts = s["group_list"]
    ends = counts.cumsum(0)
    place = torch.arange(s["cap"], device=rows.device)
    at = (ends - counts)[:, None] + torch.minimum(place, (counts - 1).clamp_min(0)[:, None])
    y = torch.bmm(rows[at.clamp_max(rows.shape[0] - 1)].float(), weight)
    i = torch.arange(rows.shape[0], device=rows.device)
    g = torch.searchsorted(ends, i, right=True)
    return y.reshape(-1, y.shape[2])[g * s["cap"] + i - (ends - counts)[g]]


def _weights(s):
    """The weights that codes, scales and zero points stand for, in 32 bits."""
    of = torch.arange(s["codes"].shape[1], device=s["codes"].device) // s["case"]["group_size"]
    zero = 8.0 if s["zeros"] is None else s["zeros"].float()[:, of]
    return (s["codes"].float() - zero) * s["scales"].float()[:, of]


def _position(s):
    """Original position of every expanded row."""
    if s["case"]["row_idx_type"] == 0:
        return s["eri"]
    p = torch.empty_like(s["eri"])
    p[s["eri"]] = torch.arange(p.numel(), device=p.device)
    return p


def _fwd_w4(s):
    return _by_expert(s, s["x"], _weights(s)).to(s["x"].dtype)


def _glu_w4(s):
    c = s["case"]
    gate, up = _by_expert(s, s["x"][_position(s) // c["topk"]], _weights(s)).chunk(2, dim=1)
    if c["act"] == "silu":
        a = gate / (1 + torch.exp(-gate))
    else:
        a = 0.5 * gate * (1 + torch.tanh(math.sqrt(2 / math.pi) * (gate + 0.044715 * gate * gate * gate)))
    return (a * up).to(s["x"].dtype)


def _slots(s):
    """Expanded row of every token's slots [batch, topk]."""
    rows = s["rows"]
    if s["case"]["row_idx_type"] == 0:
        back = torch.empty_like(rows)
        back[rows] = torch.arange(rows.numel(), device=rows.device)
        rows = back
    return rows.reshape(s["probs"].shape)


def _combined(s):
    """Intermediate values of the combination, in 32 bits."""
    y = s["permuted"][_slots(s)].float()
    c = (s["probs"][:, :, None] * y).sum(dim=1)
    r = torch.rsqrt((c * c).mean(dim=1, keepdim=True) + EPS) if s["post"] is not None else None
    a = c if r is None else c * r * s["post"].float()
    ga = a if s["gate"] is None else a * s["gate"][:, None]
    out = s["case"]["alpha"] * s["residual"].float() + ga
    q = torch.rsqrt((out * out).mean(dim=1, keepdim=True) + EPS) if s["next"] is not None else None
    return y, c, r, a, out, q


def _combine(s):
    _, _, _, _, out, q = _combined(s)
    t = s["permuted"].dtype
    return out.to(t) if q is None else (out.to(t), (out * q * s["next"].float()).to(t))


def _combine_grad(s):
    t = s["permuted"].dtype
    y, c, r, a, out, q = _combined(s)
    go = s["grad_out"].float()
    grad_next = grad_gate = grad_post = None
    if q is not None:
        gn = s["grad_normed"].float()
        grad_next = (gn * out * q).sum(dim=0)
        u = gn * s["next"].float()
        go = go + q * u - out * q * q * q * (u * out).mean(dim=1, keepdim=True)
    grad_residual = (go * s["case"]["alpha"]).to(t)
    if s["gate"] is not None:
        grad_gate = (go * a).sum(dim=1)
        go = go * s["gate"][:, None]
    if r is not None:
        grad_post = (go * c * r).sum(dim=0)
        u = go * s["post"].float()
        go = r * u - c * r * r * r * (u * c).mean(dim=1, keepdim=True)
    grad_probs = (go[:, None, :] * y).sum(dim=2)
    grad_permuted = torch.empty_like(s["permuted"])
    grad_permuted[_slots(s).reshape(-1)] = (s["probs"][:, :, None] * go[:, None, :]).to(t).reshape(-1, go.shape[1])
    grads = (grad_permuted, grad_probs, grad_residual, grad_gate, grad_post, grad_next)
    return tuple(g for g in grads if g is not None)


PLAIN = {"gate": _gate, "gate_grad": _gate_grad, "glu_w4": _glu_w4, "fwd_w4": _fwd_w4, "combine": _combine,
         "combine_grad": _combine_grad}


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _place(key):
    """Place of every entry of a row: the number of entries before it."""
    place = torch.empty(key.shape, dtype=torch.int64, device=key.device)
    index = torch.arange(key.shape[1], device=key.device)
    for e in range(key.shape[1]):
        mine = key[:, e:e + 1]
        place[:, e] = ((key > mine) | ((key == mine) & (index < e))).sum(dim=1)
    return place


def _exact_gate(s):
    c = s["case"]
    l = s["logits"].double()
    score = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, dim=1).nan_to_num(0.0)
    if c["op"] == "gate":
        key = score if s["bias"] is None else score + s["bias"].double()
        key = torch.where(torch.isinf(l), -1e300, key)   # banned
        each = c["experts"] // c["groups"]
        first, second = (key.reshape(-1, c["groups"], each).topk(min(2, each), dim=2).values.unbind(2) + (None,))[:2]
        if c["groups"] > 1:
            sums = first if second is None else first + torch.where(second < -1e299, 0.0, second)
            out = (_place(sums) >= c["topk_groups"])[:, :, None].expand(-1, -1, each).reshape(key.shape)
            key = torch.where(out, -2e300, key)
        ids = _place(key).argsort(dim=1)[:, :c["topk"]]
    else:
        ids = s["ids"]
    if c["score"] == "sigmoid":
        logs = torch.nn.functional.logsigmoid(l.gather(1, ids))
    else:
        logs = l.gather(1, ids)
    if c["renorm"]:
        w = torch.softmax(logs, dim=1).nan_to_num(0.0)
    else:
        w = score.gather(1, ids)
    if c["op"] == "gate":
        return ids, w * c["scale"]
    d = s["grad_probs"].double() * c["scale"]
    mean = (d * w).sum(dim=1, keepdim=True)
    if c["score"] == "softmax" and not c["renorm"]:
        return score * (torch.zeros_like(l).scatter(1, ids, d) - mean)
    grad = w * (d - mean) if c["renorm"] else w * d
    if c["score"] == "sigmoid":
        grad = grad * torch.sigmoid(-l.gather(1, ids))
    return torch.zeros_like(l).scatter(1, ids, grad)


def _exact_w4(s):
    c = s["case"]
    x = s["x"] if c["op"] == "fwd_w4" else s["x"][_position(s) // c["topk"]]
    y = torch.empty((x.shape[0], c["n"]), dtype=torch.float64, device="cuda")
    row, size = 0, c["group_size"]
    for g, rows in enumerate(s["group_list"].tolist()):
        if rows:
            part = torch.zeros((rows, c["n"]), dtype=torch.float64, device="cuda")
            xs = x[row:row + rows].double()
            q = s["codes"][g].double() - (8 if s["zeros"] is None else
                                          s["zeros"][g].double().repeat_interleave(size, dim=0)[:c["k"]])
            part = xs @ (q * s["scales"][g].double().repeat_interleave(size, dim=0)[:c["k"]])
            y[row:row + rows] = part
            row += rows
    if c["op"] == "fwd_w4":
        return y
    gate, up = y[:, :c["n"] // 2], y[:, c["n"] // 2:]
    if c["act"] == "silu":
        return gate * torch.sigmoid(gate) * up
    return gate * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3)) * up


def _exact_combine(s):
    c = s["case"]
    names = [n for n in ("permuted", "probs", "residual", "gate", "post", "next") if s[n] is not None]
    wide = {n: s[n].double().requires_grad_(c["op"] == "combine_grad") for n in names}
    flat = s["rows"] if c["row_idx_type"] == 1 else torch.argsort(s["rows"])
    # one slot at a time: the sum over a token's experts
    acc = 0
    for j in range(c["topk"]):
        acc = acc + wide["permuted"].index_select(0, flat[j::c["topk"]]) * wide["probs"][:, j:j + 1]
    norm = lambda v: v / (v.pow(2).mean(dim=1, keepdim=True) + EPS).sqrt()  # noqa: E731
    if "post" in wide:
        acc = norm(acc) * wide["post"]
    if "gate" in wide:
        acc = acc * wide["gate"][:, None]
    out = wide["residual"] * c["alpha"] + acc
    results = (out, norm(out) * wide["next"]) if "next" in wide else (out,)
    if c["op"] == "combine":
        return results if len(results) > 1 else out
    up = (s["grad_out"].double(),) + ((s["grad_normed"].double(),) if "next" in wide else ())
    return torch.autograd.grad(results, [wide[n] for n in names], up)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("gate", "gate_grad"):
        return _exact_gate(s)
    return _exact_combine(s) if case["op"] in ("combine", "combine_grad") else _exact_w4(s)
