"""Unpermute with the norms and the residual stream behind it, and its gradient,
against their 64-bit forms."""
import itertools

import pytest
import torch

import block_ref as ref
import ops_ref
import permute_grouped_gemm_amd as pgg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(batch, topk, H, dtype, post, gate, nxt, seed=0):
    gen = torch.Generator().manual_seed(seed)
    T = ops_ref.DTYPES[dtype]
    rand = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    s = dict(permuted=rand(batch * topk, H).to(T), eri=torch.randperm(batch * topk, generator=gen),
             probs=torch.softmax(rand(batch, topk), dim=1), residual=rand(batch, H).to(T))
    s["post"] = (1 + 0.2 * rand(H)).to(T) if post else None
    s["gate"] = rand(batch) if gate else None
    s["nxt"] = (1 + 0.2 * rand(H)).to(T) if nxt else None
    s["grad_out"], s["grad_normed"] = rand(batch, H).to(T), rand(batch, H).to(T) if nxt else None
    return s


def _dev(t):
    return None if t is None else t.to(DEV)


def _run(s, rit, alpha, eps, grad, workspace=None):
    kw = dict(row_idx_type=rit, post_weight=_dev(s["post"]), gate=_dev(s["gate"]), residual_scale=alpha,
              next_weight=_dev(s["nxt"]), eps=eps, workspace=workspace)
    args = [_dev(s[n]) for n in ("permuted", "eri", "probs", "residual")]
    if grad:
        return pgg.moe_combine_grad(_dev(s["grad_out"]), *args, grad_normed=_dev(s["grad_normed"]), **kw)
    r = pgg.moe_combine(*args, **kw)
    return r if isinstance(r, tuple) else (r,)


def _check(batch, topk, H, dtype, rit, post, gate, nxt, alpha=0.7, eps=1e-5, seed=0):
    s = _inputs(batch, topk, H, dtype, post, gate, nxt, seed)
    names = ("permuted", "eri", "probs", "residual", "post", "gate", "nxt")
    plain = {n: s[n] for n in names}
    probs = s["probs"].to(DEV)
    for grad in (False, True):
        size = pgg.combine_grad_workspace_size if grad else pgg.combine_workspace_size
        ws = torch.full((size(s["permuted"].to(DEV), probs, row_idx_type=rit),), 0xAB, dtype=torch.uint8, device=DEV)
        got = _run(s, rit, alpha, eps, grad, ws)
        torch.cuda.synchronize()
        assert pgg.read_device_error(ws) == (pgg.DEV_OK, 0)
        extra = dict(grad_out=s["grad_out"], grad_normed=s["grad_normed"]) if grad else {}
        want = ref.combine(**plain, row_idx_type=rit, alpha=alpha, eps=eps, **extra)
        order = ("permuted", "probs", "residual", "gate", "post", "next") if grad else ("out", "normed")
        for name, t in zip(order, got):
            if t is None:
                assert name not in want
                continue
            near = want.pop(name)
            ops_ref.assert_within(t, near.v, ops_ref.rounded(near.v, near.e, t.dtype), f"{name} grad={grad}")
        assert not want


# one token and many; rows shorter than a wave's piece, odd, at the kernels'
# edges (8192, 16384) and beyond one piece; more slots than stay in registers
SHAPES = [(1, 1, 1), (1, 8, 64), (3, 2, 7), (5, 3, 130), (16, 8, 520), (33, 1, 1000), (7, 9, 257), (300, 4, 96),
          (2, 17, 2048), (4, 2, 8192), (3, 3, 8200), (2, 2, 9001), (2, 5, 16384), (600, 2, 72)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("batch,topk,H", SHAPES)
def test_combine_and_gradient(batch, topk, H, dtype):
    _check(batch, topk, H, dtype, 0, True, True, True, seed=H)
    _check(batch, topk, H, dtype, 1, True, False, True, alpha=1.0, seed=H + 1)


@pytest.mark.parametrize("post,gate,nxt", list(itertools.product((False, True), repeat=3)))
def test_every_part_may_be_missing(post, gate, nxt):
    for dtype, rit, shape in (("bf16", 0, (9, 3, 200)), ("f32", 1, (300, 2, 64)), ("f16", 1, (11, 12, 129)),
                              ("bf16", 1, (2, 3, 8232))):
        _check(*shape, dtype, rit, post, gate, nxt, seed=4)


def test_large_batch():
    # more tokens than workgroups of the gradient, indexes of both kinds beyond the spare workgroup's bits
    for rit in (0, 1):
        _check(5000, 4, 40, "bf16", rit, True, True, True)


def test_rows_of_zeros():
    s = _inputs(4, 2, 96, "f32", True, True, True)
    s["permuted"][:] = 0
    s["residual"][1] = 0
    for grad in (False, True):
        for t in _run(s, 0, 1.0, 1e-6, grad):
            assert bool(t.isfinite().all())
    out, normed = _run(s, 0, 1.0, 1e-6, False)
    assert torch.equal(out.cpu(), s["residual"]) and bool((normed[1] == 0).all())


def test_nan_and_infinity_stay_in_their_tokens():
    s = _inputs(6, 2, 64, "f32", True, False, True)
    at = ref.slots(s["eri"], 6, 2, 1)
    s["permuted"][at[2, 1], 5] = float("nan")
    s["permuted"][at[4, 0], 9] = float("inf")
    clean = _inputs(6, 2, 64, "f32", True, False, True)
    for grad in (False, True):
        got, want = _run(s, 1, 1.0, 1e-6, grad), _run(clean, 1, 1.0, 1e-6, grad)
        for n, (a, b) in enumerate(zip(got, want)):
            if a is None or a.dim() == 1:
                continue
            rows = [0, 1, 3, 5] if a.shape[0] == 6 else at[[0, 1, 3, 5]].reshape(-1).tolist()
            assert torch.equal(a[rows], b[rows]), (grad, n)


def test_gradient_against_differences():
    s = _inputs(3, 2, 20, "f32", True, True, True, seed=9)
    got = dict(zip(("permuted", "probs", "residual", "gate", "post", "nxt"), _run(s, 0, 0.9, 1e-3, True)))
    wide = {n: s[n].double() for n in got}
    at = ref.slots(s["eri"], 3, 2, 0)

    def f(v):   # the definition, written out
        c = (v["permuted"][at] * v["probs"][:, :, None]).sum(dim=1)
        a = c / (c.pow(2).mean(dim=1, keepdim=True) + 1e-3).sqrt() * v["post"]
        out = 0.9 * v["residual"] + v["gate"][:, None] * a
        n = out / (out.pow(2).mean(dim=1, keepdim=True) + 1e-3).sqrt() * v["nxt"]
        return (out * s["grad_out"].double()).sum() + (n * s["grad_normed"].double()).sum()

    h = 1e-5
    for name, g in got.items():
        flat = g.cpu().double().reshape(-1)
        for i in range(0, flat.numel(), 3):
            step = torch.zeros(flat.numel(), dtype=torch.float64)
            step[i] = h
            step = step.reshape(g.shape)
            num = (f({**wide, name: wide[name] + step}) - f({**wide, name: wide[name] - step})) / (2 * h)
            # fp32 sums of some 60 terms of size up to 10: 60 * 10 * 2^-23; the difference's h^2 is below it
            assert abs(flat[i] - num) <= 1e-4 * (1 + abs(num)), (name, i)


def test_repeated_calls_give_the_same_bits():
    s = _inputs(700, 8, 264, "bf16", True, True, True)
    for grad in (False, True):
        first = _run(s, 1, 1.0, 1e-6, grad)
        for _ in range(4):
            for a, b in zip(_run(s, 1, 1.0, 1e-6, grad), first):
                assert torch.equal(a, b)


def test_both_forms_of_the_index_agree():
    s = _inputs(50, 3, 136, "f16", True, False, True)
    back = {**s, "eri": torch.empty_like(s["eri"])}
    back["eri"][s["eri"]] = torch.arange(150)
    for grad in (False, True):
        for a, b in zip(_run(s, 0, 1.0, 1e-6, grad), _run(back, 1, 1.0, 1e-6, grad)):
            assert a is None and b is None or torch.equal(a, b)


def test_agrees_with_unpermute():
    s = _inputs(40, 4, 256, "f32", False, False, False)
    s["residual"][:] = 0
    out, = _run(s, 0, 1.0, 1e-6, False)
    want = pgg.moe_unpermute(_dev(s["permuted"]), _dev(s["eri"]), 40, 4, 0, _dev(s["probs"]))
    # both add four products in slot order; one of them fuses each with its addition
    assert torch.allclose(out, want, rtol=0, atol=8 * 2.0 ** -24 * 4 * float(s["permuted"].abs().max()))


def test_bad_indexes_are_reported():
    for batch, topk in ((8, 2), (3000, 4)):
        s = _inputs(batch, topk, 64, "bf16", True, True, True)
        M = batch * topk
        for bad, code in ((torch.where(s["eri"] == 3, M, s["eri"]), pgg.DEV_INDEX_RANGE),
                          (torch.where(s["eri"] == 3, -5, s["eri"]), pgg.DEV_INDEX_RANGE),
                          (torch.where(s["eri"] == 3, 1 << 40, s["eri"]), pgg.DEV_INDEX_RANGE),
                          (torch.where(s["eri"] == 3, 4, s["eri"]), pgg.DEV_INDEX_DUP)):
            for rit in (0, 1):
                for grad in (False, True):
                    size = pgg.combine_grad_workspace_size if grad else pgg.combine_workspace_size
                    ws = torch.empty(size(_dev(s["permuted"]), _dev(s["probs"])), dtype=torch.uint8, device=DEV)
                    _run({**s, "eri": bad}, rit, 1.0, 1e-6, grad, ws)
                    assert pgg.read_device_error(ws)[0] == code, (batch, rit, grad)


def test_unaligned_tensors():
    s = _inputs(5, 2, 64, "bf16", True, True, True)

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        flat[1:] = t.to(DEV).reshape(-1)
        return flat[1:].reshape(t.shape)

    want = _run(s, 0, 1.0, 1e-6, False) + _run(s, 0, 1.0, 1e-6, True)
    moved = {n: shifted(t) for n, t in s.items()}
    for a, b in zip(_run(moved, 0, 1.0, 1e-6, False) + _run(moved, 0, 1.0, 1e-6, True), want):
        assert torch.equal(a, b)


def test_refusals():
    s = {n: _dev(t) for n, t in _inputs(4, 2, 32, "bf16", True, True, True).items()}
    ok = dict(permuted=s["permuted"], expanded_row_idx=s["eri"], probs=s["probs"], residual=s["residual"])
    for bad in (dict(permuted=s["permuted"][:7]), dict(permuted=s["permuted"].double()), dict(probs=s["probs"].half()),
                dict(probs=s["probs"][0]), dict(residual=s["residual"].float()), dict(residual=s["residual"][:3]),
                dict(expanded_row_idx=s["eri"].int()), dict(expanded_row_idx=s["eri"][:7]),
                dict(post_weight=s["post"][:31]), dict(next_weight=s["nxt"].float()), dict(gate=s["gate"].half()),
                dict(gate=s["gate"][:3]), dict(row_idx_type=2), dict(eps=-1.0), dict(normed=torch.empty_like(s["residual"])),
                dict(out=s["permuted"]), dict(permuted=s["permuted"].cpu()),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(pgg.PggError):
            pgg.moe_combine(**{**ok, **bad})
    ok["grad_out"] = s["grad_out"]
    for bad in (dict(grad_out=s["grad_out"].float()), dict(next_weight=s["nxt"]), dict(grad_normed=s["grad_normed"]),
                dict(next_weight=s["nxt"], grad_normed=s["grad_normed"][:3])):
        with pytest.raises(pgg.PggError):
            pgg.moe_combine_grad(**{**ok, **bad})
