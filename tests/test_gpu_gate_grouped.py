"""The gate over experts in groups and its gradient against their 64-bit forms."""
import math

import pytest
import torch

import block_ref as ref
import ops_ref
import permute_grouped_gemm_amd as pgg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _logits(T, E, dtype, seed, std=1.5):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=gen) * std).to(ops_ref.DTYPES[dtype])


def _check(logits, topk, **kw):
    dev = {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in kw.items()}
    ids, probs = pgg.moe_gate_grouped(logits.to(DEV), topk, **dev)
    torch.cuda.synchronize()
    want, p, ep = ref.gate_grouped(logits, topk, **kw)
    assert ids.dtype == torch.int64 and probs.dtype == torch.float32
    assert torch.equal(ids.cpu(), want)
    ops_ref.assert_within(probs, p, ep, "probs")
    return ids, probs


def _check_grad(logits, ids, seed=0, **kw):
    gen = torch.Generator().manual_seed(seed)
    gp = torch.randn(ids.shape, generator=gen)
    got = pgg.moe_gate_grouped_grad(logits.to(DEV), ids.to(DEV), gp.to(DEV), **kw)
    torch.cuda.synchronize()
    assert got.dtype == logits.dtype
    want, err = ref.gate_grouped_grad(logits, ids, gp, **kw)
    ops_ref.assert_within(got, want, ops_ref.rounded(want, err, logits.dtype), "grad")


# experts, groups, kept groups, picks: groups of whole vectors and not, of one
# expert, over several lanes; every kernel's sizes and the ones around them
SHAPES = [(1, 1, 1, 1), (8, 1, 1, 3), (16, 4, 2, 4), (60, 4, 2, 6), (60, 60, 9, 9), (64, 8, 4, 8), (65, 5, 3, 7),
          (128, 8, 2, 8), (129, 3, 1, 5), (160, 8, 3, 6), (255, 15, 4, 12), (256, 8, 4, 8), (256, 1, 1, 8),
          (258, 6, 5, 20), (512, 8, 4, 8), (384, 8, 4, 16), (513, 9, 4, 11), (1024, 64, 5, 40), (1020, 12, 7, 64),
          (1025, 5, 2, 8), (8192, 64, 3, 64), (3000, 1, 1, 9)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("E,groups,kept,k", SHAPES)
def test_gate_and_gradient(E, groups, kept, k, dtype):
    for n, (score, renorm, with_bias) in enumerate((("sigmoid", True, True), ("softmax", False, False),
                                                    ("sigmoid", False, False), ("softmax", True, True))):
        T = (1, 5, 19, 33)[n]
        logits = _logits(T, E, dtype, E + 7 * n)
        bias = None
        if with_bias:
            bias = torch.randn((E,), generator=torch.Generator().manual_seed(E)) * (0.1 if score == "sigmoid" else 0.3 / E)
        ids, _ = _check(logits, k, score=score, groups=groups, topk_groups=kept, bias=bias, renorm=renorm, scale=2.5)
        _check_grad(logits, ids.cpu(), score=score, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("E,groups,kept,k", [(16, 4, 2, 5), (60, 4, 3, 8), (256, 8, 4, 8), (2000, 8, 3, 8)])
def test_equal_keys_go_to_the_lowest_index(E, groups, kept, k):
    l = torch.zeros((5, E))
    l[1] = -0.0
    l[1, ::2] = 0.0
    l[2] = torch.arange(E) % 3
    l[3] = torch.finfo(torch.float32).min          # sigmoid scores of 0
    l[4] = 60.0 + torch.arange(E) % 5              # sigmoid scores of 1
    for dtype in (torch.float32, torch.bfloat16):
        _check(l.to(dtype), k, groups=groups, topk_groups=kept)
        _check(l[:4].to(dtype), k, groups=groups, topk_groups=kept, bias=torch.zeros(E))
        _check(l[:4].to(dtype), k, score="softmax", groups=groups, topk_groups=kept)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,kept,k", [(16, 4, 2, 5), (60, 4, 3, 8), (256, 8, 4, 8), (1100, 4, 2, 8)])
def test_excluded_experts(E, groups, kept, k, score, dtype):
    each = E // groups
    l = _logits(7, E, dtype, E)
    l[0] = -math.inf                               # nothing left
    l[1, 1:] = -math.inf                           # one expert left
    l[2, each:2 * each] = -math.inf                # a group is out
    l[3, ::2] = -math.inf
    l[4, :each - 1] = -math.inf                    # a group of one expert left
    l[5, :E - k + 1] = -math.inf                   # fewer than topk in all
    bias = -2.0 * torch.rand((E,), generator=torch.Generator().manual_seed(1))   # keys below those of nobody
    for b in (None, bias):
        for renorm in (False, True):
            ids, probs = _check(l, k, score=score, groups=groups, topk_groups=kept, bias=b, renorm=renorm)
            assert bool((probs[0] == 0).all())
            _check_grad(l, ids.cpu(), score=score, renorm=renorm)


def test_scores_too_small_for_fp32_keep_their_ratios():
    l = torch.full((2, 32), -1000.0)
    l[0, 3], l[0, 17], l[1] = -990.0, -991.0, -200.0 - torch.arange(32) * 0.5
    ids = torch.tensor([[3, 17, 0], [0, 1, 2]])
    want, p, ep = ref.gate_grouped(l[1:], 3)
    got = pgg.moe_gate_grouped(l.to(DEV), 3)
    assert torch.equal(got[0].cpu()[1:], want) and got[0][0].tolist() == [0, 1, 2]   # keys of 0 in row 0
    ops_ref.assert_within(got[1][1:], p, ep)
    _check_grad(l, ids)


def test_large_values_and_nan():
    l = _logits(4, 64, "f32", 5)
    l[0, 7] = math.nan
    l[1, 9] = math.inf
    l[2] *= 1e30
    ids, probs = pgg.moe_gate_grouped(l.to(DEV), 4, groups=8, topk_groups=4)
    torch.cuda.synchronize()
    assert ids[0, 0] == 7 and bool(probs[0].isnan().all())
    assert probs[1].isfinite().all() and 9 in ids[1].tolist()
    want, p, ep = ref.gate_grouped(l[2:], 4, groups=8, topk_groups=4)
    assert torch.equal(ids[2:].cpu(), want)
    bias = torch.zeros(64)
    bias[5], bias[6] = math.inf, -math.inf
    got = pgg.moe_gate_grouped(l[3:].to(DEV), 64, bias=bias.to(DEV))[0][0].tolist()
    assert got[0] == 5 and got[-1] == 6 and sorted(got) == list(range(64))


def test_keys_closer_than_fp32():
    # scores that differ by less than 2^-24 of 1, in either order of the index
    E, gen = 64, torch.Generator().manual_seed(2)
    l = torch.full((40, E), -3.0)
    bias = torch.full((E,), 0.25)
    for t in range(40):
        a, b = torch.randperm(E, generator=gen)[:2].tolist()
        l[t, a], l[t, b] = 9.0 + 2.0 ** -17 * (t % 3), 9.0 + 2.0 ** -17
    _check(l, 2, bias=bias, groups=8, topk_groups=2)


def test_gradient_against_differences():
    E, k = 24, 5
    l = _logits(3, E, "f32", 11)
    for score in ("sigmoid", "softmax"):
        for renorm in (False, True):
            ids = pgg.moe_gate_grouped(l.to(DEV), k, score=score, groups=4, topk_groups=3, renorm=renorm, scale=1.5)[0]
            gp = torch.randn((3, k), generator=torch.Generator().manual_seed(4))
            got = pgg.moe_gate_grouped_grad(l.to(DEV), ids, gp.to(DEV), score=score, renorm=renorm, scale=1.5).cpu()

            def f(x):   # the weights of the same experts
                s = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, dim=1)
                w = s.gather(1, ids.cpu())
                return ((w / w.sum(dim=1, keepdim=True) if renorm else w) * 1.5 * gp.double()).sum(dim=1)

            h, x = 1e-5, l.double()
            for e in range(E):
                step = torch.zeros_like(x)
                step[:, e] = h
                num = (f(x + step) - f(x - step)) / (2 * h)
                # the difference's own error h^2 / 6 |f'''| is far below fp32's
                assert bool(((got[:, e].double() - num).abs() <= 1e-6 * (1 + gp.abs().sum())).all())


def test_ids_outside_select_nothing():
    l, ids = _logits(2, 16, "f32", 1), torch.tensor([[3, -1, 5], [16, 2, 1 << 40]])
    gp = torch.ones((2, 3))
    got = pgg.moe_gate_grouped_grad(l.to(DEV), ids.to(DEV), gp.to(DEV), renorm=False).cpu()
    s = torch.sigmoid(l)
    want = torch.zeros((2, 16))
    for t, e in ((0, 3), (0, 5), (1, 2)):
        want[t, e] = s[t, e] * (1 - s[t, e])
    assert torch.allclose(got, want, rtol=1e-5, atol=0)


def test_refusals():
    l = torch.zeros((4, 16), device=DEV)
    for bad in (dict(topk=0), dict(topk=17), dict(topk=5, groups=4, topk_groups=1), dict(topk=2, groups=3),
                dict(topk=2, score="relu"), dict(topk=2, groups=4, topk_groups=5), dict(topk=2, groups=0),
                dict(topk=2, bias=torch.zeros(15, device=DEV)), dict(topk=2, bias=torch.zeros(16)),
                dict(topk=2, bias=torch.zeros(16, device=DEV).half())):
        with pytest.raises(pgg.PggError):
            pgg.moe_gate_grouped(l, **bad)
    for bad in (l.t(), l.double(), l.cpu(), l[0]):
        with pytest.raises(pgg.PggError):
            pgg.moe_gate_grouped(bad, 2)
    ids, gp = torch.zeros((4, 2), dtype=torch.int64, device=DEV), torch.zeros((4, 2), device=DEV)
    for a, b in ((ids.int(), gp), (ids, gp[:3]), (ids[:, 0], gp), (ids, gp.half())):
        with pytest.raises(pgg.PggError):
            pgg.moe_gate_grouped_grad(l, a, b)
    with pytest.raises(pgg.PggError):
        pgg.moe_gate_grouped_grad(l, ids, gp, out=torch.zeros((4, 15), device=DEV))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,kept,k", [(16, 4, 2, 5), (60, 4, 3, 8), (256, 8, 4, 8), (1100, 4, 2, 8)])
def test_biases_without_bounds(E, groups, kept, k, score):
    each = E // groups
    for low in (-math.inf, float(torch.finfo(torch.float32).min)):
        bias = torch.randn((E,), generator=torch.Generator().manual_seed(E)) * 0.1
        bias[::3] = low                        # experts kept back here and there
        bias[each:2 * each] = low              # a whole group
        bias[2 * each:3 * each - 1] = low      # all but one of a group
        bias[3 * each - 1] = 0.05
        _check(_logits(9, E, "f32", 3), k, score=score, groups=groups, topk_groups=kept, bias=bias)
    _check(_logits(3, E, "f32", 4), k, score=score, groups=groups, topk_groups=kept, bias=torch.full((E,), -math.inf))
    high = torch.zeros(E)
    high[each + 1] = math.inf
    ids, _ = _check(_logits(3, E, "f32", 5), k, score=score, groups=groups, topk_groups=kept, bias=high)
    assert bool((ids[:, 0] == each + 1).all())
