"""The router's gate and its gradient against their 64-bit forms."""
import math

import pytest
import torch

import ops_ref as ref
import permute_grouped_gemm_amd as pgg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _logits(T, E, dtype, seed, std=1.5):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=gen) * std).to(ref.DTYPES[dtype])


def _check(logits, topk, bias=None, renorm=False, scale=1.0):
    ids, probs, lse = pgg.moe_gate(logits.to(DEV), topk, bias=None if bias is None else bias.to(DEV),
                                   renorm=renorm, scale=scale)
    torch.cuda.synchronize()
    want, p, ep, l, el = ref.gate(logits, topk, bias, renorm, scale)
    assert ids.dtype == torch.int64 and probs.dtype == lse.dtype == torch.float32
    assert torch.equal(ids.cpu(), want)
    ref.assert_within(probs, p, ep, "probs")
    ref.assert_within(lse, l, el, "lse")
    return ids, probs, lse


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 16, 8), (3, 17, 1), (5, 60, 8), (64, 64, 6), (33, 65, 4),
                                   (7, 129, 8), (9, 256, 8), (6, 257, 3), (5, 513, 16), (3, 1025, 8), (2, 8192, 9)])
def test_gate(T, E, k, dtype):
    for renorm in (False, True):
        _check(_logits(T, E, dtype, 7 * T + E), k, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("E,k", [(4, 4), (16, 16), (64, 64), (70, 64), (700, 40), (1500, 64)])
def test_gate_many_picks(E, k):
    _check(_logits(5, E, "f32", E), k, renorm=True)


@pytest.mark.parametrize("E", [8, 60, 300, 2000])
def test_equal_logits_go_to_the_lowest_index(E):
    l = torch.zeros((4, E))
    l[1] = -0.0
    l[1, ::2] = 0.0                              # 0 and -0 are equal
    l[2] = torch.arange(E) % 3
    l[3] = torch.finfo(torch.float32).min
    for dtype in (torch.float32, torch.bfloat16):
        _check(l.to(dtype), min(E, 8))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("E", [8, 60, 500, 1100])
def test_excluded_experts_and_rows_with_nothing_left(E, dtype):
    l = _logits(6, E, dtype, 3 + E)
    l[0] = -math.inf                             # nothing left
    l[1, 1:] = -math.inf                         # one expert left
    l[2, : E - 2] = -math.inf
    l[3, ::2] = -math.inf
    l[4] = torch.finfo(l.dtype).min              # a mask of the lowest value leaves a uniform row
    for renorm in (False, True):
        ids, probs, lse = _check(l, min(E, 6), renorm=renorm)
        assert ids[0].tolist() == list(range(min(E, 6))) and not probs[0].any() and lse[0] == -math.inf
        assert not probs[1, 1:].any() and probs[1, 0] == 1


@pytest.mark.parametrize("E", [12, 200, 1200])
def test_infinities_and_nan_stay_in_their_rows(E):
    l = _logits(5, E, "f32", E)
    l[1, 3] = math.inf
    l[2, 5] = math.nan
    l[3, 2] = l[3, 7] = math.nan
    ids, probs, lse = pgg.moe_gate(l.to(DEV), 4)
    clean = pgg.moe_gate(l[[0, 4]].to(DEV), 4)
    assert torch.equal(ids[[0, 4]], clean[0]) and torch.equal(probs[[0, 4]], clean[1])
    assert torch.equal(lse[[0, 4]], clean[2])
    assert ids[1, 0] == 3 and ids[2, 0] == 5 and ids[3, :2].tolist() == [2, 7]
    assert lse[1:4].isnan().logical_or(lse[1:4] == math.inf).all() and probs[1:4, 0].isnan().all()


def test_bias_enters_the_choice_only():
    l = _logits(40, 60, "bf16", 5)
    bias = torch.randn(60, generator=torch.Generator().manual_seed(1))
    bias[7] = -math.inf
    bias[11] = 100.0
    ids, _, _ = _check(l, 8, bias=bias)
    assert (ids[:, 0] == 11).all() and not (ids == 7).any()


def _grad_case(T, E, k, dtype, seed, masked=False):
    l = _logits(T, E, dtype, seed)
    if masked:
        l[:, ::5] = -math.inf
        l[0] = -math.inf
    gen = torch.Generator().manual_seed(seed + 1)
    ids, _, _ = pgg.moe_gate(l.to(DEV), k)
    return l, ids, torch.randn((T, k), generator=gen), torch.randn(T, generator=gen)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 16, 8), (5, 60, 8), (33, 65, 4), (7, 129, 1), (9, 256, 8),
                                   (6, 257, 3), (3, 1025, 8), (2, 8192, 9), (4, 100, 64)])
def test_gate_grad(T, E, k, dtype):
    for masked in (False, True):
        l, ids, gp, gl = _grad_case(T, E, k, dtype, T + E, masked)
        for renorm, with_lse in ((False, False), (False, True), (True, False), (True, True)):
            lse = pgg.moe_gate(l.to(DEV), k)[2]
            got = pgg.moe_gate_grad(l.to(DEV), lse, ids, gp.to(DEV), grad_lse=gl.to(DEV) if with_lse else None,
                                    renorm=renorm, scale=2.5)
            want, err = ref.gate_grad(l, ids, gp, gl if with_lse else None, renorm, 2.5)
            assert got.dtype == l.dtype
            ref.assert_within(got, want, ref.rounded(want, err, l.dtype), f"grad {renorm} {with_lse} {masked}")


@pytest.mark.parametrize("renorm", [False, True])
def test_gate_grad_against_differences(renorm):
    # central differences of the 64-bit forward; their error: step^2 / 6 times the
    # third derivative (at most about 6 for softmax) times the sum of weights, and
    # the forward's rounding over the step
    l, ids, gp, gl = _grad_case(3, 12, 4, "f32", 21)
    lse = pgg.moe_gate(l.to(DEV), 4)[2]
    got = pgg.moe_gate_grad(l.to(DEV), lse, ids, gp.to(DEV), grad_lse=gl.to(DEV), renorm=renorm, scale=1.5).cpu().double()
    ids = ids.cpu()

    def value(x):
        over = x.gather(1, ids)
        p = torch.softmax(over, 1) if renorm else torch.softmax(x, 1).gather(1, ids)
        return (1.5 * p * gp.double()).sum() + (torch.logsumexp(x, 1) * gl.double()).sum()

    step = 1e-4
    x = l.double()
    for t in range(3):
        for e in range(12):
            hi, lo = x.clone(), x.clone()
            hi[t, e] += step
            lo[t, e] -= step
            diff = (value(hi) - value(lo)) / (2 * step)
            assert abs(got[t, e] - diff) <= 100 * step ** 2 + 1e-14 / step + 64 * 2.0 ** -22, (t, e)


def test_ids_outside_the_experts_select_nothing():
    l, ids, gp, _ = _grad_case(4, 10, 3, "f32", 9)
    lse = pgg.moe_gate(l.to(DEV), 3)[2]
    bad = ids.clone()
    bad[:, 1] = torch.tensor([-1, 10, 1 << 40, -(1 << 40)], device=DEV)
    keep = torch.stack([ids[:, 0], ids[:, 2]], 1).contiguous()
    for renorm in (False, True):
        got = pgg.moe_gate_grad(l.to(DEV), lse, bad, gp.to(DEV), renorm=renorm)
        want = pgg.moe_gate_grad(l.to(DEV), lse, keep, gp[:, [0, 2]].contiguous().to(DEV), renorm=renorm)
        assert torch.equal(got, want)


def test_gate_is_repeatable_and_follows_its_stream():
    l = _logits(500, 60, "bf16", 2).to(DEV)
    first = pgg.moe_gate(l, 8, renorm=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = pgg.moe_gate(l, 8, renorm=True, stream=side)
    side.synchronize()
    for u, v in zip(first, again):
        assert torch.equal(u, v)


def test_gate_captures_into_a_graph():
    l = _logits(300, 60, "f16", 2).to(DEV)
    graph = torch.cuda.CUDAGraph()
    gp = torch.randn((300, 8), device=DEV)
    want = pgg.moe_gate(l, 8)
    want_grad = pgg.moe_gate_grad(l, want[2], want[0], gp)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = pgg.moe_gate(l, 8)
        grad = pgg.moe_gate_grad(l, got[2], got[0], gp)
    for _ in range(3):
        for t in (*got, grad):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want)) and torch.equal(grad, want_grad)


def test_gate_refusals():
    l = torch.zeros((4, 8), device=DEV)
    for call in (lambda: pgg.moe_gate(l, 0), lambda: pgg.moe_gate(l, 9), lambda: pgg.moe_gate(l.cpu(), 2),
                 lambda: pgg.moe_gate(l.t(), 2), lambda: pgg.moe_gate(l.double(), 2), lambda: pgg.moe_gate(l[0], 1),
                 lambda: pgg.moe_gate(l[:0], 1), lambda: pgg.moe_gate(l, 2, bias=torch.zeros(7, device=DEV)),
                 lambda: pgg.moe_gate(l, 2, bias=torch.zeros(8, device=DEV, dtype=torch.float16)),
                 lambda: pgg.moe_gate(l, 2, bias=torch.zeros(8))):
        with pytest.raises(pgg.PggError) as e:
            call()
        assert e.value.status == pgg.ERR_INVALID_ARG
    for shape, k in (((2, 8193), 2), ((2, 100), 65)):
        with pytest.raises(pgg.PggError) as e:
            pgg.moe_gate(torch.zeros(shape, device=DEV), k)
        assert e.value.status == pgg.ERR_UNSUPPORTED
    ids, probs, lse = pgg.moe_gate(l, 2)
    for call in (lambda: pgg.moe_gate_grad(l, lse[:3], ids, probs), lambda: pgg.moe_gate_grad(l, lse, ids.int(), probs),
                 lambda: pgg.moe_gate_grad(l, lse, ids, probs.half()), lambda: pgg.moe_gate_grad(l, lse, ids[:, :1], probs),
                 lambda: pgg.moe_gate_grad(l, lse, ids, probs, grad_lse=lse[:2]),
                 lambda: pgg.moe_gate_grad(l, lse, ids, probs, out=torch.zeros((4, 8)))):
        with pytest.raises(pgg.PggError):
            call()
