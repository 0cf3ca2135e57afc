"""The grouped gate, the 4-bit products and the combination as they are used:
together, on a stream of the caller's, captured into a graph, at offsets past
2^31, and the example's steps (needs an MI355X)."""
import importlib.util
import os

import pytest
import torch

import block_ref as ref
import ops_ref
import permute_grouped_gemm_amd as pgg

pytestmark = pytest.mark.gpu
DEV = "cuda"
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")


def _example():
    spec = importlib.util.spec_from_file_location("moe_block", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


@pytest.mark.parametrize("sizes", [dict(), dict(tokens=1, experts=4, topk=2, groups=2, topk_groups=1),
                                   dict(tokens=77, hidden=200, ffn=72, experts=15, topk=5, groups=5, topk_groups=3,
                                        group_size=32)], ids=["default", "one token", "odd"])
def test_moe_block_example(sizes):
    # The values pass through up to five bf16 roundings of 2^-9 relative each (gate_up,
    # h, y, its gradient, the result); the router's own product rounds logits of size
    # up to 4 to 8 bits, 4 * 2^-8 of a weight, and so do the gradients behind it.  Norms
    # of the sum and of the stream pass errors on at most once more each.
    for name, error in _example().main(**sizes).items():
        assert error <= (12 if name in ("grad router", "grad x") else 8) * 2.0 ** -8, (name, error)


def _serving(tokens, seed=0):
    """Inputs of a serving step and the step itself (outputs and workspaces given)."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    E, k, H, F, gs = 16, 4, 256, 128, 64
    rand = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    codes = lambda *s: torch.randint(0, 16, s, generator=gen, device=DEV, dtype=torch.uint8)  # noqa: E731
    scales = lambda *s: ((0.5 + torch.rand(s, generator=gen, device=DEV)) * 0.02).bfloat16()  # noqa: E731
    w_in = pgg.w4_pack(codes(E, H, 2 * F), scales(E, H // gs, 2 * F), gs, gated=True)
    w_out = pgg.w4_pack(codes(E, F, H), scales(E, F // gs, H), gs)
    post, nxt = (1 + 0.1 * rand(H)).bfloat16(), (1 + 0.1 * rand(H)).bfloat16()
    inputs = dict(x=rand(tokens, H).bfloat16(), logits=rand(tokens, E).bfloat16(), residual=rand(tokens, H).bfloat16())

    def step(stream=None):
        ids, probs = pgg.moe_gate_grouped(inputs["logits"], k, groups=4, topk_groups=2, scale=2.0, stream=stream)
        counts, gather, scatter, _ = pgg.moe_routing(ids, E, stream=stream)
        h = pgg.moe_glu_w4(inputs["x"], w_in, gather, counts, k, stream=stream)
        y = pgg.moe_fwd_w4(h, w_out, None, counts, stream=stream)
        out, normed = pgg.moe_combine(y, scatter, probs, inputs["residual"], row_idx_type=1, post_weight=post,
                                      next_weight=nxt, stream=stream)
        grads = pgg.moe_combine_grad(inputs["residual"], y, scatter, probs, inputs["residual"],
                                     grad_normed=inputs["x"], row_idx_type=1, post_weight=post, next_weight=nxt,
                                     stream=stream)
        glogits = pgg.moe_gate_grouped_grad(inputs["logits"], ids, grads[1], scale=2.0, stream=stream)
        return [ids, probs, h, y, out, normed, glogits] + [g for g in grads if g is not None]

    return inputs, step


@pytest.mark.parametrize("tokens", [1, 16, 300, 2000])
def test_graph_replays_match_eager(tokens):
    inputs, step = _serving(tokens)
    eager = [t.clone() for t in step()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        results = step()
    other = torch.randn((256, 256), device=DEV)
    for _ in range(3):
        for t in results:
            t.zero_()
        float((other @ other).sum())        # eager work and a synchronisation
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(results, eager):
            assert torch.equal(a, b)
    # a replay reads the inputs anew
    fresh, _ = _serving(tokens, seed=1)
    for n in inputs:
        inputs[n].copy_(fresh[n])
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(results, [t.clone() for t in step()]):
        assert torch.equal(a, b)


def test_two_graphs_with_workspaces_of_their_own():
    steps = [_serving(40, seed=s)[1] for s in (0, 1)]
    eager = [[t.clone() for t in s()] for s in steps]
    torch.cuda.synchronize()
    graphs, results = [torch.cuda.CUDAGraph() for _ in steps], []
    for g, s in zip(graphs, steps):
        with torch.cuda.graph(g):
            results.append(s())
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for i in order:
            graphs[i].replay()
            torch.cuda.synchronize()
            for a, b in zip(results[i], eager[i]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("tokens", [16, 700])
def test_on_a_stream_of_the_callers(tokens):
    _, step = _serving(tokens)
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_two_calls_at_once():
    # the same weights and inputs on two streams, each call with buffers of its own
    _, step = _serving(300)
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [step(stream=s) for s in streams]
        torch.cuda.synchronize()
        for result in got:
            for a, b in zip(result, want):
                assert torch.equal(a, b)


def test_rows_past_2_31_elements():
    # permuted and its gradient of more than 2^31 elements: tokens at both ends
    batch, topk, H = 32800, 8, 8192
    assert batch * topk * H > 1 << 31
    permuted = torch.empty((batch * topk, H), dtype=torch.bfloat16, device=DEV).normal_(0, 0.5)
    eri = torch.arange(batch * topk, device=DEV).flip(0).contiguous()
    gen = torch.Generator(device=DEV).manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    probs, residual, grad = torch.rand((batch, topk), device=DEV), rand(batch, H).bfloat16(), rand(batch, H).bfloat16()
    post = (1 + 0.1 * rand(H)).bfloat16()
    out = pgg.moe_combine(permuted, eri, probs, residual, row_idx_type=1, post_weight=post)
    grads = pgg.moe_combine_grad(grad, permuted, eri, probs, residual, row_idx_type=1, post_weight=post)
    at = [0, 1, batch // 2, batch - 2, batch - 1]
    rows = eri.reshape(batch, topk)[at].cpu()
    mine = dict(permuted=permuted[rows.reshape(-1).to(DEV)], eri=torch.arange(len(at) * topk), probs=probs[at],
                residual=residual[at], row_idx_type=1, post=post)
    want = ref.combine(**mine)["out"]
    ops_ref.assert_within(out[at], want.v, ops_ref.rounded(want.v, want.e, torch.bfloat16))
    want = ref.combine(**mine, grad_out=grad[at])
    ops_ref.assert_within(grads[0][rows.reshape(-1).to(DEV)], want["permuted"].v,
                          ops_ref.rounded(want["permuted"].v, want["permuted"].e, torch.bfloat16))
    ops_ref.assert_within(grads[1][at], want["probs"].v, want["probs"].e)


def test_w4_weights_past_2_31_codes():
    # more than 2^32 codes in all (2^31 bytes packed): the first, a middle and the last expert
    G, K, N, gs = 70, 8192, 8192, 128
    assert G * K * N // 2 > 1 << 31
    codes = torch.randint(0, 16, (G, K, N), device=DEV, dtype=torch.uint8)
    scales = ((0.5 + torch.rand((G, K // gs, N), device=DEV)) * 0.002).bfloat16()
    weight = pgg.w4_pack(codes, scales, gs)
    gl = torch.zeros(G, dtype=torch.int64, device=DEV)
    gl[0], gl[35], gl[G - 1] = 3, 2, 4
    for many in (1, 40):     # few rows and tiles of many
        counts = gl * many
        M = int(counts.sum())
        x = torch.randn((M, K), device=DEV).bfloat16()
        y = pgg.moe_fwd_w4(x, weight, None, counts)
        cols = [0, 1, 63, 64, 4000, N - 65, N - 2, N - 1]
        row = 0
        for g in (0, 35, G - 1):
            n = int(counts[g])
            pick = [row, row + n - 1]
            want, bound = ref.w4_fwd(x[pick].cpu(), codes[g:g + 1][:, :, cols].cpu(), scales[g:g + 1][:, :, cols].cpu(),
                                     None, gs, torch.tensor([2]))
            ops_ref.assert_within(y[pick][:, cols], want, bound, f"expert {g}, {n} rows")
            row += n
    del codes, weight
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M", [130000, 270000])
def test_x_past_2_31_bytes(M):
    # x of a little less than 2^31 bytes, the most for the large tiles' 32-bit offsets,
    # and of more than 2^31 elements
    K, N, gs = 8192, 64, 128
    assert (1 << 31) - (1 << 24) - (1 << 20) < M * K * 2 < 1 << 31 or M * K > 1 << 31
    codes = torch.randint(0, 16, (2, K, N), device=DEV, dtype=torch.uint8)
    scales = ((0.5 + torch.rand((2, K // gs, N), device=DEV)) * 0.002).bfloat16()
    x = torch.empty((M, K), dtype=torch.bfloat16, device=DEV).normal_()
    gl = torch.tensor([M - 7, 7], device=DEV)
    y = pgg.moe_fwd_w4(x, pgg.w4_pack(codes, scales, gs), None, gl)
    for g, pick in ((0, [0, 1, M // 2, M - 9, M - 8]), (1, [M - 7, M - 1])):
        want, bound = ref.w4_fwd(x[pick].cpu(), codes[g:g + 1].cpu(), scales[g:g + 1].cpu(), None, gs,
                                 torch.tensor([len(pick)]))
        ops_ref.assert_within(y[pick], want, bound, f"group {g}")


@pytest.mark.parametrize("batch,H", [(16, 7168), (333, 2039), (40, 64), (3, 16384)])
def test_residual_stream_in_place(batch, H):
    gen = torch.Generator(device=DEV).manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=gen, device=DEV).bfloat16()  # noqa: E731
    permuted, eri = rand(batch * 4, H), torch.randperm(batch * 4, generator=gen, device=DEV)
    probs, residual, post, nxt = torch.rand((batch, 4), device=DEV), rand(batch, H), rand(H), rand(H)
    kw = dict(row_idx_type=1, post_weight=post, next_weight=nxt)
    out, normed = pgg.moe_combine(permuted, eri, probs, residual, **kw)
    again, normed_again = pgg.moe_combine(permuted, eri, probs, residual, out=residual, **kw)
    assert again.data_ptr() == residual.data_ptr()
    assert torch.equal(again, out) and torch.equal(normed_again, normed)


def test_two_graphs_share_a_workspace():
    # replays in any order on one stream: every call writes what it reads of it
    gen = torch.Generator(device=DEV).manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    K, N, gs, calls = 512, 128, 64, []
    w = pgg.w4_pack(torch.randint(0, 16, (300, K, N), generator=gen, device=DEV, dtype=torch.uint8),
                    (0.02 * torch.rand((300, K // gs, N), generator=gen, device=DEV)).bfloat16(), gs)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    for tokens in (40, 500):
        ids = torch.randint(0, 300, (tokens, 4), generator=gen, device=DEV)
        counts, gather, scatter, _ = pgg.moe_routing(ids, 300)
        x, probs, res = rand(tokens, K).bfloat16(), torch.rand((tokens, 4), device=DEV), rand(tokens, N).bfloat16()

        def call(x=x, counts=counts, gather=gather, scatter=scatter, probs=probs, res=res):
            y = pgg.moe_fwd_w4(x, w, gather, counts, 4, workspace=ws)
            out = pgg.moe_combine(y, gather, probs, res, workspace=ws)
            grads = pgg.moe_combine_grad(res, y, gather, probs, res, post_weight=res[0].contiguous(), workspace=ws)
            return [y, out, grads[0], grads[1], grads[4]]

        eager = [t.clone() for t in call()]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results = call()
        calls.append((g, results, eager, call))   # (call holds what the graph reads)
    for order in ((0, 1), (1, 0), (1, 1), (0, 1)):
        for i in order:
            calls[i][0].replay()
        torch.cuda.synchronize()
        for _, results, eager, _ in calls:
            for a, b in zip(results, eager):
                assert torch.equal(a, b)
