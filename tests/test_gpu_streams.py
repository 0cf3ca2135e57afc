"""Calls on an explicit stream while the current stream still uses memory that
it has freed (needs an MI355X)."""
import pytest
import torch

import permute_grouped_gemm_amd as pgg
import synth
from gpu_util import upload

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _calls():
    """{name: call(stream)}, each with inputs of its own."""
    case = synth.make_case(64, 2, 4, 128, 64, "bf16", seed=3)
    gy, w, eri, gl = upload(case)
    b, k = case.batch, case.topk
    x = torch.randn((b, w.shape[1]), device=DEV).bfloat16()
    ids = torch.randint(0, 4, (b, k), device=DEV)
    ids[:, 1] = (ids[:, 0] + 1) % 4
    probs = torch.rand((b, k), device=DEV).bfloat16()
    logits = torch.randn((b, 16), device=DEV)
    gate = pgg.moe_gate(logits, 2)
    gp = torch.randn((b, 2), device=DEV)
    w1, w2 = (torch.randn(s, device=DEV).bfloat16() for s in ((4, x.shape[1], 64), (4, 32, gy.shape[1])))
    gu = torch.randn((b * k, 64), device=DEV).bfloat16()
    base = torch.randn((x.shape[1], 48), device=DEV).bfloat16()
    a, bb = (torch.randn(s, device=DEV).bfloat16() for s in ((3, 4, x.shape[1]), (3, 4, 48)))
    own, sc = torch.randint(-1, 3, (b,), device=DEV), torch.ones(3, device=DEV)
    grad = torch.randn((b, gy.shape[1]), device=DEV).bfloat16()
    return {
        "dx": lambda s: pgg.moe_dx(gy, w, eri, gl, b, k, case.row_idx_type, stream=s),
        "fwd": lambda s: pgg.moe_fwd(x, w, eri, gl, k, case.row_idx_type, stream=s),
        "dw": lambda s: pgg.moe_dw(x, gy, eri, gl, k, case.row_idx_type, stream=s),
        "routing": lambda s: pgg.moe_routing(ids, 4, x, stream=s),
        "unpermute": lambda s: pgg.moe_unpermute(gy, eri, b, k, case.row_idx_type, probs, stream=s),
        "unpermute_grad": lambda s: pgg.moe_unpermute_grad(grad, eri, b, k, case.row_idx_type, gy, probs, stream=s),
        "gate": lambda s: pgg.moe_gate(logits, 2, stream=s),
        "gate_grad": lambda s: pgg.moe_gate_grad(logits, gate[2], gate[0], gp, stream=s),
        "glu": lambda s: pgg.moe_glu(x, w1, eri, gl, k, case.row_idx_type, save_gate_up=True, stream=s),
        "glu_grad": lambda s: pgg.moe_glu_grad(gy, w2, gu, gl, stream=s),
        "lora": lambda s: pgg.lora_fwd(x, base, a, bb, own, sc, stream=s),
    }


NAMES = ["dx", "fwd", "dw", "routing", "unpermute", "unpermute_grad", "gate", "gate_grad", "glu", "glu_grad", "lora"]


def _tuple(r):
    return r if isinstance(r, tuple) else (r,)


@pytest.mark.parametrize("name", NAMES)
def test_a_side_stream_takes_no_memory_that_the_current_one_may_use(name, monkeypatch):
    call = _calls()[name]
    want = [t.clone() for t in _tuple(call(None))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    made = []
    empty = torch.empty

    def recording(*args, **kwargs):
        t = empty(*args, **kwargs)
        if t.is_cuda:
            made.append(t.data_ptr())
        return t

    # blocks that the current stream has freed and still writes to, of every size that the call could take
    freed = [empty(n, dtype=torch.uint8, device=DEV) for n in [1 << s for s in range(9, 22)] * 3]
    torch.cuda._sleep(2000000)
    for t in freed:
        t.fill_(255)
    ranges = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in freed]
    del t, freed
    monkeypatch.setattr(torch, "empty", recording)
    got = _tuple(call(side))          # its inputs were ready before the work above was queued
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert made and not any(lo <= p < hi for p in made for lo, hi in ranges)
    on_side = [(s["address"], s["address"] + s["total_size"]) for s in torch.cuda.memory_snapshot()
               if s["stream"] == side.cuda_stream]
    assert all(any(lo <= p < hi for lo, hi in on_side) for p in made)
    for u, v in zip(got, want):
        assert torch.equal(u, v)


def test_a_freed_result_waits_for_the_current_stream():
    # a result made on `side`, read by work queued on the current stream and freed:
    # the next call on `side` must not write over it
    logits = torch.randn((4096, 64), device=DEV)
    ids = pgg.moe_gate(logits, 8)[0]
    want = ids.clone()
    other = -logits
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mine = pgg.moe_gate(logits, 8, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(2000000)
    copy = mine.clone()
    del mine
    again = pgg.moe_gate(other, 8, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
    assert torch.equal(again[0], pgg.moe_gate(other, 8)[0])
