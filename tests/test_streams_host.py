"""What a call on an explicit stream allocates comes from that stream's memory
(host only: torch's allocator and streams are replaced by records)."""
import ast
import contextlib

import torch

import permute_grouped_gemm_amd as pgg


class _Tensor:
    def __init__(self, stream):
        self.allocated_on, self.recorded = stream, []

    def record_stream(self, stream):
        self.recorded.append(stream)


def test_buffers_come_from_the_streams_own_memory(monkeypatch):
    active = ["current"]

    @contextlib.contextmanager
    def on(stream):
        active.append(stream)
        yield
        active.pop()

    monkeypatch.setattr(torch, "empty", lambda *a, **k: _Tensor(active[-1]))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: active[-1])
    t = pgg._fresh((4,), torch.float32, "cuda:0", "side")
    assert t.allocated_on == "side" and t.recorded == ["current"]
    assert pgg._fresh((4,), torch.float32, "cuda:0", None).allocated_on == "current"


def test_no_other_place_allocates_on_the_gpu():
    with open(pgg.__file__) as f:
        tree = ast.parse(f.read())
    for fn in ast.walk(tree):
        if not isinstance(fn, ast.FunctionDef) or fn.name == "_fresh":
            continue
        for call in ast.walk(fn):
            if isinstance(call, ast.Call) and isinstance(call.func, ast.Attribute) \
                    and call.func.attr in ("empty", "zeros", "ones", "full", "empty_like", "zeros_like"):
                assert not any(k.arg == "device" for k in call.keywords), (fn.name, call.lineno)
