"""The combination and its gradient at the ends of fp32's range: sums and streams
whose norms' factors cubed are no fp32 numbers, and rows of zeros under a small eps
(needs an MI355X)."""
import pytest
import torch

import block_ref as ref
import ops_ref
from test_gpu_combine import _inputs, _run

pytestmark = pytest.mark.gpu
ORDER = ("permuted", "probs", "residual", "gate", "post", "next")


def _compare(s, eps, alpha=0.7, rit=1):
    plain = {n: s[n] for n in ("permuted", "eri", "probs", "residual", "post", "gate", "nxt")}
    for grad in (False, True):
        extra = dict(grad_out=s["grad_out"], grad_normed=s["grad_normed"]) if grad else {}
        want = ref.combine(**plain, row_idx_type=rit, alpha=alpha, eps=eps, **extra)
        for name, t in zip(ORDER if grad else ("out", "normed"), _run(s, rit, alpha, eps, grad)):
            if t is not None:
                near = want[name]
                ops_ref.assert_within(t, near.v, ops_ref.rounded(near.v, near.e, t.dtype), f"{name} grad={grad}")


# rows of one and of several pieces, with ends that overlap, fewer than 8 elements,
# more than 8192, and more slots than stay in registers
SHAPES = [(5, 3, 136), (3, 2, 7), (6, 2, 2039), (2, 9, 264), (2, 3, 8200)]


def _sized(shape, dtype, post, gate, nxt, rms):
    """Inputs whose sum and stream have the size rms, and grad_out as large as what
    comes back through the norm of the stream, 1 / rms."""
    s = _inputs(*shape, dtype, post, gate, nxt, seed=shape[2])
    for n in ("permuted", "residual"):
        s[n] = s[n] * rms
    if nxt:
        s["grad_out"] = s["grad_out"] / rms
    return s


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("rms,eps", [(1e10, 1e-6), (1e15, 1e-6), (1e17, 1e-5), (1e-14, 0.0), (1e-12, 1e-30)])
def test_size_of_the_sum(rms, eps, shape, dtype):
    _compare(_sized(shape, dtype, True, True, False, rms), eps)
    _compare(_sized(shape, dtype, True, False, False, rms), eps, rit=0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("rms,eps", [(1e10, 1e-6), (1e15, 1e-6), (1e17, 1e-5), (1e-14, 0.0), (1e-12, 1e-30)])
def test_size_of_the_stream(rms, eps, shape, dtype):
    _compare(_sized(shape, dtype, False, False, True, rms), eps)
    _compare(_sized(shape, dtype, False, True, True, rms), eps, rit=0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("rms,eps", [(1e15, 1e-6), (1e-14, 0.0)])
def test_size_of_both(rms, eps, shape, dtype):
    _compare(_sized(shape, dtype, True, True, True, rms), eps)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("post,nxt,eps", [(True, False, 1e-30), (True, False, 1e-36), (False, True, 1e-30),
                                          (False, True, 1e-36), (True, True, 1e-30)])
def test_rows_of_zeros_under_a_small_eps(post, nxt, eps, shape, dtype):
    # (1 / sqrt(eps) twice, with both norms, is 1e30)
    s = _inputs(*shape, dtype, post, True, nxt, seed=1)
    at = ref.slots(s["eri"], shape[0], shape[1], 1)
    s["permuted"][at[0]] = 0
    s["residual"][0] = 0
    _compare(s, eps)
