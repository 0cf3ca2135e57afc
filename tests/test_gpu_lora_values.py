"""Precision and non-finite values of the adapters' products, at the tokens
and widths that take each of their kernels."""
import math

import pytest
import torch

import ops_ref as ref
import permute_grouped_gemm_amd as pgg

pytestmark = pytest.mark.gpu
DEV = "cuda"

# tokens, columns: split with the sums in fp32; tiles of 128 rows (columns at any
# address); the 256-row tiles
KERNELS = [(20, 136), (300, 35), (300, 136), (2300, 136)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,N", KERNELS)
def test_inner_products_keep_sixteen_bits(T, N, dtype):
    # y = z b - (z b rounded to the type), with z and b around 1: what is left is
    # 2^-9 of z b or less, so its own rounding hides nothing.  Every sum has one
    # product in it but for the last, z b + (-...): exact up to the parts of z,
    # 2^-16, and a few fp32 additions.
    dt, K = ref.DTYPES[dtype], 72
    gen = torch.Generator().manual_seed(T + N)
    scales = 1.0 + torch.rand(4, generator=gen)
    scales[0] = 1.0 + 2.0 ** -7 - 2.0 ** -23          # just below a step of bf16
    scales[1] = 1.0 + 3 * 2.0 ** -8 - 2.0 ** -20
    b = (1.0 + torch.rand((4, 1, N), generator=gen)).to(dt)
    b[0, 0, ::2] = 1.0 + 2.0 ** -7 - 2.0 ** -10 if dtype == "f16" else 1.0 + 2.0 ** -7
    a = torch.zeros((4, 1, K)).to(dt)
    a[:, 0, 1] = 1.0
    ids = torch.arange(T) // 9 % 4
    x, w = torch.zeros((T, K)).to(dt), torch.zeros((K, N)).to(dt)
    x[:, 1] = 1.0
    zb = scales.double()[:, None] * b[:, 0].double()   # of the four adapters
    for p in range(4):
        x[ids == p, 4 + p] = 1.0
        w[4 + p] = -zb[p].to(dt)
    y = pgg.lora_fwd(*[t.to(DEV) for t in (x, w, a, b, ids, scales)])
    want = (zb + w[4:8].double())[ids]
    ref.assert_within(y, want, ref.rounded(want, zb[ids] * (2.0 ** -16 + 2.0 ** -20), dt))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,N", KERNELS)
def test_infinite_values_give_the_infinities_of_their_product(T, N, dtype):
    # infinities in B against z of few and of many bits, in A (z infinite) against B
    # of few and of many bits: y is infinite with the product's sign, as in 64 bits,
    # and NaN only where the 64-bit form is
    dt, K = ref.DTYPES[dtype], 72
    gen = torch.Generator().manual_seed(N)
    x, w = torch.zeros((T, K)).to(dt), (torch.randn((K, N), generator=gen) * 0.1).to(dt)
    x[:, 1] = 1.0
    x[::2, 2] = -1.0                                   # z changes sign
    a = torch.zeros((5, 2, K)).to(dt)
    a[:, 0, 1], a[:, 0, 2], a[:, 1, 1] = 1.0, 2.0, 0.5
    b = (1.0 + torch.rand((5, 2, N), generator=gen)).to(dt)
    b[0, 0, 1], b[0, 1, 2], b[0, 0, 3] = math.inf, -math.inf, math.nan
    b[1, 0, 1], b[1, 1, 2] = -math.inf, math.inf       # z of 24 bits
    b[2, 0, ::3], b[2, 0, 1::3] = 1.0, -2.0
    b[3, 0, ::3], b[3, 0, 1] = 0.0, -0.0
    a[2, 0, 1] = a[3, 0, 1] = math.inf                 # z infinite
    scales = torch.tensor([1.0, 1.2345678, 1.0, 1.0, 0.75])
    ids = torch.arange(T) // 5 % 6 - 1
    y = pgg.lora_fwd(*[t.to(DEV) for t in (x, w, a, b, ids, scales)]).cpu().double()
    want = x.double() @ w.double()
    for t in range(T):
        if ids[t] >= 0:
            z = scales[ids[t]].double() * (a[ids[t]].double() * x[t].double()).sum(dim=1)
            want[t] += (z[:, None] * b[ids[t]].double()).sum(dim=0)
    assert torch.equal(y.isnan(), want.isnan())
    assert torch.equal(y.isinf(), want.isinf())
    at = want.isinf()
    assert at.any() and torch.equal(y[at], want[at])
    # the others: sums of terms below 8 in all, far less than the final rounding's 2^-8
    ref.assert_within(y[~at], want[~at], 2.0 ** -8 * want[~at].abs() + 8 * 2.0 ** -14)
