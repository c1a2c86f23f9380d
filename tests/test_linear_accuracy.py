"""moe_linear where float arithmetic is tried hardest, gelu's tail below zero and long sums of one sign, and depths that
its indexes do not take."""
import math

import pytest
import torch

import mixture_experts_layer_gate_gb300 as moe
from tests import op_reference as ref
from tests.op_reference import EPS32, TRUNC32
from tests.test_linear import UNSUPPORTED, call
from tests.test_operators import dev, gen, lib  # noqa: F401  (fixtures among them)

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("M", [3, 200, 700])
def test_gelu_keeps_its_bits_below_zero(dev, M):
    """v Phi(v) to a relative bound, in steps of 2^-24.  Phi(-a) = t 2^(P(t) - a^2 log2(e) / 2) with t = 1 / (1 + 0.4 a):
    t is off by 1 step (its denominator) and 2 (a reciprocal's ulp), which Phi(-a) takes at most twice (its logarithm's
    slope over t's: 0.8 / 0.4 at a = 0, less beyond); P by 1.5 of its fit and 3 of its roundings; the exponent by those of
    a^2, its factor and its sum (0.75 + 0.5 steps of v^2, and 1.8 of P); 2^x by 4 (2 ulp); two products by 1 each: 18.3 +
    1.25 v^2."""
    N, K = 256, 32
    x, w = torch.zeros(M, K).bfloat16(), torch.zeros(N, K).bfloat16()
    x[:, 0] = 1
    w[:, 0] = torch.linspace(-12.5, 12.5, N).bfloat16()
    w[3, 0], w[4, 0], w[5, 0] = -5.0, -5.5, -0.0
    out = torch.empty(M, N, device=dev)
    moe.linear(moe.linear_problem(M, N, K, out_dtype="f32", activation="gelu"), x.to(dev), w.to(dev), out,
               moe.alloc_op_workspace(dev))
    v = w[:, 0].double().expand(M, N)
    want = v * torch.special.erfc(-v / math.sqrt(2.0)) / 2
    ref.check(out, want, (2 * v * v + 20) * EPS32 * want.abs(), "gelu")


@gpu
@pytest.mark.parametrize("K", [4096, 16384, 32768])
@pytest.mark.parametrize("M", [5, 40, 2000])
def test_long_sums_of_one_sign(dev, M, K):
    """The tensor core's own sums, 16 products a step and each perhaps truncated, stay bounded however long K is: 2048
    values (128 steps, each off by 2^-23 of the sum so far, which grows evenly: half of that of the whole on average).
    Then they are joined in float, one after the other (2^-24 of the sum so far), and so are at most 8 parts of K."""
    N, g = 300, gen(M + K)
    x, w = ((torch.rand(n, K, generator=g) + 0.5).bfloat16() for n in (M, N))
    out = torch.empty(M, N, device=dev)
    moe.linear(moe.linear_problem(M, N, K, out_dtype="f32"), x.to(dev), w.to(dev), out, moe.alloc_op_workspace(dev))
    want = x.double() @ w.double().T
    steps = 128 / 2 + K / 2048 / 4 + 16
    ref.check(out, want, steps * TRUNC32 * want.abs(), "out")


def test_refuses_a_depth_past_32_bits(lib):
    p = moe.linear_problem(5, 96, 64)
    for K in (2 ** 31 - 8, (1 << 30) + 8):
        p.K = K
        assert call(lib, p) == UNSUPPORTED
