"""moe_forward_few at the ends of its ranges, against plain 64-bit forms."""
import pytest
import torch

import mixture_experts_layer_gate_gb300 as moe
from tests import op_reference as ref
from tests.few_reference import _quantised
from tests.test_operators import codes_of, gen, randn

gpu = pytest.mark.gpu


@pytest.fixture
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.load()
    return torch.device("cuda:0")


# ------------------------------------------------------------------ dynamic scales of tiny activations


def one_fp8_expert(dev, x, w13, s13, w2, s2):
    T, H = x.shape
    p = moe.problem(T, H, w2.shape[2], 1, 1, wdtype="fp8", act_scale="dynamic")
    w = moe.Weights(*[t.to(dev) for t in (w13, w2, s13, s2)])
    out, ws = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=dev), moe.alloc_few_workspace(p, dev)
    moe.forward_few(p, w, x.to(dev), torch.zeros(T, 1, device=dev), None, out, ws)
    assert moe.get_device_error(ws) == 0
    return out


@gpu
@pytest.mark.parametrize("w2_scale", [1.0, 1e-5])
def test_dynamic_scale_below_the_smallest_normal_float(dev, w2_scale):
    """max |act| / 448 is subnormal, its reciprocal infinite, and its product with an expert's scale has few bits."""
    g, T, H, I = gen(3), 3, 256, 256
    x = (1e-18 * randn(g, T, H)).to(torch.bfloat16)
    x[1] = 0
    w13, w2 = codes_of(g, 1, 2 * I, H), codes_of(g, 1, H, I)
    s13, s2 = torch.tensor([4e-4]), torch.tensor([w2_scale])
    got = one_fp8_expert(dev, x, w13, s13, w2, s2)
    a1 = float((x.float().abs().max() / 448.0))
    m13, m2 = ref.e4m3_values(w13[0]) * float(s13), ref.e4m3_values(w2[0]) * float(s2)
    xq = ref.e4m3_round((x.float() / a1).double()) * a1
    h, size = xq @ m13.T, xq.abs() @ m13.abs().T
    v, d = ref.swiglu(h, (H / 16 + 48) * ref.TRUNC32 * size)
    tiny = 2.0 ** -149                     # what a step among subnormal floats is
    d = d + 2 * tiny
    amax = float(v.abs().max())
    assert 2.0 ** -149 * 1e4 < amax / 448.0 < 2.0 ** -128  # 1 / scale is past the largest float
    scale = amax / 448.0
    rel = 4 * ref.TRUNC32 + float(d.max()) / amax + tiny / scale
    q, dq = _quantised(v, d, scale, rel)
    want = q @ m2.T
    tol = dq @ m2.abs().T + (I / 16 + 48 + 66) * ref.TRUNC32 * (q.abs() @ m2.abs().T) + 2 * tiny
    half, least = ref.half_step(torch.bfloat16)
    ref.check(got, want, half * want.abs() + least + 1.01 * tol, "out")
    assert float(want.abs().max()) > 100 * least and bool((got[1] == 0).all())


@gpu
def test_dynamic_scale_that_would_be_zero(dev):
    """max |act| / 448 below the smallest float: scale 1, codes and output of zero."""
    T, H, I = 2, 128, 128
    x = torch.full((T, H), 2.0 ** -72, dtype=torch.bfloat16)
    x[1] = 0
    w13, w2 = torch.full((1, 2 * I, H), 0x38, dtype=torch.uint8), torch.full((1, H, I), 0x38, dtype=torch.uint8)
    # every gate and up value is 128 * 2^-72 * 2^-7 = 2^-72, their product's half 2^-145: 16 steps of a float
    out = one_fp8_expert(dev, x, w13, torch.tensor([2.0 ** -7]), w2, torch.tensor([1.0]))
    assert bool((out == 0).all())
