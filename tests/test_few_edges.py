"""moe_forward_few at the ends of its ranges, against plain 64-bit forms."""
import ctypes

import pytest
import torch

import mixture_experts_layer_gate_gb300 as moe
from tests import op_reference as ref
from tests.few_reference import _quantised
from tests.test_operators import codes_of, few_weights, gen, randn, run_few

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


# ------------------------------------------------------------------ a NaN in the gate's correction bias


def few_of(dev, p, w, x, logits, bias):
    out, ws = torch.full((p.T, p.H), float("nan"), dtype=torch.bfloat16, device=dev), moe.alloc_few_workspace(p, dev)
    moe.forward_few(p, w, x, logits, bias, out, ws)
    return out, moe.get_device_error(ws)


@gpu
@pytest.mark.parametrize("E,k,gate", [(8, 2, {}), (64, 6, {}), (300, 4, dict(renormalize=False)),
                                      (64, 8, dict(n_group=8, topk_group=4)), (64, 8, dict(n_group=8, topk_group=2)),
                                      (256, 8, dict(n_group=8, topk_group=4, routed_scaling_factor=2.5))])
@pytest.mark.parametrize("T", [1, 5])
def test_an_expert_with_a_nan_bias_is_not_chosen(dev, T, E, k, gate):
    H, I = 256, 128
    p = moe.problem(T, H, I, E, k, scoring="sigmoid", **gate)
    g = gen(E + T)
    wd = moe.Weights(*[None if t is None else t.to(dev) for t in few_weights(p, False, 5)])
    x, logits = randn(g, T, H).to(torch.bfloat16).to(dev), (1.5 * randn(g, T, E)).to(dev)
    bias = (0.2 * torch.rand(E, generator=g) - 0.1).to(dev)
    out = [1] if E == 8 else [1, 3, E - 1]
    bias[out] = float("nan")
    ids, weights = torch.empty((T, k), dtype=torch.int32, device=dev), torch.empty((T, k), device=dev)
    moe.gate_topk(p, logits, bias, ids, weights)
    assert not any(bool((ids == e).any()) for e in out)
    low = torch.where(torch.isnan(bias), torch.full_like(bias, -1e30), bias)  # the last of all, and chosen by nobody
    got, err = few_of(dev, p, wd, x, logits, bias)
    want, _ = few_of(dev, p, wd, x, logits, low)
    assert err == 0 and torch.equal(got, want)


@gpu
@pytest.mark.parametrize("wdtype", ["bf16", "int4"])
@pytest.mark.parametrize("n_group", [0, 2])
def test_fewer_experts_than_choices(dev, wdtype, n_group):
    """Two of four experts usable for three choices: the third is reported and counts nothing."""
    T, H, I, E, k = 3, 256, 128, 4, 3
    gate = dict(scoring="sigmoid", wdtype=wdtype, n_group=n_group, topk_group=n_group)
    p, p2 = moe.problem(T, H, I, E, k, **gate), moe.problem(T, H, I, E, 2, **gate)
    g = gen(2)
    wd = moe.Weights(*[None if t is None else t.to(dev) for t in few_weights(p, False, 5)])
    x, logits = randn(g, T, H).to(torch.bfloat16).to(dev), randn(g, T, E).to(dev)
    nan = float("nan")
    bias, low = torch.tensor([nan, 0.1, nan, 0.0], device=dev), torch.tensor([-1e30, 0.1, -1e30, 0.0], device=dev)
    ids, weights = torch.empty((T, k), dtype=torch.int32, device=dev), torch.empty((T, k), device=dev)
    moe.gate_topk(p, logits, bias, ids, weights)
    assert bool((weights[:, 2] == 0).all()) and bool(((ids[:, 2] < 0) | (ids[:, 2] >= E)).all())
    got, err = few_of(dev, p, wd, x, logits, bias)
    want, none = few_of(dev, p2, wd, x, logits, low)
    assert err == 5 and none == 0 and torch.equal(got, want)
    got, err = few_of(dev, p, wd, x, logits, torch.full_like(bias, nan))  # no expert at all
    assert err == 5 and bool((got == 0).all())


# ------------------------------------------------------------------ the widest tokens of each format


WIDEST = {"int4": {1: 60416, 2: 31872, 3: 21632, 4: 16384, 8: 8192}, "bf16": {1: 65664, 2: 32768, 3: 21888, 8: 8192}}
WIDEST["int4_paired"], WIDEST["fp8"], WIDEST["int8"] = WIDEST["int4"], WIDEST["bf16"], WIDEST["bf16"]


@pytest.mark.parametrize("wdtype", list(WIDEST))
def test_limits_of_the_token_width(wdtype):
    moe.load()
    for T, H in WIDEST[wdtype].items():
        p, over = moe.problem(T, H, 128, 2, 1, wdtype=wdtype), moe.problem(T, H + 128, 128, 2, 1, wdtype=wdtype)
        assert moe.few_workspace_size(p) > 0 and moe.few_workspace_size(over) == 0, (T, H)
        w, lib = moe.binding.WeightsStruct(4096, 4096, 4096, 4096, 4096, 4096), moe.load()
        if wdtype != "fp8":
            w.a1_scale = w.a2_scale = None
        if wdtype == "bf16":
            w.w13_scale = w.w2_scale = None
        assert lib.moe_forward_few(ctypes.byref(over), ctypes.byref(w), 4096, 4096, None, 4096, 4096, 1 << 30, None) == 2
    for T in range(1, 9):
        for H in range(128, 8193, 128):
            assert moe.few_workspace_size(moe.problem(T, H, 128, 2, 1, wdtype=wdtype)) > 0


@gpu
@pytest.mark.parametrize("wdtype,zero", [("int4", False), ("int4", True), ("int4_paired", False), ("bf16", False),
                                         ("fp8", False), ("int8", True)])
@pytest.mark.parametrize("T", [1, 2, 3])
def test_widest_tokens(dev, wdtype, zero, T):
    run_few(dev, T, WIDEST[wdtype][T], 128, 2, 1, zero=zero, wdtype=wdtype)
