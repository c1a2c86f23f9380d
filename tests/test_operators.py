"""The operators around the layer: refusals (no GPU), and each against its plain 64-bit form at the sizes, strides and
values where it can go wrong."""
import ctypes

import pytest
import torch

import mixture_experts_layer_gate_gb300 as moe
from mixture_experts_layer_gate_gb300 import binding
from tests import few_reference
from tests import op_reference as ref

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    import os
    from mixture_experts_layer_gate_gb300 import build
    if not os.path.exists(moe.LIB_PATH) or not os.path.exists(build.OPS):
        build.build()
    return moe.load()


@pytest.fixture
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.load()
    return torch.device("cuda:0")


def far(t, stride, dev):
    """t on the device with rows `stride` elements apart (memory between them as it is)."""
    w = torch.empty((t.shape[0] - 1) * stride + t.shape[1], dtype=t.dtype, device=dev)
    v = torch.as_strided(w, t.shape, (stride, 1))
    v.copy_(t)
    return v


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g)


def wide(t, pad, dev, fill=float("nan")):
    """t on the device inside rows that are `pad` longer and start `pad` in; what lies between must not be read."""
    if not pad:
        return t.to(dev)
    w = torch.full((t.shape[0], t.shape[1] + 2 * pad), fill).to(t.dtype)
    w[:, pad:pad + t.shape[1]] = t
    return w.to(dev)[:, pad:pad + t.shape[1]]


# ------------------------------------------------------------------ refusals (CPU)


P = 4096  # an address that is never dereferenced: the checks come before any launch


def test_struct_layouts():
    assert ctypes.sizeof(moe.NormProblem) == 24
    assert ctypes.sizeof(moe.RouterProblem) == 16
    assert ctypes.sizeof(moe.Fp8GemmProblem) == 20


def call_norm(lib, n, x=P, xs=None, r=None, rs=0, w=P, ro=None, ros=0, y=P, ys=None, codes=None, scales=None):
    H = n.H if n is not None else 0
    return lib.moe_add_rms_norm(ctypes.byref(n) if n is not None else None, x, H if xs is None else xs, r, rs, w, ro,
                                ros, y, H if ys is None else ys, codes, scales, None)


def test_norm_refusals(lib):
    n = moe.norm_problem(4, 256)
    bad = [dict(x=None), dict(w=None), dict(x=P + 1), dict(xs=255), dict(y=None), dict(ys=8), dict(y=P + 1),
           dict(ro=P, ros=256), dict(r=P, rs=100), dict(r=P, rs=256, ro=P, ros=512), dict(codes=P, scales=P),
           dict(scales=P)]
    for kw in bad:
        assert call_norm(lib, n, **kw) == INVALID, kw
    q = moe.norm_problem(4, 256, quant="block")
    for kw in (dict(), dict(codes=P), dict(scales=P), dict(codes=P, scales=P + 2)):
        assert call_norm(lib, q, **kw) == INVALID, kw
    assert call_norm(lib, None) == INVALID
    for kw in (dict(T=-1, H=8), dict(T=1, H=0), dict(T=1, H=8, eps=-1.0), dict(T=1, H=8, eps=float("nan"))):
        assert call_norm(lib, moe.norm_problem(**kw)) == INVALID, kw
    assert call_norm(lib, moe.norm_problem(1, 16385)) == UNSUPPORTED
    odd = moe.norm_problem(1, 8)
    odd.dtype = 3
    assert call_norm(lib, odd) == INVALID
    odd = moe.norm_problem(1, 8, dtype="f32")
    odd.weight_dtype = 0
    assert call_norm(lib, odd) == INVALID
    odd = moe.norm_problem(1, 8)
    odd.quant = 3
    assert call_norm(lib, odd) == INVALID
    assert call_norm(lib, moe.norm_problem(0, 8), x=None, w=None, y=None) == 0


def test_router_refusals(lib):
    def call(r, x=P, xs=None, w=P, ws_=None, out=P, ws=P, n=256):
        return lib.moe_router_logits(ctypes.byref(r), x, r.H if xs is None else xs, w, r.H if ws_ is None else ws_,
                                     out, ws, n, None)
    r = moe.router_problem(4, 256, 8)
    for kw in (dict(x=None), dict(w=None), dict(out=None), dict(x=P + 8), dict(w=P + 8), dict(xs=248), dict(xs=260),
               dict(ws_=260), dict(out=P + 2)):
        assert call(r, **kw) == INVALID, kw
    for kw in (dict(ws=None), dict(ws=P + 16), dict(n=255)):
        assert call(r, **kw) == WORKSPACE, kw
    for kw in (dict(T=-1, H=256, E=8), dict(T=1, H=12, E=8), dict(T=1, H=0, E=8), dict(T=1, H=8, E=0)):
        assert call(moe.router_problem(**kw)) == INVALID, kw
    assert call(moe.router_problem(1, 8, 8, dtype="f32")) == INVALID
    assert call(moe.router_problem(1, 8, 1025)) == UNSUPPORTED
    assert call(moe.router_problem(0, 8, 8), x=None, out=None) == 0


def test_fp8_gemm_refusals(lib):
    def call(g, a=P, as_=None, sc=P, ss=None, w=P, ws_=None, wsc=P, out=P, os_=None, ws=P, n=256):
        kb = -(-g.K // 128)
        return lib.moe_gemm_fp8_block(ctypes.byref(g), a, g.K if as_ is None else as_, sc, kb if ss is None else ss, w,
                                      g.K if ws_ is None else ws_, wsc, out, g.N if os_ is None else os_, ws, n, None)

    def call_swiglu(g, codes=P, scales=P, a=P):
        kb = -(-g.K // 128)
        return lib.moe_gemm_fp8_block_swiglu(ctypes.byref(g), a, g.K, P, kb, P, g.K, P, codes, scales, P, 256, None)
    g = moe.fp8_gemm_problem(4, 256, 256)
    for kw in (dict(a=None), dict(sc=None), dict(w=None), dict(wsc=None), dict(out=None), dict(a=P + 8), dict(w=P + 8),
               dict(as_=240), dict(as_=264), dict(ws_=264), dict(ss=1), dict(os_=255), dict(out=P + 1),
               dict(wsc=P + 2)):
        assert call(g, **kw) == INVALID, kw
    for kw in (dict(ws=None), dict(ws=P + 16), dict(n=255)):
        assert call(g, **kw) == WORKSPACE, kw
    for kw in (dict(M=-1, N=8, K=16), dict(M=1, N=-8, K=16), dict(M=1, N=8, K=0), dict(M=1, N=8, K=24)):
        assert call(moe.fp8_gemm_problem(**kw)) == INVALID, kw
    g3 = moe.fp8_gemm_problem(4, 256, 256)
    g3.out_dtype = 3
    assert call(g3) == INVALID
    g3 = moe.fp8_gemm_problem(4, 256, 256)
    g3.accumulate = 2
    assert call(g3) == INVALID
    assert call(moe.fp8_gemm_problem(0, 8, 16), a=None) == 0
    assert call(moe.fp8_gemm_problem(8, 0, 16), w=None) == 0
    for kw in (dict(codes=None), dict(scales=None), dict(codes=P + 8), dict(a=None)):
        assert call_swiglu(g, **kw) == INVALID, kw
    assert call_swiglu(moe.fp8_gemm_problem(4, 192, 256)) == INVALID
    assert call_swiglu(moe.fp8_gemm_problem(4, 256, 256, accumulate=True)) == INVALID
    assert call_swiglu(moe.fp8_gemm_problem(0, 256, 256), codes=None) == 0


def test_few_refusals(lib):
    def call(p, w=None, x=P, logits=P, out=P, ws=P, n=1 << 30):
        w = w or binding.WeightsStruct(P, P)
        return lib.moe_forward_few(ctypes.byref(p), ctypes.byref(w), x, logits, None, out, ws, n, None)
    p = moe.problem(4, 256, 512, 8, 2)
    for kw in (dict(x=None), dict(logits=None), dict(out=None), dict(x=P + 8), dict(out=P + 8),
               dict(w=binding.WeightsStruct(P, None)), dict(w=binding.WeightsStruct(P, P + 8))):
        assert call(p, **kw) == INVALID, kw
    size = moe.few_workspace_size(p)
    for kw in (dict(ws=None), dict(ws=P + 16), dict(n=size - 1)):
        assert call(p, **kw) == WORKSPACE, kw
    assert call(moe.problem(9, 256, 512, 8, 2)) == UNSUPPORTED
    assert call(moe.problem(8, 8320, 128, 8, 2)) == UNSUPPORTED
    assert moe.few_workspace_size(moe.problem(8, 8320, 128, 8, 2)) == 0
    assert moe.few_workspace_size(moe.problem(8, 8192, 128, 8, 2)) > 0
    p4 = moe.problem(4, 256, 512, 8, 2, wdtype="int4")
    assert call(p4, w=binding.WeightsStruct(P, P, P + 2, P)) == INVALID
    assert call(p4, w=binding.WeightsStruct(P, P, P, P, None, None, P + 2, P)) == INVALID
    assert moe.few_workspace_size(moe.problem(9, 256, 512, 8, 2)) == 0
    assert moe.few_workspace_size(moe.problem(4, 100, 512, 8, 2)) == 0
    assert call(moe.problem(4, 256, 512, 8, 2, wdtype="fp8")) == INVALID  # no scales
    assert call(moe.problem(4, 256, 512, 8, 2, wdtype="int4", group_size=64)) == UNSUPPORTED
    assert call(moe.problem(0, 256, 512, 8, 2), x=None, out=None) == 0
    with pytest.raises(moe.MoEError):
        moe.alloc_few_workspace(moe.problem(9, 256, 512, 8, 2), "cpu")


def test_binding_refuses_tensors_that_are_not_what_the_problem_says(lib):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.zeros(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on a GPU
        moe.add_rms_norm(moe.norm_problem(4, 256), x, w, y=x)
    with pytest.raises(ValueError):
        moe.router_logits(moe.router_problem(4, 256, 8), x, x, x, x)


def test_binding_refuses_what_is_no_tensor_or_problem(lib):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    n = moe.norm_problem(4, 256)
    with pytest.raises(TypeError):
        moe.add_rms_norm(n, [1.0], x)
    with pytest.raises((TypeError, BufferError)):
        moe.add_rms_norm(None, x, x)
    with pytest.raises(ValueError):
        moe.add_rms_norm(moe.router_problem(4, 256, 8), x, x)
    with pytest.raises(TypeError):
        moe.router_logits(moe.router_problem(0, 256, 0), None, None, None, None)


@gpu
def test_binding_refuses_shapes_types_and_strides(dev):
    n = moe.norm_problem(4, 256, quant="block")
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    x, w = bf(4, 256), bf(256)
    codes, scales = torch.zeros(4, 256, dtype=torch.uint8, device=dev), torch.zeros(4, 2, device=dev)
    moe.add_rms_norm(n, x, w, codes=codes, scales=scales)
    for bad in (dict(x=bf(4, 255)), dict(x=bf(5, 256)), dict(x=bf(4 * 256)), dict(x=x.float()), dict(x=bf(256, 4).T),
                dict(x=x.cpu()), dict(weight=bf(255)), dict(weight=bf(512)[::2]), dict(codes=codes[:3]),
                dict(scales=scales.half()), dict(residual=bf(3, 256)), dict(y=bf(4, 8))):
        args = dict(dict(x=x, weight=w, codes=codes, scales=scales), **bad)
        with pytest.raises(ValueError):
            moe.add_rms_norm(n, **args)
    with pytest.raises(moe.MoEError):
        moe.add_rms_norm(n, x, w, y=x.clone())   # quantises, but has nowhere to put the codes
    ws = moe.alloc_op_workspace(dev)
    logits = torch.zeros(4, 8, device=dev)
    with pytest.raises(ValueError):
        moe.router_logits(moe.router_problem(4, 256, 8), x, bf(7, 256), logits, ws)
    with pytest.raises(ValueError):
        moe.router_logits(moe.router_problem(4, 256, 8), x, bf(8, 256), logits, ws.cpu())
    with pytest.raises(moe.MoEError):
        moe.router_logits(moe.router_problem(4, 256, 8), x, bf(8, 256), logits, ws[:128])
    stream = torch.cuda.current_stream().cuda_stream
    moe.router_logits(moe.router_problem(4, 256, 8), x, bf(8, 256), logits, ws, stream)
    moe.router_logits(moe.router_problem(1, 256, 8), x[:1], bf(8, 256), logits[:1], ws, stream=stream)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ residual + RMS norm


def run_norm(dev, T, H, dtype, wdtype, residual, quant, pad, seed=0, x=None, eps=1e-6, in_place=False, y=True):
    g = gen(seed)
    x = randn(g, T, H).to(DT[dtype]) if x is None else x
    r = (3 * randn(g, T, H)).to(DT[dtype]) if residual else None
    w = (1 + 0.2 * randn(g, H)).to(DT[wdtype])
    n = moe.norm_problem(T, H, dtype=dtype, weight_dtype=wdtype, eps=eps, quant=quant)
    xd, rd = wide(x, pad, dev), wide(r, pad, dev) if residual else None
    yd = wide(torch.zeros(T, H, dtype=DT[dtype]), pad, dev) if y else None
    ro = (rd if in_place else wide(torch.zeros(T, H, dtype=DT[dtype]), pad, dev)) if residual else None
    nb = {"none": 0, "block": -(-H // 128), "token": 1}[quant]
    codes = torch.full((T, H), 0xAA, dtype=torch.uint8, device=dev) if nb else None
    scales = torch.full((T, nb), -1.0, device=dev) if nb else None
    moe.add_rms_norm(n, xd, w.to(dev), residual=rd, residual_out=ro, y=yd, codes=codes, scales=scales)
    torch.cuda.synchronize()
    s, v, dv = ref.norm(x, r, w, eps)
    rel, tiny = ref.half_step(DT[dtype])
    if residual:
        ref.check(ro, s, (rel + ref.EPS32) * s.abs() + tiny, "residual")
    if y:
        ref.check(yd, v, rel * v.abs() + 1.1 * dv + tiny, "y")
    if nb:
        ref.check_quantised(codes, scales, v, dv, 128 if quant == "block" else H, "norm")


@gpu
@pytest.mark.parametrize("H", [1, 7, 8, 127, 128, 129, 256, 264, 520, 1000, 1024, 1032, 2571, 4096, 7168, 8200, 16384])
@pytest.mark.parametrize("quant", ["none", "block", "token"])
def test_norm_widths(dev, H, quant):
    run_norm(dev, 3, H, "bf16", "bf16", True, quant, 0)


@gpu
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("H,pad", [(384, 0), (384, 8), (384, 3), (1000, 1), (2571, 5), (5120, 16)])
def test_norm_types_and_strides(dev, dtype, wdtype, H, pad):
    run_norm(dev, 5, H, dtype, wdtype, pad != 8, "block", pad)


@gpu
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 300])
@pytest.mark.parametrize("H", [64, 200, 1536])
def test_norm_rows(dev, T, H):
    run_norm(dev, T, H, "bf16", "bf16", False, "token", 0)


@gpu
@pytest.mark.parametrize("T,H,dtype,wdtype", [(700, 1032, "bf16", "bf16"), (1900, 1536, "f16", "f32"),
                                              (901, 8191, "bf16", "f32"), (305, 2048, "f32", "f32"),
                                              (320, 16384, "bf16", "bf16")])
@pytest.mark.parametrize("quant", ["none", "block", "token"])
def test_norm_more_rows_than_ctas(dev, T, H, dtype, wdtype, quant):
    run_norm(dev, T, H, dtype, wdtype, True, quant, 0, in_place=quant == "block")
    if quant == "none":
        run_norm(dev, T, H, dtype, wdtype, False, quant, 0)


@gpu
@pytest.mark.parametrize("T,H,dtype", [(1500, 1032, "bf16"), (1000, 2048, "f32"), (160, 7168, "bf16"), (400, 7168, "f16"),
                                       (500, 7167, "bf16"), (153, 8192, "bf16")])
@pytest.mark.parametrize("quant", ["none", "block", "token"])
def test_norm_rows_that_fit_the_sms_and_more(dev, T, H, dtype, quant):
    run_norm(dev, T, H, dtype, dtype, quant != "token", quant, 0)


@gpu
def test_norm_offsets_past_32_bits(dev):
    g, H, far_apart = gen(8), 520, 2 ** 30 + 8
    x, r, w = randn(g, 3, H).to(torch.bfloat16), randn(g, 3, H).to(torch.bfloat16), torch.ones(H, dtype=torch.bfloat16)
    n = moe.norm_problem(3, H)
    want, total = torch.empty_like(x, device=dev), torch.empty_like(x, device=dev)
    moe.add_rms_norm(n, x.to(dev), w.to(dev), residual=r.to(dev), residual_out=total, y=want)
    xd, rd = far(x, far_apart, dev), far(r, far_apart + 8, dev)
    yd = far(torch.zeros_like(x), far_apart + 16, dev)
    moe.add_rms_norm(n, xd, w.to(dev), residual=rd, residual_out=rd, y=yd)
    assert torch.equal(yd, want) and torch.equal(rd, total)


@gpu
def test_norm_in_place_and_without_y(dev):
    run_norm(dev, 9, 1100, "bf16", "bf16", True, "block", 0, in_place=True)
    run_norm(dev, 9, 1024, "bf16", "bf16", True, "block", 8, in_place=True, y=False)
    run_norm(dev, 9, 40, "f16", "f16", True, "token", 0, in_place=True)


@gpu
def test_norm_rows_of_zeros_large_and_tiny_values(dev):
    x = randn(gen(3), 6, 512)
    x[0] = 0.0          # all zero: v = 0, scale 1, codes 0
    x[1] *= 1e15        # squares near the top of float
    x[2] *= 1e-12       # eps decides
    x[3, :] = 0.0
    x[3, 200] = 1.0     # one block with a value, three of zeros
    x[4] *= 1e-30       # squares underflow
    for quant in ("block", "token"):
        run_norm(dev, 6, 512, "f32", "f32", False, quant, 0, x=x)


@gpu
@pytest.mark.parametrize("quant", ["block", "token"])
@pytest.mark.parametrize("H", [512, 515])
def test_norm_nan_stays_in_its_row(dev, quant, H):
    x = randn(gen(4), 4, H).to(torch.bfloat16)
    x[2, 100] = float("nan")
    n = moe.norm_problem(4, H, quant=quant)
    w = torch.ones(H, dtype=torch.bfloat16, device=dev)
    y = torch.zeros(4, H, dtype=torch.bfloat16, device=dev)
    nb = -(-H // 128) if quant == "block" else 1
    codes = torch.zeros(4, H, dtype=torch.uint8, device=dev)
    scales = torch.zeros(4, nb, device=dev)
    moe.add_rms_norm(n, x.to(dev), w, y=y, codes=codes, scales=scales)
    assert torch.isnan(y[2]).all() and torch.isnan(scales[2]).all() and bool(((codes[2] & 127) == 127).all())
    keep = [0, 1, 3]
    assert torch.isfinite(y[keep]).all() and torch.isfinite(scales[keep]).all()


@gpu
@pytest.mark.parametrize("quant", ["block", "token"])
@pytest.mark.parametrize("H", [256, 259, 1280])
def test_norm_values_below_any_scale(dev, quant, H):
    """max |v| / 448 below the smallest float: scale 1 and codes of zero, no division by zero."""
    x = torch.full((3, H), 3e-43)
    x[1] = 0.5
    n = moe.norm_problem(3, H, dtype="f32", eps=1.0, quant=quant)
    nb = -(-H // 128) if quant == "block" else 1
    codes, scales = torch.full((3, H), 0xAA, dtype=torch.uint8, device=dev), torch.zeros(3, nb, device=dev)
    moe.add_rms_norm(n, x.to(dev), torch.ones(H, device=dev), codes=codes, scales=scales)
    for t in (0, 2):
        assert bool((scales[t] == 1).all()) and bool((codes[t] == 0).all())
    assert bool((codes[1] == 0x7E).all())  # each value is its block's largest: 448


# ------------------------------------------------------------------ router scores


@gpu
@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 17, 64, 127, 128, 129, 300])
@pytest.mark.parametrize("H,E", [(8, 1), (264, 8), (1024, 60), (3584, 64), (7168, 256), (520, 300)])
def test_router(dev, T, H, E):
    for dtype, pad in (("bf16", 0), ("f16", 8)):
        g = gen(T * 7 + E)
        x, w = randn(g, T, H).to(DT[dtype]), (0.02 * randn(g, E, H)).to(DT[dtype])
        logits = torch.full((T, E), float("nan"), device=dev)
        ws = moe.alloc_op_workspace(dev)
        moe.router_logits(moe.router_problem(T, H, E, dtype=dtype), wide(x, pad, dev), wide(w, pad, dev), logits, ws)
        want, tol = ref.router(x, w)
        ref.check(logits, want, tol, "logits")
        assert moe.get_device_error(ws) == 0


@gpu
def test_router_most_experts_and_many_tokens(dev):
    for T, H, E in ((1000, 512, 1024), (4100, 256, 3), (1, 4096, 1024)):
        g = gen(E)
        x, w = randn(g, T, H).to(torch.bfloat16), randn(g, E, H).to(torch.bfloat16)
        logits = torch.full((T, E), float("nan"), device=dev)
        ws = moe.alloc_op_workspace(dev)
        moe.router_logits(moe.router_problem(T, H, E), x.to(dev), w.to(dev), logits, ws)
        want, tol = ref.router(x, w)
        ref.check(logits, want, tol, "logits")
        assert moe.get_device_error(ws) == 0


@gpu
@pytest.mark.parametrize("T,H,E", [(1, 24, 1024), (2, 2056, 1024), (3, 1032, 683), (3, 1032, 682), (4, 9000, 512),
                                   (4, 512, 513), (2, 32768, 5), (130, 32768, 40), (8, 7168, 256), (8, 1032, 257),
                                   (5, 4096, 409), (6, 264, 8), (7, 9000, 292), (7, 512, 293)])
def test_router_few_tokens_and_long_rows(dev, T, H, E):
    g = gen(E)
    x, w = randn(g, T, H).to(torch.float16), (0.02 * randn(g, E, H)).to(torch.float16)
    logits = torch.full((T, E), float("nan"), device=dev)
    ws = moe.alloc_op_workspace(dev)
    moe.router_logits(moe.router_problem(T, H, E, dtype="f16"), wide(x, 8, dev), wide(w, 8, dev), logits, ws)
    want, tol = ref.router(x, w)
    ref.check(logits, want, tol, "logits")
    assert moe.get_device_error(ws) == 0


@gpu
@pytest.mark.parametrize("T", [3, 9])
def test_router_offsets_past_32_bits(dev, T):
    g, H, E = gen(T), 520, 3
    x, w = randn(g, T, H).to(torch.bfloat16), randn(g, E, H).to(torch.bfloat16)
    ws, r = moe.alloc_op_workspace(dev), moe.router_problem(T, H, E)
    want, got = torch.zeros((T, E), device=dev), torch.zeros((T, E), device=dev)
    moe.router_logits(r, x.to(dev), w.to(dev), want, ws)
    moe.router_logits(r, far(x, 2 ** 31 // (T - 1) + 8, dev), far(w, 2 ** 30 + 8, dev), got, ws)
    assert moe.get_device_error(ws) == 0 and torch.equal(got, want)


@gpu
@pytest.mark.parametrize("T", [1, 40])
def test_router_nan_stays_in_its_token(dev, T):
    g = gen(9)
    x, w = randn(g, T, 1024).to(torch.bfloat16), randn(g, 16, 1024).to(torch.bfloat16)
    x[T - 1, 700] = float("nan")
    logits = torch.zeros((T, 16), device=dev)
    moe.router_logits(moe.router_problem(T, 1024, 16), x.to(dev), w.to(dev), logits, moe.alloc_op_workspace(dev))
    assert torch.isnan(logits[T - 1]).all() and torch.isfinite(logits[:T - 1]).all()


@gpu
def test_products_back_to_back(dev):
    """Launches that follow each other without a wait, over long sums, wide tiles and split ones."""
    g = gen(21)
    x, w = randn(g, 1024, 7168).to(torch.bfloat16), randn(g, 256, 7168).to(torch.bfloat16)
    logits = torch.full((1024, 256), float("nan"), device=dev)
    ws = moe.alloc_op_workspace(dev)
    xd, wd = x.to(dev), w.to(dev)
    a, sa, b, sb = product_inputs(1, 4096, 7168, 2)
    ad = [t.to(dev) for t in (a, sa, b, sb)]
    codes, scales = torch.empty((1, 2048), dtype=torch.uint8, device=dev), torch.empty((1, 16), device=dev)
    out = torch.empty((1, 4096), device=dev)
    for _ in range(40):
        moe.router_logits(moe.router_problem(1024, 7168, 256), xd, wd, logits, ws)
        moe.gemm_fp8_block_swiglu(moe.fp8_gemm_problem(1, 2048, 7168), *ad, codes, scales, ws)
        moe.gemm_fp8_block(moe.fp8_gemm_problem(1, 4096, 7168, out_dtype="f32"), *ad, out, ws)
    assert moe.get_device_error(ws) == 0
    want, tol = ref.router(x, w)
    ref.check(logits, want, tol, "logits")
    h, dh = ref.product(a, sa, b, sb)
    ref.check(out, h, 1.01 * dh + ref.EPS32 * h.abs(), "out")
    ref.check_quantised(codes, scales, *ref.swiglu(h, dh), 128, "swiglu")


# ------------------------------------------------------------------ block-scaled 8-bit product


def codes_of(g, *shape):
    return (100 * randn(g, *shape)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def product_inputs(M, rows, K, seed):
    g = gen(seed)
    kb = -(-K // 128)
    rand = lambda *s: torch.rand(s, generator=g)  # noqa: E731
    return (codes_of(g, M, K), rand(M, kb) * 0.01 + 0.001, codes_of(g, rows, K),
            rand(-(-rows // 128), kb) * 3e-4 + 1e-5)


def run_gemm(dev, M, N, K, out="bf16", pad=0, accumulate=False, seed=0):
    a, sa, w, sw = product_inputs(M, N, K, seed + M + N + K)
    dt = DT[out]
    old = randn(gen(5), M, N).to(dt)
    od = wide(old, pad, dev, fill=7.0)
    ws = moe.alloc_op_workspace(dev)
    moe.gemm_fp8_block(moe.fp8_gemm_problem(M, N, K, out_dtype=out, accumulate=accumulate), wide(a, pad, dev, fill=127),
                       wide(sa, pad, dev), wide(w, pad, dev, fill=127), sw.to(dev), od, ws)
    assert moe.get_device_error(ws) == 0
    want, tol = ref.product(a, sa, w, sw)
    if accumulate:
        want = want + old.double()
        tol = tol + ref.EPS32 * want.abs()
    rel, tiny = ref.half_step(dt)
    ref.check(od, want, rel * want.abs() + 1.01 * tol + tiny, "out")
    if pad:  # what lies between the rows is left alone
        whole = torch.as_strided(od, (M, pad), (od.stride(0), 1), od.storage_offset() + N)
        assert bool((whole == 7.0).all())


@gpu
@pytest.mark.parametrize("M", [1, 2, 16, 17, 64, 127, 128, 129, 200])
@pytest.mark.parametrize("N,K", [(1, 16), (8, 128), (127, 144), (128, 256), (257, 1104), (520, 2048)])
def test_gemm_sizes(dev, M, N, K):
    run_gemm(dev, M, N, K)


@gpu
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K,pad", [(5, 100, 1024, 16), (130, 301, 400, 32), (300, 640, 1152, 0), (1, 2048, 7168, 0)])
def test_gemm_types_strides_and_accumulation(dev, out, M, N, K, pad):
    run_gemm(dev, M, N, K, out, pad)
    run_gemm(dev, M, N, K, out, pad, accumulate=True)


@gpu
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K,pad", [(1030, 5000, 144, 16), (2049, 4360, 272, 0), (131, 40000, 144, 8), (100, 40008, 144, 8)])
def test_gemm_wide_tiles(dev, out, M, N, K, pad):
    """Tiles of 256 columns, whole and cut, several per CTA: stored as rows of 16-byte pieces where the strides allow it."""
    run_gemm(dev, M, N, K, out, 2 * pad)
    run_gemm(dev, M, N, K, out, 2 * pad + 16, accumulate=True)


@gpu
@pytest.mark.parametrize("M,N,K", [(8, 40, 16384), (3, 130, 30000), (1, 20, 65552), (5, 4900, 400), (8, 9000, 272)])
def test_gemm_few_rows_long_sums_and_many_columns(dev, M, N, K):
    run_gemm(dev, M, N, K, "f32")


@gpu
@pytest.mark.parametrize("M", [3, 20])
def test_gemm_offsets_past_32_bits(dev, M):
    N, K = 40, 272
    far_apart, far_w = (2 ** 31 // (n - 1) // 16 * 16 + 16 for n in (M, N))
    a, sa, w, sw = [t.to(dev) for t in product_inputs(M, N, K, M)]
    ws, p = moe.alloc_op_workspace(dev), moe.fp8_gemm_problem(M, N, K, out_dtype="f32")
    want, got = torch.zeros((M, N), device=dev), far(torch.zeros(M, N), far_apart, dev)
    moe.gemm_fp8_block(p, a, sa, w, sw, want, ws)
    moe.gemm_fp8_block(p, far(a, far_apart, dev), far(sa, far_apart, dev), far(w, far_w, dev), sw, got, ws)
    assert moe.get_device_error(ws) == 0 and torch.equal(got, want)


@gpu
def test_gemm_many_tiles(dev):
    run_gemm(dev, 1030, 5000, 640)
    run_gemm(dev, 700, 1000, 7168, "f32")


def run_swiglu(dev, M, N, K, pad=0, ws=None):
    a, sa, w, sw = product_inputs(M, 2 * N, K, M + N + K)
    codes = torch.full((M, N), 0xAA, dtype=torch.uint8, device=dev)
    scales = torch.full((M, N // 128), -1.0, device=dev)
    ws = moe.alloc_op_workspace(dev) if ws is None else ws
    moe.gemm_fp8_block_swiglu(moe.fp8_gemm_problem(M, N, K), wide(a, pad, dev, fill=127), wide(sa, pad, dev),
                              wide(w, pad, dev, fill=127), sw.to(dev), codes, scales, ws)
    assert moe.get_device_error(ws) == 0
    v, dv = ref.swiglu(*ref.product(a, sa, w, sw))
    ref.check_quantised(codes, scales, v, dv, 128, "swiglu")


@gpu
@pytest.mark.parametrize("M", [1, 3, 16, 100, 128, 129, 260])
@pytest.mark.parametrize("N,K,pad", [(128, 16, 0), (128, 1104, 16), (384, 512, 0), (2048, 256, 0)])
def test_swiglu_sizes(dev, M, N, K, pad):
    run_swiglu(dev, M, N, K, pad)


@gpu
def test_swiglu_many_tiles(dev):
    run_swiglu(dev, 1, 2048, 7168)
    run_swiglu(dev, 1500, 1280, 384)


@gpu
def test_swiglu_of_few_rows_shares_a_workspace(dev):
    """Widths in turn, and each again: every call finds the counters of the workspace at zero."""
    ws = moe.alloc_op_workspace(dev)
    for M, N, K in ((8, 256, 128), (1, 16384, 128), (8, 256, 128), (3, 9088, 144), (8, 16384, 16)):
        run_swiglu(dev, M, N, K, ws=ws)


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 2048, 7168), (8, 128, 272)])
def test_swiglu_of_few_rows_without_scratch(dev, M, N, K):
    run_swiglu(dev, M, N, K, ws=torch.zeros(256, dtype=torch.uint8, device=dev))


@gpu
def test_product_of_zeros_and_nan(dev):
    M, N, K = 20, 256, 384
    a, sa, w, sw = product_inputs(M, 2 * N, K, 1)
    a[3] = 0
    a[7, 130] = 0x7F  # NaN in one row
    ws = moe.alloc_op_workspace(dev)
    out = torch.zeros(M, 2 * N, device=dev)
    dw = [t.to(dev) for t in (a, sa, w, sw)]
    moe.gemm_fp8_block(moe.fp8_gemm_problem(M, 2 * N, K, out_dtype="f32"), *dw, out, ws)
    others = [m for m in range(M) if m != 7]
    assert bool((out[3] == 0).all()) and torch.isnan(out[7]).all() and torch.isfinite(out[others]).all()
    codes = torch.full((M, N), 0xAA, dtype=torch.uint8, device=dev)
    scales = torch.zeros((M, N // 128), device=dev)
    moe.gemm_fp8_block_swiglu(moe.fp8_gemm_problem(M, N, K), *dw, codes, scales, ws)
    assert bool(((codes[3] & 127) == 0).all()) and bool((scales[3] == 1).all())
    assert torch.isnan(scales[7]).all() and bool(((codes[7] & 127) == 127).all())
    assert torch.isfinite(scales[others]).all()


@gpu
@pytest.mark.parametrize("M,scratch", [(1, True), (8, True), (8, False), (130, False)])
def test_swiglu_values_below_any_scale(dev, M, scratch):
    N, K = 256, 16
    ones = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device=dev)  # noqa: E731
    ws = moe.alloc_op_workspace(dev)[:None if scratch else 256]
    codes, scales = torch.full((M, N), 0xAA, dtype=torch.uint8, device=dev), torch.zeros(M, N // 128, device=dev)
    w_scale = torch.full((2 * N // 128, 1), 2e-23, device=dev)  # gate and up 3.2e-22 each, silu(gate) up 5e-44
    moe.gemm_fp8_block_swiglu(moe.fp8_gemm_problem(M, N, K), ones(M, K), torch.ones(M, 1, device=dev), ones(2 * N, K),
                              w_scale, codes, scales, ws)
    assert moe.get_device_error(ws) == 0
    assert bool((scales == 1).all()) and bool((codes == 0).all())


# ------------------------------------------------------------------ the layer for a few tokens


def few_weights(p, zero, seed):
    g = gen(seed)
    E, H, I = p.E, p.H, p.I
    rand = lambda *s: torch.rand(s, generator=g)  # noqa: E731
    byte = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8)  # noqa: E731
    if p.wdtype == 0:
        return ((0.05 * randn(g, E, 2 * I, H)).to(torch.bfloat16), (0.05 * randn(g, E, H, I)).to(torch.bfloat16),
                None, None, None, None, None, None)
    if p.wdtype == 1:
        a = (None, None) if p.act_scale else (torch.tensor([4.0 / 448]), torch.tensor([3.0 / 448]))
        return (codes_of(g, E, 2 * I, H), codes_of(g, E, H, I), rand(E) * 4e-4 + 2e-4, rand(E) * 4e-4 + 2e-4, *a,
                None, None)
    per, q = (1, 255) if p.wdtype == 3 else (2, 15)
    scale = lambda *s: ((rand(*s) + 0.5) * 0.15 / q).half()  # noqa: E731
    z = (lambda *s: torch.randint(0, q + 1, s, generator=g, dtype=torch.uint8)) if zero else (lambda *s: None)
    return (byte(E, 2 * I, H // per), byte(E, H, I // per), scale(E, 2 * I, H // 128), scale(E, H, I // 128), None, None,
            z(E, 2 * I, H // 128), z(E, H, I // 128))


def run_few(dev, T, H, I, E, k, zero=False, seed=0, bias=False, x=None, logits=None, **gate):
    p = moe.problem(T, H, I, E, k, **gate)
    g = gen(seed + 100)
    x = randn(g, T, H).to(torch.bfloat16) if x is None else x
    logits = 1.5 * randn(g, T, E) if logits is None else logits
    b = 0.2 * torch.rand(E, generator=g) - 0.1 if bias else None
    w = few_weights(p, zero, seed)
    wd = [None if t is None else t.to(dev) for t in w]
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=dev)
    ws = moe.alloc_few_workspace(p, dev)
    args = (moe.Weights(*wd), x.to(dev), logits.to(dev), None if b is None else b.to(dev))
    moe.forward_few(p, *args, out, ws)
    assert moe.get_device_error(ws) == 0
    want, tol = few_reference.few(p, w, x, logits, b)
    ref.check(out, want, ref.half_step(torch.bfloat16)[0] * want.abs() + 1.01 * tol, "out")
    again = torch.empty_like(out)
    moe.forward_few(p, *args, again, ws)
    assert torch.equal(out, again)


FORMATS = [("bf16", False, "static"), ("fp8", False, "static"), ("fp8", False, "dynamic"), ("int4", False, "static"),
           ("int4", True, "static"), ("int4_paired", False, "static"), ("int4_paired", True, "static"),
           ("int8", False, "static"), ("int8", True, "static")]


@gpu
@pytest.mark.parametrize("wdtype,zero,act", FORMATS)
@pytest.mark.parametrize("T", [1, 2, 3, 8])
def test_few_formats(dev, wdtype, zero, act, T):
    run_few(dev, T, 384, 256, 8, 2, zero=zero, wdtype=wdtype, act_scale=act)


@gpu
@pytest.mark.parametrize("wdtype", ["bf16", "fp8", "int4", "int8"])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 128, 128, 1, 1), (8, 128, 128, 4, 4), (5, 1280, 128, 16, 3),
                                       (4, 128, 1408, 16, 8), (1, 2048, 1024, 32, 8), (7, 640, 384, 33, 5)])
def test_few_shapes(dev, wdtype, T, H, I, E, k):
    run_few(dev, T, H, I, E, k, wdtype=wdtype, renormalize=(T % 2 == 0))


@gpu
@pytest.mark.parametrize("wdtype", ["bf16", "fp8", "int4", "int8"])
def test_few_widest_tokens(dev, wdtype):
    run_few(dev, 8, 8192, 128, 4, 2, zero=wdtype.startswith("int"), wdtype=wdtype)
    run_few(dev, 1, 16384, 128, 4, 2, wdtype=wdtype)


@gpu
@pytest.mark.parametrize("wdtype,zero,act", FORMATS)
def test_few_all_tokens_on_the_same_experts(dev, wdtype, zero, act):
    logits = torch.zeros(8, 16)
    logits[:, 5], logits[:, 11] = 3.0, 2.0
    run_few(dev, 8, 256, 640, 16, 2, zero=zero, wdtype=wdtype, act_scale=act, logits=logits)


@gpu
@pytest.mark.parametrize("T", [1, 6])
def test_few_gates(dev, T):
    run_few(dev, T, 256, 128, 64, 8, scoring="sigmoid", n_group=8, topk_group=4, routed_scaling_factor=2.5, bias=True,
            wdtype="int4")
    run_few(dev, T, 256, 128, 64, 6, scoring="sigmoid", n_group=8, topk_group=2, renormalize=False)
    run_few(dev, T, 256, 128, 16, 1, scoring="sigmoid", renormalize=False)
    run_few(dev, T, 256, 128, 40, 32, scoring="softmax")
    run_few(dev, T, 128, 128, 1024, 4, scoring="softmax", renormalize=False)


@gpu
def test_few_ties_nan_logits_and_zero_tokens(dev):
    logits = torch.zeros(4, 16)              # token 0: all equal, the lowest ids win
    logits[1, 5:] = float("nan")             # NaN ranks last
    logits[2] = torch.arange(16.0) % 4       # ties in fours
    logits[3, 7] = 40.0                      # one expert takes all the weight
    x = randn(gen(1), 4, 256).to(torch.bfloat16)
    x[2] = 0
    for wdtype, act in (("bf16", "static"), ("fp8", "dynamic"), ("int4", "static")):
        run_few(dev, 4, 256, 256, 16, 3, wdtype=wdtype, act_scale=act, logits=logits, x=x)
    run_few(dev, 2, 256, 256, 16, 3, wdtype="fp8", act_scale="dynamic", x=torch.zeros(2, 256, dtype=torch.bfloat16))
    # every logit NaN under the sigmoid gate: all scores 0, all weights 0
    run_few(dev, 2, 256, 128, 8, 2, scoring="sigmoid", bias=True, logits=torch.full((2, 8), float("nan")))


@gpu
def test_few_binding_refuses_what_does_not_fit(dev):
    p = moe.problem(2, 256, 128, 8, 2, scoring="sigmoid")
    w = moe.Weights(*[None if t is None else t.to(dev) for t in few_weights(p, False, 1)])
    x, logits = torch.zeros(2, 256, dtype=torch.bfloat16, device=dev), torch.zeros(2, 8, device=dev)
    ws = moe.alloc_few_workspace(p, dev)
    out = torch.empty_like(x)
    moe.forward_few(p, w, x, logits, None, out, ws)
    for bad in (dict(x=x[:1]), dict(x=x.float()), dict(x=x.cpu()), dict(logits=logits[:, :7]), dict(logits=logits.half()),
                dict(bias=torch.zeros(7, device=dev)), dict(out=torch.zeros(2, 512, dtype=torch.bfloat16, device=dev)[:, ::2])):
        with pytest.raises(ValueError):
            moe.forward_few(p, w, **dict(dict(x=x, logits=logits, bias=None, out=out, ws=ws), **bad))
    with pytest.raises(moe.MoEError):
        moe.forward_few(p, w, x, logits, None, out, ws[:256])
    torch.cuda.synchronize()
    assert moe.get_device_error(ws) == 0


@gpu
def test_few_in_a_graph_and_on_another_stream(dev):
    p = moe.problem(3, 512, 256, 8, 2, wdtype="fp8", act_scale="dynamic")
    w = few_weights(p, False, 3)
    wd = moe.Weights(*[None if t is None else t.to(dev) for t in w])
    g = gen(11)
    x, logits = randn(g, 3, 512).to(torch.bfloat16).to(dev), randn(g, 3, 8).to(dev)
    out = torch.empty_like(x)
    ws = moe.alloc_few_workspace(p, dev)
    moe.forward_few(p, wd, x, logits, None, out, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        moe.forward_few(p, wd, x, logits, None, other, ws)
    torch.cuda.synchronize()
    for seed in (1, 2):
        x.copy_(randn(gen(seed), 3, 512).to(torch.bfloat16))
        logits.copy_(randn(gen(seed + 5), 3, 8))
        moe.forward_few(p, wd, x, logits, None, out, ws)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, other)


# ------------------------------------------------------------------ the block that runs them together


@gpu
@pytest.mark.parametrize("T", [0, 1, 8, 9, 40])
@pytest.mark.parametrize("shared", [True, False])
def test_block(dev, T, shared):
    H, I, E, k = 512, 256, 16, 4
    g = gen(T)
    gate = dict(scoring="sigmoid", n_group=4, topk_group=2, routed_scaling_factor=2.5, wdtype="int4")
    p = moe.problem(T, H, I, E, k, **gate)
    w = few_weights(p, False, 7)
    wd = moe.Weights(*[None if t is None else t.to(dev) for t in w])
    nw, rw = (1 + 0.1 * randn(g, H)).to(torch.bfloat16), (0.05 * randn(g, E, H)).to(torch.bfloat16)
    bias = 0.2 * torch.rand(E, generator=g) - 0.1
    sh = None
    if shared:
        rand = lambda *s: torch.rand(s, generator=g)  # noqa: E731
        sh = (codes_of(g, 2 * I, H), rand(2 * I // 128, H // 128) * 4e-4, codes_of(g, H, I), rand(H // 128, I // 128) * 4e-4)
    block = moe.MoEBlock(H, I, E, k, wd, nw.to(dev), rw.to(dev),
                         moe.SharedExpert(*[t.to(dev) for t in sh]) if shared else None, 64, dev,
                         router_bias=bias.to(dev), **gate)
    x, r = randn(g, T, H).to(torch.bfloat16), randn(g, T, H).to(torch.bfloat16)
    out, total = block(x.to(dev), r.to(dev))
    assert block.device_error() == 0
    assert out.shape == (T, H) and total.shape == (T, H)
    if T == 0:
        return
    s, v, _ = ref.norm(x, r, nw, 1e-6)
    rel, tiny = ref.half_step(torch.bfloat16)
    ref.check(total, s, (rel + ref.EPS32) * s.abs() + tiny, "residual")
    y = v.to(torch.bfloat16)
    logits = y.double() @ rw.double().T
    want = torch.zeros(T, H, dtype=torch.float64)
    for t, chosen in enumerate(few_reference.route(p, logits, bias)):
        for e, weight in chosen:
            h = few_reference.matrix(p, w[0], w[2], None, e) @ y[t].double()
            act = h[:I] / (1 + torch.exp(-h[:I])) * h[I:]
            want[t] += weight * (few_reference.matrix(p, w[1], w[3], None, e) @ act)
    if shared:
        big = lambda q, s_: ref.e4m3_values(q) * s_.double().repeat_interleave(128, 0).repeat_interleave(128, 1)  # noqa: E731
        h = v @ big(*sh[:2]).T
        want += h[:, :I] / (1 + torch.exp(-h[:, :I])) * h[:, I:] @ big(*sh[2:]).T
    # two quantisations to e4m3 (2^-4 at most, a fifth of that on average) and bf16 roundings between the stages
    err = float((out.cpu().double() - want).norm() / want.norm())
    assert err <= 4e-2, err


@gpu
@pytest.mark.parametrize("max_tokens,T", [(8, 8), (8, 3), (2, 4), (0, 1)])
def test_block_of_wide_rows(dev, max_tokens, T):
    """H = 16384: the few-token layer takes 4 tokens at most, and the block calls the general one beyond."""
    H, I, E, k = 16384, 128, 4, 2
    g = gen(T)
    w = few_weights(moe.problem(T, H, I, E, k), False, 9)
    nw, rw = torch.ones(H, dtype=torch.bfloat16), (0.01 * randn(g, E, H)).to(torch.bfloat16)
    wd = moe.Weights(*[None if t is None else t.to(dev) for t in w])
    block = moe.MoEBlock(H, I, E, k, wd, nw.to(dev), rw.to(dev), None, max_tokens, dev)
    x = randn(g, T, H).to(torch.bfloat16).to(dev)
    out, _ = block(x)
    assert block.device_error() == 0
    y, logits = torch.empty_like(x), torch.empty((T, E), device=dev)
    moe.add_rms_norm(moe.norm_problem(T, H), x, nw.to(dev), y=y)
    moe.router_logits(moe.router_problem(T, H, E), y, rw.to(dev), logits, moe.alloc_op_workspace(dev))
    want, _ = few_reference.few(moe.problem(T, H, I, E, k), w, y.cpu(), logits.cpu(), None)
    # moe_forward rounds the activations and each expert's output to bf16
    err = float((out.cpu().double() - want).norm() / want.norm())
    assert err <= 1e-2, err


@gpu
@pytest.mark.parametrize("T", [3, 20])
def test_block_in_a_graph_and_on_another_stream(dev, T):
    H, I, E, k = 512, 256, 16, 4
    g = gen(T)
    rand = lambda *s: torch.rand(s, generator=g)  # noqa: E731
    w = few_weights(moe.problem(T, H, I, E, k, wdtype="int8"), False, 7)
    wd = moe.Weights(*[None if t is None else t.to(dev) for t in w])
    sh = (codes_of(g, 2 * I, H), rand(2 * I // 128, H // 128) * 4e-4, codes_of(g, H, I), rand(H // 128, I // 128) * 4e-4)
    block = moe.MoEBlock(H, I, E, k, wd, torch.ones(H, dtype=torch.bfloat16, device=dev),
                         (0.05 * randn(g, E, H)).to(torch.bfloat16).to(dev), moe.SharedExpert(*[t.to(dev) for t in sh]), 64,
                         dev, wdtype="int8")
    x, r = randn(g, T, H).to(torch.bfloat16).to(dev), randn(g, T, H).to(torch.bfloat16).to(dev)
    block(x, r)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, total = block(x, r)
    for seed in (1, 2, 3):
        x.copy_(randn(gen(seed), T, H).to(torch.bfloat16))
        torch.cuda.synchronize()
        want, sums = block(x, r)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(total, sums)
    with torch.cuda.stream(side):
        again, sums = block(x, r)
    side.synchronize()
    assert torch.equal(again, want) and torch.equal(sums, total)
    assert block.device_error() == 0
