"""moe_linear: refusals (no GPU), and the operator against its plain 64-bit form."""
import ctypes
import math

import pytest
import torch

import mixture_experts_layer_gate_gb300 as moe
from tests import attention_reference as att
from tests import op_reference as ref
from tests.test_operators import dev, far, gen, lib, randn, wide  # noqa: F401  (fixtures among them)

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = 4096  # an address that is never dereferenced: the checks come before any launch


def call(lib, p, x=P, xs=None, w=P, ws_=None, bias=None, r=None, rs=None, out=P, os=None, ws=P, ws_bytes=256):
    K, N = (p.K, p.N) if p is not None else (0, 0)
    own = lambda s, n: n if s is None else s  # noqa: E731
    return lib.moe_linear(ctypes.byref(p) if p is not None else None, x, own(xs, K), w, own(ws_, K), bias, r, own(rs, N),
                          out, own(os, N), ws, ws_bytes, None)


def test_refusals(lib):
    assert ctypes.sizeof(moe.LinearProblem) == 24
    p = moe.linear_problem(5, 96, 64)
    assert call(lib, None) == INVALID
    for kw in (dict(x=None), dict(w=None), dict(out=None), dict(x=P + 8), dict(w=P + 2), dict(out=P + 1), dict(xs=56),
               dict(xs=68), dict(ws_=60), dict(os=95), dict(r=P + 1), dict(r=P + 2, rs=95), dict(bias=P + 1),
               dict(r=P, rs=104)):
        assert call(lib, p, **kw) == INVALID, kw
    for n, v in (("M", -1), ("N", -1), ("K", 0), ("K", 60), ("dtype", 2), ("dtype", -1), ("out_dtype", 3),
                 ("activation", 5), ("activation", -1)):
        p = moe.linear_problem(5, 96, 64)
        setattr(p, n, v)
        assert call(lib, p) == INVALID, n
    for n in ("M", "N"):
        p = moe.linear_problem(5, 96, 64)
        setattr(p, n, (1 << 22) + 1)
        assert call(lib, p) == UNSUPPORTED
    p = moe.linear_problem(5, 96, 64)
    assert call(lib, p, ws=None) == WORKSPACE and call(lib, p, ws_bytes=255) == WORKSPACE
    assert call(lib, moe.linear_problem(0, 96, 64)) == 0 and call(lib, moe.linear_problem(5, 0, 64)) == 0
    with pytest.raises(KeyError):
        moe.linear_problem(1, 1, 8, activation="swish")


CASES = [  # M, N, K, dtype, out, bias, act, residual, pad of the rows
    (1, 6144, 4096, "bf16", "bf16", True, "none", False, 0),
    (1, 1, 8, "f16", "f32", True, "silu", True, 8),
    (8, 333, 520, "bf16", "f32", False, "gelu", True, 0),
    (9, 16, 40, "f16", "f16", True, "gelu_tanh", False, 8),
    (16, 1000, 2056, "bf16", "bf16", True, "relu", True, 8),
    (17, 100, 72, "bf16", "bf16", True, "none", True, 0),
    (64, 1536, 4096, "f16", "f16", True, "silu", True, 0),
    (77, 1001, 1104, "bf16", "f32", True, "gelu", True, 8),
    (128, 2048, 512, "bf16", "bf16", True, "gelu_tanh", False, 0),
    (129, 4097, 136, "f16", "f16", False, "relu", True, 8),
    (300, 2504, 1000, "bf16", "bf16", True, "none", True, 8),
    (513, 8200, 264, "f16", "f16", True, "gelu", True, 0),
    (1024, 4096, 2048, "bf16", "bf16", True, "silu", True, 0),
    (2000, 4104, 1544, "bf16", "f32", True, "none", True, 0),
    (1111, 3000, 96, "bf16", "f16", True, "gelu_tanh", True, 0),
]


@gpu
@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
@pytest.mark.parametrize("in_place", [False, True])
def test_matches_plain(dev, case, in_place):
    M, N, K, dtype, out, bias, act, residual, pad = case
    if in_place and not residual:
        pytest.skip("no residual to write over")
    dt, odt, g = DT[dtype], DT[out], gen(M + N + K)
    x, w = randn(g, M, K).to(dt), (randn(g, N, K) * 3 * K ** -0.5).to(dt)
    b = randn(g, N).to(dt) if bias else None
    r = (randn(g, M, N) * 3).to(odt) if residual else None
    rd = wide(r, pad, dev) if residual else None
    od = rd if in_place else wide(torch.full((M, N), 7.0).to(odt), pad, dev, fill=7.0)
    ws = moe.alloc_op_workspace(dev)
    p = moe.linear_problem(M, N, K, dtype=dtype, out_dtype=out, activation=act)
    moe.linear(p, wide(x, pad, dev), wide(w, pad, dev), od, ws, bias=b.to(dev) if bias else None, residual=rd)
    assert moe.get_device_error(ws) == 0
    want, dv = att.linear(x, w, b, act, r)
    rel, tiny = ref.half_step(odt)
    ref.check(od, want, dv + (want.abs() + dv) * rel + tiny, "out")
    if pad and not in_place:  # what lies between the rows stays
        base = torch.as_strided(od, (M, N + 2 * pad), (od.stride(0), 1), od.storage_offset() - pad)
        assert bool((base[:, :pad] == 7.0).all()) and bool((base[:, N + pad:] == 7.0).all())


@gpu
@pytest.mark.parametrize("M", [3, 12, 40, 600])
def test_unaligned_rows_and_bias(dev, M):
    """out, residual and bias at any element."""
    N, K, g = 259, 64, gen(M)
    x, w = randn(g, M, K).bfloat16(), randn(g, N, K).bfloat16()
    b, r = randn(g, N + 1).bfloat16(), randn(g, M, N).bfloat16()
    od = wide(torch.zeros(M, N).bfloat16(), 3, dev)
    moe.linear(moe.linear_problem(M, N, K), x.to(dev), w.to(dev), od, moe.alloc_op_workspace(dev), bias=b.to(dev)[1:],
               residual=wide(r, 5, dev))
    want, dv = att.linear(x, w, b[1:], "none", r)
    rel, tiny = ref.half_step(torch.bfloat16)
    ref.check(od, want, dv + (want.abs() + dv) * rel + tiny, "out")


@gpu
@pytest.mark.parametrize("M", [2, 200])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh", "relu"])
def test_far_values(dev, M, act):
    """Sums far on both sides of zero, infinite ones and NaN."""
    N, K = 64, 32
    x, w = torch.zeros(M, K).bfloat16(), torch.zeros(N, K).bfloat16()
    x[:, 0] = 1
    w[:, 0] = torch.linspace(-110, 110, N).bfloat16()
    w[5, 0], w[6, 0], w[7, 0], w[8, 0] = math.inf, -math.inf, math.nan, -1e30
    x[1, 0] = -1
    od = torch.empty(M, N, device=dev)
    moe.linear(moe.linear_problem(M, N, K, out_dtype="f32", activation=act), x.to(dev), w.to(dev), od,
               moe.alloc_op_workspace(dev))
    # (a column with an infinity: 0 * inf only where x is 0 there, which it is not)
    want, dv = att.linear(x, w, None, act, None)
    got = od.cpu().double()
    finite = torch.isfinite(want)
    assert bool(((got - want).abs() <= dv + want.abs() * 2.0 ** -23 + 1e-35)[finite].all())
    assert bool(got[:, 7].isnan().all())
    if act in ("none", "relu"):
        assert torch.equal(got[:, 5:7][0], want[:, 5:7][0])


@gpu
def test_in_a_graph_and_on_a_stream(dev):
    g = gen(1)
    M, N, K = 40, 320, 256
    x, w, r = (t.to(dev) for t in (randn(g, M, K).bfloat16(), randn(g, N, K).bfloat16(), randn(g, M, N).bfloat16()))
    p, ws = moe.linear_problem(M, N, K), moe.alloc_op_workspace(dev)
    want, out = torch.empty_like(r), torch.empty_like(r)
    moe.linear(p, x, w, want, ws, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.linear(p, x, w, out, ws, residual=r, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.linear(p, x, w, out, ws, residual=r)
    x.mul_(2)
    graph.replay()
    moe.linear(p, x, w, want, ws, residual=r)
    assert torch.equal(out, want)


@gpu
def test_python_refusals(dev):
    M, N, K = 2, 16, 64
    p, ws = moe.linear_problem(M, N, K), moe.alloc_op_workspace(dev)
    x, w, o = (torch.zeros(s, dtype=torch.bfloat16, device=dev) for s in ((M, K), (N, K), (M, N)))
    for bad in (dict(x=x.half()), dict(x=x.cpu()), dict(x=x[:1]), dict(w=w[:, :32]), dict(out=o.float()),
                dict(bias=torch.zeros(N, device=dev)), dict(bias=o[0, :8]), dict(residual=o.float()),
                dict(x=x.t().contiguous().t())):
        kw = dict(x=x, w=w, out=o, bias=None, residual=None)
        kw.update(bad)
        with pytest.raises(ValueError):
            moe.linear(p, kw["x"], kw["w"], kw["out"], ws, bias=kw["bias"], residual=kw["residual"])


PAIR_CASES = [  # of CTA pairs that share 128 columns: a few hundred rows, last tiles of few rows and columns
    (1000, 2300, 264, "bf16", "bf16", True, "silu", True, 0),
    (1100, 1901, 520, "f16", "f32", True, "none", True, 8),
    (700, 3001, 200, "bf16", "bf16", False, "gelu", False, 8),
    (257, 4100, 136, "f16", "f16", True, "relu", True, 0),
]


@gpu
@pytest.mark.parametrize("case", PAIR_CASES, ids=["-".join(map(str, c)) for c in PAIR_CASES])
def test_pairs_of_narrow_tiles(dev, case):
    for in_place in (False, True) if case[7] else (False,):
        test_matches_plain(dev, case, in_place)
