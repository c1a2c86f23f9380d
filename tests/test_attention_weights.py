"""What a row's weights are relative to when they are rounded to 16 bits: nothing that the row does not see reaches it
through a value scale of an 8-bit cache, a seen key counts by its weight and its scale together, and small f16 weights
keep their bits beside a key that takes nearly all of the weight."""
import math

import pytest
import torch

from tests import op_reference as ref
from tests.op_reference import EPS32
from tests.test_attention import DT, build, run
from tests.test_operators import dev, gen, lib, randn  # noqa: F401  (fixtures among them)

gpu = pytest.mark.gpu
# the largest weight (8-bit: weight times scale) of a row is at least this where it is rounded to f16
LEAST, LEAST_SCALED = 2.0 ** 7, 2.0 ** 3


def attend(q, k, codes, scales, past, scale, half, least=LEAST):
    """One sequence: q [n, Hq, D], k [L, Hkv, D], values codes [L, Hkv, D] * scales [L, Hkv], all float64; new token i
    sees keys [0, past + i].  out, lse and how far each may be from it before out's own rounding.  A product weight *
    scale is off by `half` of itself, or by 2^-25 among f16's subnormals, where the row's largest one is `least` or more."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, dout = (torch.zeros(n, Hq, D, dtype=torch.float64) for _ in range(2))
    lse, dlse = (torch.zeros(n, Hq, dtype=torch.float64) for _ in range(2))
    for i in range(n):
        seen = past + i + 1
        for h in range(k.shape[1]):
            heads = slice(h * G, (h + 1) * G)
            kk, c, s = k[:seen, h], codes[:seen, h], scales[:seen, h]
            x = q[i, heads] @ kk.T * scale
            # a score: D products 16 at a time (the tensor core may truncate), then its factors; of each key by itself
            dx = (D / 16 + 2) * 2 * EPS32 * (q[i, heads].abs() @ kk.abs().T) * scale + 4 * EPS32 * x.abs()
            top = x.amax(dim=1, keepdim=True)
            w = torch.exp(x - top)
            total = w.sum(dim=1, keepdim=True)
            # a weight: its score's error, the exponent's argument in float (scores and what they are relative to, at
            # most the scales' logarithm and 15 apart, times log2 e) and exp2
            dw = dx + 4 * EPS32 * ((x - top).abs() + x.abs().amax(dim=1, keepdim=True) + 160) + 8 * EPS32
            steps = (seen / 16 + 64) * 2 * EPS32  # joins and rescalings of the sums
            p = w / total
            part = p * s.abs()
            dl = (p * dw).sum(dim=1, keepdim=True) + steps
            out[i, heads] = (p * s) @ c
            lse[i, heads] = (top + torch.log(total))[:, 0]
            small = 2.0 ** -25 / least * part.amax(dim=1, keepdim=True) * c.abs().sum(dim=0)
            dout[i, heads] = (part * (2 * dw + half)) @ c.abs() + (dl + steps) * (part @ c.abs()) + small
            dlse[i, heads] = dl[:, 0] + 8 * EPS32 * (1 + lse[i, heads].abs())
    return out, lse, dout, dlse


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


SIZES = [(4, 200), (8, 130), (3, 6000), (100, 300), (200, 200), (130, 5000)]


@gpu
@pytest.mark.parametrize("power", [16, 30, 60, 120])
@pytest.mark.parametrize("new,L", SIZES)
def test_unseen_value_scale(dev, new, L, power):
    """A finite value scale of a later new token, 2^16 to 2^120 times the others', leaves the rows before it their bits."""
    problem, args, *_ = build(dev, [new], [L], 4, 2, 128, "bf16", "e4m3", 16, "head", spare=0)
    clean, clean_lse, _ = run(problem, args, dev)
    at, first = L - 1 - new // 2, new - 1 - new // 2  # the key, and the first new token that sees it
    page, place = int(args["page_table"][0, at // 16]), at % 16
    for sign in (1, -1):
        broken = dict(args, v_scale=args["v_scale"].clone())
        broken["v_scale"][page, :, place] *= sign * 2.0 ** power
        out, lse, _ = run(problem, broken, dev)
        assert same(out[:first], clean[:first]) and same(lse[:first], clean_lse[:first])
        assert bool(torch.isfinite(out).all()) and not same(out[first:], clean[first:])


@gpu
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("new,L", SIZES)
def test_unseen_value_scale_that_is_not_finite(dev, new, L, bad):
    problem, args, *_ = build(dev, [new], [L], 4, 2, 128, "bf16", "e4m3", 16, "head", spare=0)
    clean, clean_lse, _ = run(problem, args, dev)
    at, first = L - 1 - new // 2, new - 1 - new // 2
    broken = dict(args, v_scale=args["v_scale"].clone())
    broken["v_scale"][int(args["page_table"][0, at // 16]), 1, at % 16] = bad
    out, lse, _ = run(problem, broken, dev)
    assert same(out[:first], clean[:first]) and same(lse[:first], clean_lse[:first])
    # heads 2 and 3 read value head 1, whose weights, and so the logarithm of their sum, do not depend on it
    out, clean = out.view(new, 4, 128), clean.view(new, 4, 128)
    assert same(out[:, :2], clean[:, :2]) and not bool(torch.isfinite(out[first:, 2:]).any())
    assert same(lse[:, :2], clean_lse[:, :2])
    assert bool(((lse - clean_lse).abs() <= 2.0 ** -17 * (1 + clean_lse.abs())).all())


def scaled_case(dev, new, L, change):
    """Four query heads over two key heads of 128, e4m3; change(k codes, v codes, k scales, v scales, q) alters keys in
    the sequence's order, [L, Hkv, D] and [L, Hkv]."""
    problem, args, q, keys, cu, _ = build(dev, [new], [L], 4, 2, 128, "bf16", "e4m3", 16, "head", spare=0)
    pages = args["page_table"][0, :-(-L // 16)].long()

    def rows(name):
        t = args[name + "_cache"][pages].reshape(-1, 2, 128)[:L].cpu()
        return t, args[name + "_scale"][pages].transpose(1, 2).reshape(-1, 2)[:L].cpu()

    (kc, ks), (vc, vs) = rows("k"), rows("v")
    change(kc, vc, ks, vs, q)
    for name, codes, scales in (("k", kc, ks), ("v", vc, vs)):
        cache, scale = args[name + "_cache"].clone(), args[name + "_scale"].clone()
        j = torch.arange(L, device=dev)
        cache[pages[j // 16], j % 16] = codes.to(dev)
        scale[pages[j // 16], :, j % 16] = scales.to(dev)
        args[name + "_cache"], args[name + "_scale"] = cache, scale
    args["q"] = q.to(dev)
    problem.scale = 128 ** -0.5
    out, lse, ws = run(problem, args, dev)
    k = ref.e4m3_values(kc) * ks.double()[..., None]
    want, wl, dout, dl = attend(q.double().view(new, 4, 128), k, ref.e4m3_values(vc), vs.double(), L - new, problem.scale,
                                2.0 ** -11, LEAST_SCALED)
    rel, tiny = ref.half_step(torch.bfloat16)
    ref.check(out.reshape(new, 4, 128), want, dout + (want.abs() + dout) * rel + tiny, "out")
    ref.check(lse, wl, dl, "lse")


@gpu
@pytest.mark.parametrize("factor", [1e6, 1e9])
@pytest.mark.parametrize("new,L", SIZES)
def test_large_scale_of_next_to_no_weight(dev, new, L, factor):
    """A seen key some 60 nats below the others, whose value scale is a million times theirs and more, costs them nothing."""
    def change(kc, vc, ks, vs, q):
        q.view(new, 4, 128)[:, :, 0] = 8.0
        kc[:, :, 0] = 0
        kc[L // 3] = 0
        kc[L // 3, :, 0] = 0xF3  # -176
        ks[L // 3] = 0.5         # -88 * 8 / sqrt(128) = -62
        vs[L // 3] *= factor

    scaled_case(dev, new, L, change)


@gpu
@pytest.mark.parametrize("new,L", SIZES)
def test_scales_over_the_whole_range(dev, new, L):
    """Scales from 2^-60 to 2^30 along the keys, negative ones and zeros among them."""
    def change(kc, vc, ks, vs, q):
        g = gen(new + L)
        vs.copy_(torch.exp2(torch.rand(L, 2, generator=g) * 90 - 60) * torch.where(torch.rand(L, 2, generator=g) < 0.3, -1.0, 1.0))
        vs[torch.rand(L, 2, generator=g) < 0.1] = 0.0

    scaled_case(dev, new, L, change)


@gpu
@pytest.mark.parametrize("power", [-70, 90])
@pytest.mark.parametrize("new,L", [(4, 200), (100, 300)])
def test_scales_far_from_one(dev, new, L, power):
    def change(kc, vc, ks, vs, q):
        vs.mul_(2.0 ** power)

    scaled_case(dev, new, L, change)


@gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("sink", [7.0, 12.0, 18.0])
@pytest.mark.parametrize("new", [1, 6, 40])
def test_small_weights_beside_a_sink(dev, new, sink, dtype):
    """The first key takes nearly all of the weight and its value is zero: the output is what the others add."""
    L, D, Hq, Hkv = 8193 + new, 64, 4, 2
    problem, args, q, keys, cu, _ = build(dev, [new], [L], Hq, Hkv, D, dtype, dtype, 64, "head", spare=0)
    problem.scale = D ** -0.5
    k, v = keys[0]
    g = gen(new)
    q.copy_(0.1 * randn(g, new, Hq * D))
    q.view(new, Hq, D)[:, :, 0] = 8.0
    k[:, :, 0] = 0.0
    k[0], v[0] = 0.0, 0.0
    k[0, :, 0] = sink / (8.0 * problem.scale)
    v.copy_(v.abs())
    k, v = k.to(DT[dtype]), v.to(DT[dtype])
    pages, j = args["page_table"][0, :-(-L // 64)].long(), torch.arange(L, device=dev)
    for name, t in (("k_cache", k), ("v_cache", v)):
        args[name] = args[name].clone()
        args[name][pages[j // 64], j % 64] = t.to(dev)
    args["q"] = q.to(dev)
    out, lse, _ = run(problem, args, dev)
    half, _ = ref.half_step(DT[dtype])
    ones = torch.ones(L, Hkv, dtype=torch.float64)
    want, wl, dout, dl = attend(q.double().view(new, Hq, D), k.double(), v.double(), ones, L - new, problem.scale, half)
    assert float(torch.exp(sink - wl.double()).min()) > 0.05  # (the first key's share)
    rel, tiny = ref.half_step(DT[dtype])
    ref.check(out.reshape(new, Hq, D), want, dout + (want.abs() + dout) * rel + tiny, "out")
    ref.check(lse, wl, dl, "lse")


@gpu
@pytest.mark.parametrize("new", [3, 40])
def test_scores_that_vanish(dev, new):
    """Queries and a scale so small that their product is under float's range: every weight is the same, masked keys none."""
    problem, args, q, keys, cu, _ = build(dev, [new], [300], 4, 2, 64, "bf16", "e4m3", 16, "token", spare=0)
    problem.scale = 2.0 ** -60
    q.mul_(2.0 ** -105)
    args["q"] = q.to(dev)
    out, lse, _ = run(problem, args, dev)
    rel, tiny = ref.half_step(torch.bfloat16)
    for i in range(new):
        n = 300 - new + i + 1
        want = keys[0][1][:n].mean(dim=0).repeat_interleave(2, dim=0)
        size = keys[0][1][:n].abs().mean(dim=0).repeat_interleave(2, dim=0)
        tol = size * (2.0 ** -11 + 2.0 ** -16) + want.abs() * rel + tiny  # a weight's rounding, the sums'
        ref.check(out[i].reshape(4, 64), want, tol, "out")
        assert bool(((lse[i].cpu().double() - math.log(n)).abs() < 2.0 ** -18).all())
