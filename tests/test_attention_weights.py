"""What a row's weights are relative to when they are rounded to 16 bits: small f16 weights keep their bits beside a key
that takes nearly all of the weight."""
import pytest
import torch

from tests import op_reference as ref
from tests.op_reference import EPS32
from tests.test_attention import DT, build, run
from tests.test_operators import dev, gen, lib, randn  # noqa: F401  (fixtures among them)

gpu = pytest.mark.gpu
LIFT = 2.0 ** 7  # the largest weight (8-bit: weight times scale) of a row is at least half of this where it is rounded


def attend(q, k, codes, scales, past, scale, half):
    """One sequence: q [n, Hq, D], k [L, Hkv, D], values codes [L, Hkv, D] * scales [L, Hkv], all float64; new token i
    sees keys [0, past + i].  out, lse and how far each may be from it before out's own rounding.  A product weight *
    scale is off by `half` of itself, or by 2^-25 among f16's subnormals, where the row's largest one is LIFT / 2 or
    more (its scale's power of two is at most twice the scale)."""
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
            # most 128 + LIFT's logarithm and the scales' apart, times log2 e) and exp2
            dw = dx + 4 * EPS32 * ((x - top).abs() + x.abs().amax(dim=1, keepdim=True) + 160) + 8 * EPS32
            steps = (seen / 16 + 64) * 2 * EPS32  # joins and rescalings of the sums
            p = w / total
            part = p * s.abs()
            dl = (p * dw).sum(dim=1, keepdim=True) + steps
            out[i, heads] = (p * s) @ c
            lse[i, heads] = (top + torch.log(total))[:, 0]
            small = 2.0 ** -25 * 2 / LIFT * part.amax(dim=1, keepdim=True) * c.abs().sum(dim=0)
            dout[i, heads] = (part * (2 * dw + half)) @ c.abs() + (dl + steps) * (part @ c.abs()) + small
            dlse[i, heads] = dl[:, 0] + 8 * EPS32 * (1 + lse[i, heads].abs())
    return out, lse, dout, dlse


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
