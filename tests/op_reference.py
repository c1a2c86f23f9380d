"""Plain 64-bit forms of the operators around the layer, for their tests, with
how far 32-bit arithmetic may be from them.

Every kernel holds its sums in 32 bits.  A sum of n rounded steps over terms t
is within n * 2^-24 * sum |t| of the exact one (2^-23 where a tensor core may
truncate); the number of steps is what each tolerance below counts, and a value
stored in fewer bits is off by at most half a step more.
"""
from __future__ import annotations

import torch

EPS32 = 2.0 ** -24
TRUNC32 = 2.0 ** -23
BLOCK = 128


def half_step(dtype):
    """Largest relative error of one rounding to dtype, and its absolute one among subnormals."""
    f = torch.finfo(dtype)
    return f.eps / 2, f.smallest_normal * f.eps / 2


def e4m3_values(codes):
    """float64 values of e4m3 codes (uint8): sign, 4 exponent bits, 3 mantissa bits, 0x7F / 0xFF NaN."""
    c = codes.cpu().to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * torch.exp2((e - 7).double()))
    v = torch.where((c & 127) == 127, torch.full_like(v, float("nan")), v)
    return torch.where(c > 127, -v, v)


def e4m3_round(v):
    """Nearest e4m3 value (ties to even, saturating at 448) of float64 values."""
    a = v.abs().clamp(max=448.0)
    step = torch.exp2(torch.frexp(a).exponent.clamp(min=-5).double() - 4)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), v)


def check(got, want, tol, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    ok = torch.isnan(want) | ((got - want).abs() <= tol)
    if not bool(ok.all()):
        i = int((~ok).flatten().nonzero()[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} off, first at {i}: {got.flatten()[i]} "
                             f"for {want.flatten()[i]}, tolerance {tol.flatten()[i]}")


def check_quantised(codes, scales, v, dv, block, what):
    """codes [T, n] and one scale per `block` columns, of values v known to within dv."""
    T, n = v.shape
    codes = codes.view(torch.uint8)
    scales = scales.cpu().double().view(T, -1)
    nb = -(-n // block)
    assert scales.shape[1] == nb
    for b in range(nb):
        p, d = v[:, b * block:(b + 1) * block], dv[:, b * block:(b + 1) * block]
        amax, off = p.abs().amax(dim=1), d.amax(dim=1)
        want = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        check(scales[:, b], want, off / 448.0 + 2 * EPS32 * want, f"{what} scale {b}")
        s = scales[:, b:b + 1]
        got = e4m3_values(codes[:, b * block:(b + 1) * block]) * s
        # half a step of e4m3 (2^-4 of the value, 2^-10 among subnormals), the division's and the value's own error
        check(got, p, (2.0 ** -4 + 2.0 ** -20) * p.abs() + 2.0 ** -10 * s + 1.1 * d, f"{what} codes {b}")


# ------------------------------------------------------------------ the operators


def norm(x, residual, weight, eps):
    """(s, v, |error| of v in 32 bits)."""
    s = x.cpu().double()
    if residual is not None:
        s = s + residual.cpu().double()
    v = s / torch.sqrt((s * s).mean(dim=1, keepdim=True) + eps) * weight.cpu().double()
    # the sum's longest chain is at most 64 columns of a thread, 5 shuffles and 8 warps; half of its relative error
    # reaches v, with that of the residual's addition, the division, the root (2 ulp) and two products
    steps = (64 + 5 + 8) / 2 + 1 + 1 + 4 + 2
    return s, v, steps * EPS32 * v.abs()


def router(x, w):
    x, w = x.cpu().double(), w.cpu().double()
    steps = x.shape[1] / 16 + 32  # 16 products a step, then joins
    return x @ w.T, steps * TRUNC32 * (x.abs() @ w.abs().T)


def product(a, a_scale, w, w_scale):
    """(out, |error| in 32 bits) of the block-scaled product."""
    a, w = e4m3_values(a.view(torch.uint8)), e4m3_values(w.view(torch.uint8))
    K, N = a.shape[1], w.shape[0]
    a = a * a_scale.cpu().double().repeat_interleave(BLOCK, dim=1)[:, :K]
    ws = w_scale.cpu().double().view(-1, -(-K // BLOCK))
    w = w * ws.repeat_interleave(BLOCK, dim=1)[:, :K].repeat_interleave(BLOCK, dim=0)[:N]
    steps = -(-K // BLOCK) + 128 / 16 + 16  # one step per block, those within a block, the scales and joins
    return a @ w.T, steps * TRUNC32 * (a.abs() @ w.abs().T)


def swiglu(h, dh):
    n = h.shape[1] // 2
    g, u, dg, du = h[:, :n], h[:, n:], dh[:, :n], dh[:, n:]
    silu = g / (1.0 + torch.exp(-g))
    # the slope of silu stays below 1.1; exp, division and product in 32 bits take 2 + |g| + 4 half ulps
    return silu * u, 1.1 * dg * u.abs() + silu.abs() * du + 1.1 * dg * du + (8 + g.abs()) * TRUNC32 * (silu * u).abs()
