"""Plain 64-bit forms of the attention half's operators, for their tests, with how far 32-bit arithmetic may be from
them (tests/op_reference.py: a rounded step is off by at most half a step of its type)."""
from __future__ import annotations

import math

import torch

from tests.op_reference import EPS32


def frequencies(rot, theta=10000.0, factor=1.0, original=0, low=1.0, high=1.0):
    """Radians a position of each pair, pair by pair."""
    out = []
    for i in range(rot // 2):
        f = theta ** (-2.0 * i / rot)
        if factor != 1.0:
            seen = original * f / (2.0 * math.pi)
            keep = 0.0 if not original else min(1.0, max(0.0, (seen - low) / (high - low)))
            f = keep * f + (1.0 - keep) * f / factor
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def norm_rotate(x, weight, positions, freq, interleaved, eps, magnitude):
    """x [T, heads, D] -> the normed and rotated heads in float64, and how far float arithmetic may be from them."""
    x = x.double()
    D, rot = x.shape[2], 2 * freq.numel()
    dx = torch.zeros_like(x)
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(dim=2, keepdim=True) + eps) * weight.double()
        # a sum of D squares: 8 steps a lane and up to 5 joins (halved by the root); the mean, eps, root, quotient and
        # two products round once each
        dx = x.abs() * (13 / 2 + 6) * EPS32
    out, dout = x.clone(), dx.clone()
    if rot:
        # angles are reduced in whole numbers of 2^-64 of a turn; their upper half rounds to float (2^-26 of a turn),
        # sine and cosine are off by 2 ulp at most, the magnitude's product by half a one
        angle = positions.double()[:, None] * freq[None, :]
        cos, sin = (f(angle)[:, None, :] * magnitude for f in (torch.cos, torch.sin))
        dturn = abs(magnitude) * (2 * math.pi * 2.0 ** -26 + 5 * EPS32)
        pick = [slice(0, rot, 2), slice(1, rot, 2)] if interleaved else [slice(0, rot // 2), slice(rot // 2, rot)]
        a, b = x[:, :, pick[0]], x[:, :, pick[1]]
        out[:, :, pick[0]], out[:, :, pick[1]] = a * cos - b * sin, b * cos + a * sin
        da, db = dx[:, :, pick[0]], dx[:, :, pick[1]]
        # float64's own angle: position * frequency is off by 2^-53 of itself
        dturn = dturn + (angle.abs() * 2.0 ** -52 * abs(magnitude))[:, None, :]
        both = (a.abs() + b.abs()) * dturn + abs(magnitude) * (da + db + 2 * EPS32 * (a.abs() + b.abs()))
        dout[:, :, pick[0]], dout[:, :, pick[1]] = both, both
    return out, dout


def linear(x, w, bias, act, residual):
    """act(x w^T + bias) + residual in float64, and how far float arithmetic may be from it before the last rounding."""
    x, w = x.cpu().double(), w.cpu().double()
    v = x @ w.T
    # 16 products a step and the joins of partial sums; the tensor core may truncate
    dv = (x.shape[1] / 16 + 32) * 2 * EPS32 * (x.abs() @ w.abs().T)
    if bias is not None:
        v = v + bias.cpu().double()
        dv = dv + EPS32 * v.abs()
    y = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3) if act == "gelu_tanh" else v
    if act in ("silu", "gelu_tanh"):
        out = v / (1 + torch.exp(-y))
        own = (8 + y.abs()) * 4 * EPS32 * out.abs() + 2.0 ** -100
    elif act == "gelu":
        out = v * torch.special.ndtr(v)
        own = 8 * EPS32 * v.abs()  # erf is off by 2 ulp of 1 at most, then 1 + erf, and two products
    else:
        out = torch.where(v < 0, torch.zeros_like(v), v) if act == "relu" else v
        own = torch.zeros_like(v)
    dv = 1.13 * dv + own  # (no activation is steeper than 1.13)
    if residual is not None:
        out = out + residual.cpu().double()
        dv = dv + EPS32 * out.abs()
    return out, dv


def attend(q, k, v, past, scale, p_half_step, unit=None):
    """One sequence: q [n, Hq, D], k and v [L, Hkv, D] in float64; new token i sees keys [0, past + i].  Returns out,
    lse and how far each may be from it before out's own rounding.  p_half_step: half a step of the type that weights
    are rounded to; unit: what weights are relative to where not 1 (8-bit values' largest scale)."""
    n, Hq, D = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    out, dout = torch.zeros(n, Hq, D, dtype=torch.float64), torch.zeros(n, Hq, D, dtype=torch.float64)
    lse, dlse = torch.full((n, Hq), -math.inf, dtype=torch.float64), torch.zeros(n, Hq, dtype=torch.float64)
    for i in range(n):
        seen = past + i + 1
        if seen <= 0:
            continue
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            kk, vv = k[:seen, h], v[:seen, h]
            x = q[i, heads] @ kk.T * scale
            # a score: D products 16 at a time (the tensor core may truncate), then its factors
            dx = ((D / 16 + 2) * 2 * EPS32 * (q[i, heads].abs() @ kk.abs().T) * scale + 4 * EPS32 * x.abs()).amax(dim=1)
            top = x.amax(dim=1, keepdim=True)
            w = torch.exp(x - top)
            l = w.sum(dim=1, keepdim=True)
            p = w / l
            out[i, heads] = p @ vv
            lse[i, heads] = (top + torch.log(l))[:, 0]
            # a weight: its score's error, the exponent's argument (scores times log2 e, the subtraction) and exp2
            dw = dx + 4 * EPS32 * (x - top).abs().amax(dim=1) + 8 * EPS32 + 4 * EPS32 * x.abs().amax(dim=1)
            size = p @ vv.abs()
            steps = seen / 16 + 64  # joins and rescalings of the sums
            # weights under f16's normal range are off by 2^-25 of what they are relative to: 1, or the unit of the
            # 8-bit values' scales (at most twice the largest) times codes of at most 448
            small = (2.0 ** -25 * vv.abs().sum(dim=0)[None, :] if unit is None else
                     torch.full_like(size, 2.0 ** -25 * 2 * unit * 448 * seen)) / l
            dout[i, heads] = (2 * dw[:, None] + p_half_step + 2 * steps * 2 * EPS32) * size + small
            dlse[i, heads] = dw + steps * 2 * EPS32 + 8 * EPS32 * (1 + lse[i, heads].abs())
    return out, lse, dout, dlse

