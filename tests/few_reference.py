"""Plain 64-bit form of the MoE layer for a few tokens, with how far 32-bit sums may be from it."""
from __future__ import annotations

import math

import torch

from tests.op_reference import BLOCK, TRUNC32, e4m3_round, e4m3_values, swiglu


def route(p, logits, bias):
    """Per token [(expert, weight)], by the gate's rule: a NaN logit counts as -inf, ties to the lower expert."""
    out = []
    for row in logits.cpu().double().tolist():
        row = [-math.inf if v != v else v for v in row]
        E = p.E
        if p.scoring == 0:
            top = max(row)
            num = [math.exp(v - top) for v in row]
            z = math.fsum(num)
            score, keys = [v / z for v in num], row
        else:
            score = [1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0 for v in row]
            if bias is not None:
                keys = [a + float(b) for a, b in zip(score, bias.cpu().double())]
            else:
                keys = score if p.n_group else row
        allowed = list(range(E))
        if p.n_group:
            n = E // p.n_group
            best = [sum(sorted(keys[i:i + n])[-2:]) for i in range(0, E, n)]
            groups = sorted(range(p.n_group), key=lambda i: (-best[i], i))[:p.topk_group]
            allowed = [e for e in allowed if e // n in groups]
        ids = sorted(allowed, key=lambda e: (-keys[e], e))[:p.top_k]
        total = math.fsum(score[e] for e in ids)
        inv = (1.0 / total if total > 0 else 0.0) if p.renormalize else 1.0
        out.append([(e, score[e] * inv * p.routed_scaling_factor) for e in ids])
    return out


def matrix(p, codes, scale, zero, e):
    """float64 [rows, K] of expert e; the scale of fp8 experts included."""
    m = codes[e].cpu()
    if p.wdtype == 0:
        return m.double()
    s = scale[e].cpu().double()
    if p.wdtype == 1:
        return e4m3_values(m.view(torch.uint8)) * s
    if p.wdtype == 3:
        v = m.double() if zero is not None else m.view(torch.int8).double()
    else:
        nib = torch.stack([m & 15, m >> 4], dim=2).flatten(1)
        if p.wdtype == 4:  # even K indices in the low half of a word, odd ones in the high
            nib = nib.view(m.shape[0], -1, 2, 4).transpose(2, 3).flatten(1)
        v = nib.double()
        if zero is None:
            v = torch.where(v > 7, v - 16, v)
    if zero is not None:
        v = v - zero[e].cpu().double().repeat_interleave(BLOCK, dim=1)
    return v * s.repeat_interleave(BLOCK, dim=1)


def _quantised(v, dv, scale, rel):
    """e4m3(v / scale) * scale, and how far it may move where v is off by dv and scale by the factor 1 + rel."""
    d = dv + v.abs() * rel
    q = e4m3_round(v / scale) * scale
    lo, hi = e4m3_round((v - d) / scale) * scale, e4m3_round((v + d) / scale) * scale
    return q, torch.maximum((hi - q).abs(), (q - lo).abs()) + q.abs() * rel


def few(p, w, x, logits, bias):
    """(out, tolerance before the rounding to bf16): w = (w13, w2, w13_scale, w2_scale, a1, a2, w13_zero, w2_zero)."""
    w13, w2, s13, s2, a1, a2, z13, z2 = w
    T, I = p.T, p.I
    routes = route(p, logits, bias)
    x = x.cpu().double()
    fp8 = p.wdtype == 1
    if fp8:
        if a1 is None:
            m = x.abs().max().float() if T else torch.zeros(())
            a1 = m / 448.0 if float(m) > 0 else torch.ones(())
        a1 = float(a1.float().cpu())  # its 32-bit value: x / a1 then meets the same borders
        x, dx = e4m3_round((x.float() / a1).double()) * a1, None
    steps_h, steps_i = p.H / 16 + 48, I / 16 + 48  # 16 products a step, then group scales and joins
    chosen = sorted({e for r in routes for e, _ in r})
    act = {}
    for e in chosen:
        m = matrix(p, w13, s13, z13, e)
        for t in range(T):
            if e in dict(routes[t]):
                h = (m @ x[t])[None]
                dh = (steps_h * TRUNC32 * (m.abs() @ x[t].abs()))[None]
                act[t, e] = tuple(v[0] for v in swiglu(h, dh))
    if fp8:
        rel = 4 * TRUNC32
        if a2 is None:
            top = max(act.values(), key=lambda v: float(v[0].abs().max()))
            i = int(top[0].abs().argmax())
            amax = float(top[0][i].abs())
            scale = amax / 448.0 if amax > 0 else 1.0
            rel += max(float(d.max()) for _, d in act.values()) / amax if amax > 0 else 0.0
        else:
            scale = float(a2.float().cpu())
        act = {at: _quantised(v, d, scale, rel) for at, (v, d) in act.items()}
    out = torch.zeros((T, p.H), dtype=torch.float64)
    tol = torch.zeros_like(out)
    for e in chosen:
        m = matrix(p, w2, s2, z2, e)
        for t in range(T):
            for f, weight in routes[t]:
                if f == e:
                    v, d = act[t, e]
                    out[t] += weight * (m @ v)
                    size = m.abs() @ v.abs()
                    # the gate's weight is within 16 half ulps times the logits' size of its own
                    tol[t] += abs(weight) * (m.abs() @ d + (steps_i + p.top_k + 64) * TRUNC32 * size)
    return out, tol
