"""The operators around the mixture-of-experts layer, their plain forms and the cases they are measured on.

One pre-norm MoE block of a decoder is: add the residual and normalise (moe_add_rms_norm, optionally to 8-bit codes),
score the experts (moe_router_logits), run the routed experts (moe_forward, or moe_forward_few for a few tokens) and
the shared expert or a dense layer in block-scaled 8-bit floating point (moe_gemm_fp8_block_swiglu, then
moe_gemm_fp8_block).  Each case is one of these calls.

With `own` false, run() computes a case in elementary torch operations in 32 bits; with `own` true it calls this
repository's package.
"""
import math

import torch

own = False

BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    """Sizes are those of the DeepSeek-V3 layer (H = 7168, I = 2048, E = 256), the Mixtral-8x7B and the
    Qwen2-57B-A14B layers, and generic odd ones."""
    return [
        # --- residual + RMS norm
        # decode: one token's residual, normed to bf16 (router, routed experts) and to 8-bit codes (shared expert)
        dict(name="norm decode", op="norm", T=1, H=7168, dtype="bf16", wdtype="bf16", residual=True, y=True,
             quant="block", pad=0),
        # a ragged batch of odd rows inside wider rows, no residual, one scale per token
        dict(name="norm odd", op="norm", T=333, H=2571, dtype="f16", wdtype="f32", residual=False, y=True,
             quant="token", pad=37),
        # prefill: the whole block input at once
        dict(name="norm prefill", op="norm", T=4096, H=7168, dtype="bf16", wdtype="bf16", residual=True, y=True,
             quant="block", pad=0),
        # --- router scores
        # decode: one token against 256 experts
        dict(name="router decode", op="router", T=1, H=7168, E=256, dtype="bf16", pad=0),
        # a ragged batch, a small expert count
        dict(name="router ragged", op="router", T=333, H=3584, E=60, dtype="f16", pad=8),
        # prefill
        dict(name="router prefill", op="router", T=4096, H=7168, E=256, dtype="bf16", pad=0),
        # --- 8-bit product with a scale per block of 128
        # decode: the shared expert's gate and up projections with SwiGLU, one token
        dict(name="fp8 swiglu decode", op="swiglu", M=1, N=2048, K=7168, out="e4m3", pad=0),
        # a ragged batch into an odd width, a depth that ends inside a block
        dict(name="fp8 ragged", op="gemm", M=77, N=1001, K=1104, out="f32", pad=16),
        # prefill: the shared expert's gate and up projections with SwiGLU, then its down projection
        dict(name="fp8 swiglu prefill", op="swiglu", M=4096, N=2048, K=7168, out="e4m3", pad=0),
        dict(name="fp8 down prefill", op="gemm", M=4096, N=7168, K=2048, out="bf16", pad=0),
        # --- the whole layer for a few tokens
        # single-stream decode, DeepSeek-V3 routing over int4 experts
        dict(name="few dsv3 int4", op="few", T=1, H=7168, I=2048, E=256, k=8, wdtype="int4_paired", zero=False,
             scoring="sigmoid", renorm=True, bias=True, n_group=8, topk_group=4, factor=2.5, act="static"),
        # a small batch of streams, Mixtral routing over bf16 experts
        dict(name="few mixtral bf16", op="few", T=8, H=4096, I=14336, E=8, k=2, wdtype="bf16", zero=False,
             scoring="softmax", renorm=True, bias=False, n_group=0, topk_group=0, factor=1.0, act="static"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "router", "swiglu", "gemm", "few"])
    if op == "norm":
        H = _log(rng, 8, 8192)
        if rng.random() < 0.6:
            H = max(8, H // 8 * 8)
        return dict(op=op, T=_log(rng, 1, 4096), H=H, dtype=rng.choice(["bf16", "f16", "f32"]),
                    wdtype=rng.choice(["f32", "same"]), residual=rng.random() < 0.6, y=True,
                    quant=rng.choice(["none", "block", "token"]), pad=rng.choice([0, 0, 8, 3]))
    if op == "router":
        return dict(op=op, T=_log(rng, 1, 4096), H=_log(rng, 16, 896) * 8, E=_log(rng, 2, 512),
                    dtype=rng.choice(["bf16", "f16"]), pad=rng.choice([0, 8]))
    if op == "swiglu":
        return dict(op=op, M=_log(rng, 1, 4096), N=rng.randint(1, 16) * 128, K=_log(rng, 8, 448) * 16, out="e4m3",
                    pad=rng.choice([0, 16]))
    if op == "gemm":
        return dict(op=op, M=_log(rng, 1, 4096), N=_log(rng, 16, 7168), K=_log(rng, 8, 448) * 16,
                    out=rng.choice(["bf16", "f16", "f32"]), pad=rng.choice([0, 16]))
    wdtype = rng.choice(["bf16", "fp8", "fp8", "int4", "int4_paired", "int8"])
    k = rng.choice([1, 2, 3, 6, 8])
    T = rng.randint(1, 8)
    E = max(k, rng.choice([4, 8, 13, 16, 64, 128, 256]))
    H = _log(rng, 2, 40) * 128
    most = 1_500_000_000 // (E * H * 3)  # weights of at most 1.5 G values, as the largest listed layer
    most = min(most, 1_000_000_000 // (T * k * H * 3))  # and no more read than there
    I = max(1, min(_log(rng, 1, 64), most // 128)) * 128
    scoring = rng.choice(["softmax", "sigmoid"])
    groups = scoring == "sigmoid" and E % 8 == 0 and E >= 16 and rng.random() < 0.6
    topk_group = max(2, -(-k // (E // 8))) if groups else 0
    return dict(op=op, T=T, H=H, I=I, E=E, k=k, wdtype=wdtype,
                zero=wdtype.startswith("int") and rng.random() < 0.5, scoring=scoring, renorm=rng.random() < 0.6,
                bias=scoring == "sigmoid" and rng.random() < 0.6, n_group=8 if groups else 0, topk_group=topk_group,
                factor=rng.choice([1.0, 2.5]), act=rng.choice(["static", "dynamic"]) if wdtype == "fp8" else "static")


# ------------------------------------------------------------------------------------------------ inputs


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rows(v, pad):
    """The rows of v inside rows that are `pad` values longer, as a slice of a wider tensor."""
    if not pad:
        return v
    wide = torch.zeros((v.shape[0], v.shape[1] + pad), dtype=v.dtype, device=v.device)
    wide[:, :v.shape[1]] = v
    return wide[:, :v.shape[1]]


def _e4m3(v):
    """Values of any size in e4m3: rounded to nearest even, saturating."""
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _codes(g, *shape):
    """e4m3 codes as a quantised normal tensor has them."""
    flat = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    for part in flat.view(-1).split(1 << 28):
        part.copy_(_e4m3(torch.randn(part.shape, generator=g, device="cuda") * 100.0))
    return flat


def _gate(case):
    return dict(scoring=case["scoring"], renormalize=case["renorm"], n_group=case["n_group"],
                topk_group=case["topk_group"], routed_scaling_factor=case["factor"], wdtype=case["wdtype"],
                act_scale=case["act"])


def prepare(case, seed):
    """Inputs of one call, its output buffers and (own) the problem, weights and workspace that a program keeps."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    s = dict(case=case)
    empty = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    op = case["op"]
    if op == "norm":
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        wdt = dt if case["wdtype"] == "same" else DTYPES[case["wdtype"]]
        s["x"] = _rows(_randn(g, T, H).to(dt), case["pad"])
        s["residual"] = _rows((_randn(g, T, H) * 3.0).to(dt), case["pad"]) if case["residual"] else None
        s["weight"] = (1.0 + 0.1 * _randn(g, H)).to(wdt)
        s["eps"] = 1e-6
        s["residual_out"] = empty(T, H, dtype=dt) if case["residual"] else None
        s["y"] = empty(T, H, dtype=dt) if case["y"] else None
        nb = {"none": 0, "block": -(-H // BLOCK), "token": 1}[case["quant"]]
        s["codes"] = empty(T, H, dtype=torch.float8_e4m3fn) if nb else None
        s["scales"] = empty(T, nb, dtype=torch.float32) if nb else None
        if own:
            import mixture_experts_layer_gate_gb300 as moe
            s["problem"] = moe.norm_problem(T, H, dtype=case["dtype"],
                                            weight_dtype=case["dtype"] if case["wdtype"] == "same" else case["wdtype"],
                                            eps=s["eps"], quant=case["quant"])
    elif op == "router":
        T, H, E, dt = case["T"], case["H"], case["E"], DTYPES[case["dtype"]]
        s["x"] = _rows(_randn(g, T, H).to(dt), case["pad"])
        s["w"] = (_randn(g, E, H) * 0.02).to(dt)
        s["logits"] = empty(T, E, dtype=torch.float32)
        if own:
            import mixture_experts_layer_gate_gb300 as moe
            s["problem"] = moe.router_problem(T, H, E, dtype=case["dtype"])
            s["ws"] = moe.alloc_op_workspace(s["x"].device)
    elif op in ("gemm", "swiglu"):
        M, N, K = case["M"], case["N"], case["K"]
        rows = 2 * N if op == "swiglu" else N
        s["a"] = _rows(_codes(g, M, K), case["pad"])
        s["w"] = _codes(g, rows, K)
        kb, nb = -(-K // BLOCK), -(-rows // BLOCK)
        s["a_scale"] = torch.rand((M, kb), generator=g, device="cuda") * 0.01 + 0.002
        s["w_scale"] = torch.rand((nb, kb), generator=g, device="cuda") * 2e-4 + 1e-4
        if op == "gemm":
            s["out"] = empty(M, N, dtype=DTYPES[case["out"]])
        else:
            s["codes"] = empty(M, N, dtype=torch.float8_e4m3fn)
            s["scales"] = empty(M, N // BLOCK, dtype=torch.float32)
        if own:
            import mixture_experts_layer_gate_gb300 as moe
            s["problem"] = moe.fp8_gemm_problem(M, N, K, out_dtype=case["out"] if op == "gemm" else "bf16")
            s["ws"] = moe.alloc_op_workspace(s["a"].device)
    else:
        T, H, I, E, wd = case["T"], case["H"], case["I"], case["E"], case["wdtype"]
        s["x"] = _randn(g, T, H).to(torch.bfloat16)
        s["logits"] = _randn(g, T, E) * 1.5
        s["bias"] = torch.rand((E,), generator=g, device="cuda") * 0.2 - 0.1 if case["bias"] else None
        s["w13_scale"] = s["w2_scale"] = s["w13_zero"] = s["w2_zero"] = s["a1"] = s["a2"] = None
        u = lambda *shape: torch.rand(shape, generator=g, device="cuda")  # noqa: E731
        if wd == "bf16":
            for name, shape in (("w13", (E, 2 * I, H)), ("w2", (E, H, I))):
                s[name] = empty(*shape, dtype=torch.bfloat16)
                for part in s[name]:
                    part.copy_(_randn(g, *part.shape) * 0.02)
        elif wd == "fp8":
            s["w13"], s["w2"] = _codes(g, E, 2 * I, H), _codes(g, E, H, I)
            s["w13_scale"], s["w2_scale"] = ((u(E) * 0.5 + 0.75) * 2e-4 for _ in range(2))
            if case["act"] == "static":  # the largest token value, and six deviations of gate and up, map to 448
                s["a1"] = torch.full((1,), 5.0 / 448.0, device="cuda")
                s["a2"] = torch.full((1,), (6.0 * 0.02) ** 2 * H / 448.0, device="cuda")
        else:
            per, q = (2, 15) if wd.startswith("int4") else (1, 255)
            for name, rows, k in (("w13", 2 * I, H), ("w2", H, I)):
                s[name] = torch.randint(0, 256, (E, rows, k // per), generator=g, device="cuda", dtype=torch.uint8)
                s[name + "_scale"] = ((u(E, rows, k // BLOCK) + 0.5) * (0.07 / q)).half()
                if case["zero"]:
                    s[name + "_zero"] = torch.randint(q // 2 - q // 8, q // 2 + q // 8 + 1, (E, rows, k // BLOCK),
                                                      generator=g, device="cuda", dtype=torch.uint8)
        s["out"] = empty(T, H, dtype=torch.bfloat16)
        if own:
            import mixture_experts_layer_gate_gb300 as moe
            s["problem"] = moe.problem(T, H, I, E, case["k"], **_gate(case))
            s["weights"] = moe.Weights(s["w13"], s["w2"], s["w13_scale"], s["w2_scale"], s["a1"], s["a2"],
                                       s["w13_zero"], s["w2_zero"])
            s["ws"] = moe.alloc_few_workspace(s["problem"], s["x"].device)
    return s


# ------------------------------------------------------------------------------------------- plain forms


def _quantise(v, block):
    """[T, n] values to codes and one scale (the largest magnitude / 448; 1 for zeros) per `block` columns."""
    T, n = v.shape
    nb = -(-n // block)
    wide = torch.zeros((T, nb * block), dtype=v.dtype, device=v.device)
    wide[:, :n] = v
    wide = wide.view(T, nb, block)
    amax = wide.abs().amax(dim=2)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return _e4m3(wide / scale[:, :, None]).view(T, nb * block)[:, :n].contiguous(), scale


def _norm_plain(s):
    x, case = s["x"].float(), s["case"]
    out = {}
    if case["residual"]:
        x = x + s["residual"].float()
        out["residual"] = x.to(s["x"].dtype)
    v = x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + s["eps"]) * s["weight"].float()
    out["y"] = v.to(s["x"].dtype)
    if case["quant"] != "none":
        out["codes"], out["scales"] = _quantise(v, BLOCK if case["quant"] == "block" else case["H"])
    return out


def _product_plain(s):
    a, w = (s[n].float() for n in ("a", "w"))
    N, K = w.shape
    a = a * s["a_scale"].repeat_interleave(BLOCK, dim=1)[:, :K]
    w = w * s["w_scale"].repeat_interleave(BLOCK, dim=1)[:, :K].repeat_interleave(BLOCK, dim=0)[:N]
    return a @ w.T


def _swiglu_plain(s):
    h, N = _product_plain(s), s["case"]["N"]
    codes, scales = _quantise(h[:, :N] * torch.sigmoid(h[:, :N]) * h[:, N:], BLOCK)
    return {"codes": codes, "scales": scales}


def _first(keys, k):
    """The k largest keys of each row, ties to the lower index: their columns."""
    return torch.sort(keys, dim=1, descending=True, stable=True).indices[:, :k]


def _select_plain(logits, bias, case):
    T, E = logits.shape
    if case["scoring"] == "softmax":
        e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        keys, score = logits, e / e.sum(dim=1, keepdim=True)
    else:
        score = torch.sigmoid(logits)
        keys = score if bias is None else score + bias
        if bias is None and not case["n_group"]:
            keys = logits
    if case["n_group"]:
        groups = keys.view(T, case["n_group"], -1)
        best = torch.sort(groups, dim=2, descending=True).values[:, :, :2].sum(dim=2)
        allowed = torch.zeros_like(best, dtype=torch.bool).scatter_(1, _first(best, case["topk_group"]), True)
        keys = torch.where(allowed[:, :, None], groups, torch.full_like(groups, -math.inf)).view(T, E)
    ids = _first(keys, case["k"])
    w = score.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids, w * case["factor"]


def _weights_plain(s, name, ids):
    """The chosen experts' matrices, [n, rows, columns]."""
    case, wd = s["case"], s["case"]["wdtype"]
    if wd == "bf16":
        return s[name][ids].float()
    scale = s[name + "_scale"][ids].float()
    codes = s[name].view(torch.uint8)[ids]
    if wd == "fp8":
        return codes.view(torch.float8_e4m3fn).float() * scale[:, None, None]
    if wd == "int8":
        v = (codes if case["zero"] else codes.view(torch.int8)).float()
    else:
        # eight codes of a word: in order, or the even ones in the low half and the odd ones in the high half
        at = [0, 4, 8, 12, 16, 20, 24, 28] if wd == "int4" else [0, 16, 4, 20, 8, 24, 12, 28]
        v = (codes.view(torch.int32)[..., None] >> torch.tensor(at, device=codes.device, dtype=torch.int32)) & 15
        v = v.flatten(2)
        v = v.float() if case["zero"] else ((v ^ 8) - 8).float()
    n, rows, k = v.shape
    v = v.view(n, rows, k // BLOCK, BLOCK)
    if case["zero"]:
        v = v - s[name + "_zero"][ids].float()[..., None]
    return (v * scale[..., None]).view(n, rows, k)


def _codes_plain(v, scale):
    return _e4m3(v / scale).float() * scale


def _few_plain(s):
    case = s["case"]
    T, I, k = case["T"], case["I"], case["k"]
    ids, w = _select_plain(s["logits"], s["bias"], case)
    x = s["x"].float()
    a1, a2 = s["a1"], s["a2"]
    if case["wdtype"] == "fp8":
        x = _codes_plain(x, a1 if a1 is not None else x.abs().amax() / 448.0)
    h = _weights_plain(s, "w13", ids.flatten()) @ x.repeat_interleave(k, dim=0)[:, :, None]
    h = h[:, :, 0]
    act = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]
    if case["wdtype"] == "fp8":
        act = _codes_plain(act, a2 if a2 is not None else act.abs().amax() / 448.0)
    y = (_weights_plain(s, "w2", ids.flatten()) @ act[:, :, None])[:, :, 0]
    return (y.view(T, k, -1) * w[:, :, None]).sum(dim=1).to(torch.bfloat16)


def _plain(s):
    op = s["case"]["op"]
    if op == "norm":
        return _norm_plain(s)
    if op == "router":
        return {"logits": s["x"].float() @ s["w"].float().T}
    if op == "gemm":
        return {"out": _product_plain(s).to(s["out"].dtype)}
    if op == "swiglu":
        return _swiglu_plain(s)
    return {"out": _few_plain(s)}


# ------------------------------------------------------------------------------------------------- calls


def _call(s):
    import mixture_experts_layer_gate_gb300 as moe
    op = s["case"]["op"]
    if op == "norm":
        moe.add_rms_norm(s["problem"], s["x"], s["weight"], residual=s["residual"], residual_out=s["residual_out"],
                         y=s["y"], codes=s["codes"], scales=s["scales"])
        out = {"y": s["y"]}
        if s["residual"] is not None:
            out["residual"] = s["residual_out"]
        if s["codes"] is not None:
            out["codes"], out["scales"] = s["codes"], s["scales"]
        return out
    if op == "router":
        moe.router_logits(s["problem"], s["x"], s["w"], s["logits"], s["ws"])
        return {"logits": s["logits"]}
    if op == "gemm":
        moe.gemm_fp8_block(s["problem"], s["a"], s["a_scale"], s["w"], s["w_scale"], s["out"], s["ws"])
        return {"out": s["out"]}
    if op == "swiglu":
        moe.gemm_fp8_block_swiglu(s["problem"], s["a"], s["a_scale"], s["w"], s["w_scale"], s["codes"], s["scales"],
                                  s["ws"])
        return {"codes": s["codes"], "scales": s["scales"]}
    moe.forward_few(s["problem"], s["weights"], s["x"], s["logits"], s["bias"], s["out"], s["ws"])
    return {"out": s["out"]}


def run(state):
    return _call(state) if own else _plain(state)


# ------------------------------------------------------------------------------------ work and exact values


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
    if op == "norm":
        T, H, b = case["T"], case["H"], size[case["dtype"]]
        moved = T * H * b * (2 + 2 * case["residual"]) + H * size.get(case["wdtype"], b)
        if case["quant"] != "none":
            moved += T * H + 4 * T * (-(-H // BLOCK) if case["quant"] == "block" else 1)
        return {"bytes": moved, "flops": 4 * T * H}
    if op == "router":
        T, H, E = case["T"], case["H"], case["E"]
        return {"bytes": 2 * T * H + 2 * E * H + 4 * T * E, "flops": 2 * T * H * E}
    if op in ("gemm", "swiglu"):
        M, N, K = case["M"], case["N"], case["K"]
        rows, kb = N * (2 if op == "swiglu" else 1), -(-K // BLOCK)
        moved = M * K + rows * K + 4 * kb * (M + -(-rows // BLOCK)) + M * N * size[case["out"]]
        if op == "swiglu":
            moved += 4 * M * (N // BLOCK)
        return {"bytes": moved, "flops": 2 * M * rows * K}
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    touched = E * (1.0 - (1.0 - k / E) ** T)  # expected distinct experts of T tokens
    per = {"bf16": 2.0, "fp8": 1.0, "int8": 1.0}.get(case["wdtype"], 0.5)
    if case["wdtype"].startswith("int"):
        per += (2 + case["zero"]) / BLOCK
    return {"bytes": int(touched * 3 * H * I * per + 4 * T * E + 4 * T * H), "flops": 6 * T * k * H * I}


def _e4m3_64(v):
    """Nearest e4m3 value, ties to the even one, saturating, of 64-bit values."""
    size = v.abs()
    exponent = torch.frexp(size).exponent.clamp(min=-5).double() - 4.0
    step = torch.exp2(exponent)
    return torch.copysign((torch.round(size / step) * step).clamp(max=448.0), v)


def _blocks_64(v, block):
    """e4m3 values and scales, block by block."""
    parts = [(p, p.abs().amax(dim=1, keepdim=True) / 448.0) for p in v.split(block, dim=1)]
    scales = torch.cat([torch.where(m > 0, m, 1.0) for _, m in parts], dim=1)
    return {"codes": torch.cat([_e4m3_64(p / scales[:, i:i + 1]) for i, (p, _) in enumerate(parts)], dim=1),
            "scales": scales}


def _exact_norm(s):
    x = s["x"].double()
    out = {}
    if s["residual"] is not None:
        x = x + s["residual"].double()
        out["residual"] = x
    v = s["weight"].double() * x / torch.sqrt(torch.linalg.vecdot(x, x) / x.shape[1] + s["eps"])[:, None]
    out["y"] = v
    quant = s["case"]["quant"]
    return out if quant == "none" else {**out, **_blocks_64(v, BLOCK if quant == "block" else v.shape[1])}


def _exact_product(s):
    a, w = s["a"].double(), s["w"].double()
    total = torch.zeros((a.shape[0], w.shape[0]), dtype=torch.float64, device=a.device)
    rows = torch.arange(w.shape[0], device=a.device) // BLOCK
    for b in range(s["a_scale"].shape[1]):
        cut = slice(b * BLOCK, (b + 1) * BLOCK)
        part = a[:, cut] @ w[:, cut].T
        total += part * s["a_scale"][:, b].double()[:, None] * s["w_scale"][rows, b].double()[None, :]
    return total


def _exact_route(row, bias, case):
    """One token's experts and weights, by going through the rule in 64 bits."""
    row, E = [float(v) for v in row], len(row)
    if case["scoring"] == "softmax":
        z = math.fsum(math.exp(v - max(row)) for v in row)
        score, keys = [math.exp(v - max(row)) / z for v in row], row
    else:
        score = [1.0 / (1.0 + math.exp(-v)) for v in row]
        keys = [v + b for v, b in zip(score, bias)] if bias else (score if case["n_group"] else row)
    allowed = range(E)
    if case["n_group"]:
        n = E // case["n_group"]
        best = [sum(sorted(keys[i:i + n])[-2:]) for i in range(0, E, n)]
        groups = sorted(range(case["n_group"]), key=lambda i: (-best[i], i))[:case["topk_group"]]
        allowed = [e for e in range(E) if e // n in groups]
    ids = sorted(allowed, key=lambda e: (-keys[e], e))[:case["k"]]
    total = math.fsum(score[e] for e in ids) if case["renorm"] else 1.0
    return [(e, score[e] / total * case["factor"]) for e in ids]


def _exact_matrix(s, name, e):
    case, wd, m = s["case"], s["case"]["wdtype"], s[name][e]
    if wd == "bf16":
        return m.double()
    scale = s[name + "_scale"][e].double()
    if wd == "fp8":
        return m.double() * scale
    zero = s[name + "_zero"][e].double() if case["zero"] else torch.zeros_like(scale)
    if wd == "int8":
        v = m.double()
        if not case["zero"]:
            v = torch.where(v > 127, v - 256, v)
    else:
        nibbles = torch.stack([m & 15, m >> 4], dim=2).flatten(1).double()  # lowest nibble of each byte first
        if wd == "int4_paired":
            nibbles = nibbles.view(m.shape[0], -1, 2, 4).transpose(2, 3).flatten(1)
        v = nibbles if case["zero"] else torch.where(nibbles > 7, nibbles - 16, nibbles)
    wide = lambda t: t.repeat_interleave(BLOCK, dim=1)  # noqa: E731
    return (v - wide(zero)) * wide(scale)


def _exact_few(s):
    case = s["case"]
    T, I = case["T"], case["I"]
    bias = s["bias"].tolist() if s["bias"] is not None else None
    routes = [_exact_route(row, bias, case) for row in s["logits"].tolist()]
    x = s["x"].double()
    fp8 = case["wdtype"] == "fp8"
    quantised = lambda v, q: _e4m3_64(v / q) * q  # noqa: E731
    if fp8:
        x = quantised(x, s["a1"].double() if s["a1"] is not None else x.abs().max() / 448.0)
    chosen = sorted({e for r in routes for e, _ in r})
    acts = {}
    for e in chosen:
        w13 = _exact_matrix(s, "w13", e)
        for t in range(T):
            if e in dict(routes[t]):
                h = w13 @ x[t]
                acts[t, e] = h[:I] / (1.0 + torch.exp(-h[:I])) * h[I:]
    if fp8:
        q = s["a2"].double() if s["a2"] is not None else max(v.abs().max() for v in acts.values()) / 448.0
        acts = {at: quantised(v, q) for at, v in acts.items()}
    out = torch.zeros_like(x)
    for e in chosen:
        w2 = _exact_matrix(s, "w2", e)
        for t in range(T):
            for f, weight in routes[t]:
                if f == e:
                    out[t] += weight * (w2 @ acts[t, e])
    return out


def exact(case, seed):
    """The outputs of run() from the definitions, in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm(s)
    if op == "router":
        return {"logits": s["x"].double() @ s["w"].double().T}
    if op == "gemm":
        return {"out": _exact_product(s)}
    if op == "swiglu":
        h, N = _exact_product(s), case["N"]
        return _blocks_64(h[:, :N] / (1.0 + torch.exp(-h[:, :N])) * h[:, N:], BLOCK)
    return {"out": _exact_few(s)}
