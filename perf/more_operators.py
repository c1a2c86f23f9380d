"""The operators of a decoder block's attention half, their plain forms and the cases they are measured on.

Beside the pre-norm MoE block a decoder layer has an attention block: the query, key and value projection in 16 bits
(linear: a product with bias, activation and residual), norms of each query and key head with the rotation of their
positions, which write the new keys and values into the paged cache, in 16 bits or in 8 with a scale per token and head
(qk_norm_rope), and attention of the new tokens over the cache (paged_attention), or over the packed prompts themselves
(prompt_attention).  Each case is one of these calls.

With `own` false, run() computes a case in elementary torch operations in 32 bits; with `own` true it calls this
repository's package.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    """Sizes are those of the decoders whose MoE layers this repository measures (32 or 28 or 40 query heads over 8 or 4
    key heads of 128; hidden widths of 4096 and 3584), and generic odd ones."""
    return [
        # --- products of the projections
        # decode: one token's query, key and value projection
        dict(name="linear decode", op="linear", M=1, N=6144, K=4096, dtype="bf16", out="bf16", bias=True, act="none",
             residual=False, pad=0),
        # prefill: the output projection, added to the residual stream
        dict(name="linear prefill", op="linear", M=4096, N=4096, K=4096, dtype="bf16", out="bf16", bias=False,
             act="none", residual=True, pad=0),
        # --- norm and rotation of queries and keys into the cache
        # decode: a batch of streams at far positions of a scaled context, into an 8-bit cache
        dict(name="rope decode", op="rope", T=16, Hq=28, Hkv=4, D=128, rot=128, layout="half", dtype="bf16", norm=True,
             wdtype="f32", far=1_000_000, factor=32.0, page=64, cache="e4m3", order="token", skip=False),
        # prefill: a prompt into a 16-bit cache
        dict(name="rope prefill", op="rope", T=4096, Hq=32, Hkv=8, D=128, rot=128, layout="half", dtype="bf16",
             norm=True, wdtype="bf16", far=0, factor=1.0, page=16, cache="bf16", order="head", skip=False),
        # --- attention over the paged cache
        # decode: one stream, short context
        dict(name="decode short", op="paged", B=1, new=1, new_hi=1, past=500, past_hi=500, Hq=32, Hkv=8, D=128,
             dtype="bf16", cache="bf16", page=16, order="token", spare=0),
        # decode: a batch whose contexts differ by a factor of 160
        dict(name="decode ragged", op="paged", B=64, new=1, new_hi=1, past=100, past_hi=16384, Hq=32, Hkv=8, D=128,
             dtype="bf16", cache="bf16", page=16, order="head", spare=0),
        # decode: two streams of long documents over an 8-bit cache
        dict(name="decode long 8-bit", op="paged", B=2, new=1, new_hi=1, past=90001, past_hi=131071, Hq=28, Hkv=4,
             D=128, dtype="bf16", cache="e4m3", page=64, order="head", spare=0),
        # verification of drafted tokens: a few new tokens a stream
        dict(name="drafts", op="paged", B=16, new=1, new_hi=6, past=1111, past_hi=9000, Hq=40, Hkv=8, D=128,
             dtype="f16", cache="f16", page=32, order="token", spare=3),
        # chunks of prompts and single tokens in one batch
        dict(name="mixed chunks", op="paged", B=8, new=1, new_hi=1024, past=1, past_hi=20000, Hq=32, Hkv=8, D=128,
             dtype="bf16", cache="bf16", page=16, order="head", spare=0),
        # one chunk of a long prompt over an 8-bit cache
        dict(name="chunk 8-bit", op="paged", B=1, new=2048, new_hi=2048, past=30011, past_hi=30011, Hq=28, Hkv=4,
             D=128, dtype="bf16", cache="e4m3", page=64, order="token", spare=0),
        # --- attention over whole prompts
        # a few short prompts, odd sizes
        dict(name="prompts odd", op="prompt", B=5, new=1, new_hi=777, Hq=6, Hkv=2, D=72, dtype="f16", spare=5),
        # prefill: packed prompts
        dict(name="prompts packed", op="prompt", B=4, new=513, new_hi=7001, Hq=32, Hkv=8, D=128, dtype="bf16",
             spare=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    Hkv = rng.choice([1, 2, 3, 4, 8])
    return Hkv * rng.choice([1, 2, 4, 5, 7, 8]), Hkv, rng.choice([64, 128, 128, 128, _log(rng, 1, 16) * 8])


def _depth(D, cache):
    """Rows of a cache are whole pieces of 16 bytes."""
    return -(-D // 16) * 16 if cache == "e4m3" else D


def draw(rng):
    op = rng.choice(["linear", "rope", "paged", "paged", "paged", "prompt"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 4096), N=_log(rng, 16, 4096), K=_log(rng, 2, 512) * 8, dtype=dtype,
                    out=rng.choice(["f32", dtype, dtype]), bias=rng.random() < 0.5,
                    act=rng.choice(["none", "none", "silu", "gelu", "gelu_tanh", "relu"]),
                    residual=rng.random() < 0.5, pad=rng.choice([0, 8]))
    Hq, Hkv, D = _heads(rng)
    if op == "rope":
        layout = rng.choice(["half", "interleaved"])
        rot = max(16, D // rng.choice([1, 1, 2, 4]) // 16 * 16)
        cache = rng.choice([dtype, "e4m3"])
        D = _depth(max(D, rot), cache)
        T = min(_log(rng, 1, 4096), 4096 * 40 * 128 // ((Hq + Hkv) * D))
        return dict(op=op, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, layout=layout, dtype=dtype, norm=rng.random() < 0.7,
                    wdtype=rng.choice(["f32", dtype]), far=rng.choice([0, 0, 5000, 1_000_000]),
                    factor=rng.choice([1.0, 8.0, 32.0]), page=rng.choice([16, 32, 64, 256]),
                    cache=cache, order=rng.choice(["token", "head"]), skip=rng.random() < 0.3)
    if op == "prompt":
        hi = _log(rng, 1, 7001)
        return dict(op=op, B=rng.randint(1, 4), new=_log(rng, 1, hi), new_hi=hi, Hq=Hq // Hkv * min(Hkv, 4),
                    Hkv=min(Hkv, 4), D=D, dtype=dtype, spare=rng.choice([0, 0, 7]))
    # paged: single tokens, a few, or chunks; no more keys than in the ragged batch, no more products than in the chunk
    new_hi = rng.choice([1, 1, _log(rng, 2, 12), _log(rng, 13, 2048)])
    B = _log(rng, 1, 64)
    while B > 1 and B * new_hi * Hq > 40000:
        B //= 2
    most = min(131071, 1_600_000 // (B * Hkv), int(1.7e9 / (B * new_hi * Hq)))
    past_hi = _log(rng, 1, max(1, most))
    cache = rng.choice([dtype, "e4m3"])
    return dict(op=op, B=B, new=_log(rng, 1, new_hi), new_hi=new_hi, past=_log(rng, 1, past_hi), past_hi=past_hi,
                Hq=Hq, Hkv=Hkv, D=_depth(D, cache), dtype=dtype, cache=cache,
                page=rng.choice([16, 32, 64, 256]), order=rng.choice(["token", "head"]), spare=rng.choice([0, 0, 3]))


# ------------------------------------------------------------------------------------------------ inputs


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly by logarithm."""
    if n == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]


def _lengths(case):
    """New tokens and earlier ones of each sequence, in an order that the case alone gives."""
    mix = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    new = _spread(case["new"], case["new_hi"], case["B"])
    past = _spread(case["past"], case["past_hi"], case["B"]) if case["op"] == "paged" else [0] * case["B"]
    mix.shuffle(new)
    mix.shuffle(past)
    return new, past


def _inv_freq(case):
    """Radians a position of each rotated pair; for a context stretched by `factor` the pairs that turn fewer than 1
    time over the original 8192 positions are slowed by it, those beyond 32 turns are not, and those between in
    proportion."""
    rot = case["rot"]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if case["factor"] == 1.0:
        return f
    keep = ((8192.0 * f / (2.0 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return keep * f + (1.0 - keep) * f / case["factor"]


def _magnitude(case):
    return 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _normal(g, shape, dtype):
    """Normal values, made in parts."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.view(-1).split(1 << 27):
        part.copy_(_randn(g, part.numel()))
    return out


def _e4m3(v):
    """Values of any size in e4m3: rounded to nearest even, saturating."""
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _codes(g, shape):
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    for part in out.view(-1).split(1 << 27):
        part.copy_(_e4m3(_randn(g, part.numel()) * 100.0))
    return out


def _cache(g, pages, case):
    """Keys or values [pages, page, Hkv, D], in memory by tokens or by heads, and the scales [pages, Hkv, page]."""
    page, Hkv, D = case["page"], case["Hkv"], case["D"]
    shape = (pages, page, Hkv, D) if case["order"] == "token" else (pages, Hkv, page, D)
    scale = None
    if case["cache"] == "e4m3":
        c = _codes(g, shape)
        scale = (torch.rand((pages, Hkv, page), generator=g, device="cuda") + 0.5) * 0.01
    else:
        c = _normal(g, shape, DTYPES[case["cache"]])
    return c if case["order"] == "token" else c.transpose(1, 2), scale


def _seed_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    return g


def prepare(case, seed):
    """Inputs of one call, its output buffers and (own) the problem, tables and workspace that a program keeps."""
    g = _seed_of(seed)
    s = dict(case=case)
    op, dt = case["op"], DTYPES[case["dtype"]]
    if own:
        import mixture_experts_layer_gate_gb300 as moe
    if op == "linear":
        M, N, K, odt = case["M"], case["N"], case["K"], DTYPES[case["out"]]
        s["x"] = _randn(g, M, K + case["pad"]).to(dt)[:, :K]
        s["w"] = (_randn(g, N, K) * K ** -0.5).to(dt)
        s["bias"] = (_randn(g, N) * 0.5).to(dt) if case["bias"] else None
        s["residual"] = (_randn(g, M, N) * 3.0).to(odt) if case["residual"] else None
        s["out"] = torch.empty((M, N), dtype=odt, device="cuda")
        if own:
            s["problem"] = moe.linear_problem(M, N, K, dtype=case["dtype"], out_dtype=case["out"],
                                              activation=case["act"])
            s["ws"] = moe.alloc_op_workspace(s["x"].device)
        return s
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if op == "rope":
        T, page = case["T"], case["page"]
        s["qkv"] = _randn(g, T, (Hq + 2 * Hkv) * D).to(dt)  # as one projection writes them
        # a prompt's positions in order, or streams anywhere up to `far`
        s["positions"] = (torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
                          if case["far"] else torch.arange(T, device="cuda", dtype=torch.int32))
        pages = -(-T // page) + 2
        at = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        slots = at[t // page] * page + t % page
        if case["skip"]:  # tokens of a padded batch have no place in the cache
            slots = torch.where(torch.rand((T,), generator=g, device="cuda") < 0.1, -1, slots)
        s["slots"] = slots.int()
        s["k_cache"], s["k_scale"] = _cache(g, pages, case)
        s["v_cache"], s["v_scale"] = _cache(g, pages, case)
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"], s["k_weight"] = ((1.0 + 0.1 * _randn(g, D)).to(DTYPES[case["wdtype"]]) for _ in range(2))
        s["eps"] = 1e-6
        s["inv_freq"] = _inv_freq(case).cuda()
        s["q_out"] = torch.empty((T, Hq * D), dtype=dt, device="cuda")
        if own:
            s["problem"] = moe.rope_problem(T, Hq, Hkv, D, rot=case["rot"], layout=case["layout"], dtype=case["dtype"],
                                            weight_dtype=case["wdtype"], eps=s["eps"], magnitude=_magnitude(case),
                                            cache_dtype=case["cache"], page_size=page, num_pages=pages)
            s["table"] = moe.rope_table(case["rot"], theta=10000.0, factor=case["factor"], original=8192, low=1.0,
                                        high=32.0, device="cuda")
            s["ws"] = moe.alloc_op_workspace(s["qkv"].device)
        return s
    new, past = _lengths(case)
    T = sum(new) + case["spare"]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["new"], s["past"], s["cu"] = new, past, cu  # (host copies, for the plain form's loop)
    s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["scale"] = D ** -0.5
    s["out"] = torch.zeros((T, Hq * D), dtype=dt, device="cuda")
    s["lse"] = torch.zeros((T, Hq), dtype=torch.float32, device="cuda")
    if op == "prompt":
        qkv = _normal(g, (T, (Hq + 2 * Hkv) * D), dt)
        s["q"], s["k"], s["v"] = qkv.split((Hq * D, Hkv * D, Hkv * D), dim=1)
        if own:
            s["problem"] = moe.attention_problem(T, case["B"], Hq, Hkv, D, max_q=max(new), dtype=case["dtype"],
                                                 scale=s["scale"])
    else:
        page = case["page"]
        s["q"] = _normal(g, (T, Hq * D), dt)
        need = [-(-(n + p) // page) for n, p in zip(new, past)]
        pages, wide = sum(need) + 3, max(need) + 1
        s["k_cache"], s["k_scale"] = _cache(g, pages, case)
        s["v_cache"], s["v_scale"] = _cache(g, pages, case)
        at = torch.randperm(pages, generator=g, device="cuda").int()
        s["page_table"] = torch.full((case["B"], wide), -1, dtype=torch.int32, device="cuda")
        first = 0
        for b, n in enumerate(need):
            s["page_table"][b, :n] = at[first:first + n]
            first += n
        s["kv_len"] = torch.tensor([n + p for n, p in zip(new, past)], dtype=torch.int32, device="cuda")
        if own:
            s["problem"] = moe.attention_problem(T, case["B"], Hq, Hkv, D, max_q=max(new), dtype=case["dtype"],
                                                 cache_dtype=case["cache"], page_size=page, num_pages=pages,
                                                 max_pages=wide, scale=s["scale"])
    if own:
        s["ws"] = moe.alloc_attention_workspace(s["problem"], s["q"].device)
    return s


# ------------------------------------------------------------------------------------------- plain forms


def _linear_plain(s):
    v = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        v = v + s["bias"].float()
    act = s["case"]["act"]
    if act == "silu":
        v = v / (1.0 + torch.exp(-v))
    elif act == "gelu":
        v = 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        v = 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    elif act == "relu":
        v = torch.where(v < 0, torch.zeros_like(v), v)
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return {"out": v.to(s["out"].dtype)}


def _norm_rotate_plain(x, weight, s):
    """x [T, heads, D] in float."""
    case = s["case"]
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=2, keepdim=True) + s["eps"]) * weight.float()
    rot = case["rot"]
    angle = s["positions"].double()[:, None] * s["inv_freq"][None, :]
    cos = (torch.cos(angle) * _magnitude(case)).float()[:, None, :]
    sin = (torch.sin(angle) * _magnitude(case)).float()[:, None, :]
    out = x.clone()
    if case["layout"] == "half":
        a, b = x[:, :, :rot // 2], x[:, :, rot // 2:rot]
        out[:, :, :rot // 2], out[:, :, rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[:, :, 0:rot:2], x[:, :, 1:rot:2]
        out[:, :, 0:rot:2], out[:, :, 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return out


def _store_plain(cache, scales, v, slots, page):
    """v [T, Hkv, D] in float to the cache's slots (those that are not negative)."""
    kept = (slots >= 0).nonzero()[:, 0]
    at = slots[kept].long()
    v = v[kept]
    if scales is None:
        cache[at // page, at % page] = v.to(cache.dtype)
        return
    amax = v.abs().amax(dim=2)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    cache.view(torch.uint8)[at // page, at % page] = _e4m3(v / scale[:, :, None]).view(torch.uint8)
    scales[at // page, :, at % page] = scale


def _rope_plain(s):
    case = s["case"]
    T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
    q, k, v = (t.reshape(T, -1, D).float() for t in s["qkv"].split((Hq * D, Hkv * D, Hkv * D), dim=1))
    q = _norm_rotate_plain(q, s["q_weight"], s).to(s["q_out"].dtype).view(T, -1)
    k = _norm_rotate_plain(k, s["k_weight"], s)
    _store_plain(s["k_cache"], s["k_scale"], k, s["slots"], case["page"])
    _store_plain(s["v_cache"], s["v_scale"], v, s["slots"], case["page"])
    return _rope_out(s, q)


def _rope_out(s, q):
    out = {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["k_scale"] is not None:
        out["k_scale"], out["v_scale"] = s["k_scale"], s["v_scale"]
    return out


def _keys_plain(s, b, name):
    """Keys or values of sequence b in float, [Hkv, L, D]."""
    case = s["case"]
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "prompt":
        rows = s[name][s["cu"][b]:s["cu"][b + 1]]
        return rows.reshape(-1, Hkv, D).float().transpose(0, 1)
    L, page = s["new"][b] + s["past"][b], case["page"]
    pages = s["page_table"][b, :-(-L // page)].long()
    if s["k_scale"] is None:
        v = s[name + "_cache"][pages].float()
    else:
        v = s[name + "_cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
        v = v * s[name + "_scale"][pages].transpose(1, 2)[..., None]
    return v.reshape(-1, Hkv, D)[:L].transpose(0, 1)


def _attention_plain(s):
    case = s["case"]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    out, lse = s["out"].clone(), s["lse"].clone()
    for b, (n, past) in enumerate(zip(s["new"], s["past"])):
        rows = slice(s["cu"][b], s["cu"][b + 1])
        q = s["q"][rows].float().reshape(n, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3)
        k, v = _keys_plain(s, b, "k"), _keys_plain(s, b, "v")
        unseen = None
        if n > 1:
            at = torch.arange(n + past, device=k.device)
            unseen = at[None, :] > at[past:, None]
        # key heads together while their scores are few, else one at a time
        step = Hkv if Hq * n * (n + past) < 1 << 26 else 1
        for h in range(0, Hkv, step):
            e = q[h:h + step].reshape(-1, Hq // Hkv * n, D) @ k[h:h + step].transpose(1, 2) * s["scale"]
            if unseen is not None:
                e.view(-1, Hq // Hkv, n, n + past).masked_fill_(unseen, -math.inf)
            top = e.amax(dim=2, keepdim=True)
            e = torch.exp(e - top)
            total = e.sum(dim=2, keepdim=True)
            o = ((e @ v[h:h + step]) / total).view(-1, Hq // Hkv, n, D).permute(2, 0, 1, 3)
            heads = slice(h * (Hq // Hkv), (h + step) * (Hq // Hkv))
            out[rows].view(n, Hq, D)[:, heads] = o.reshape(n, -1, D).to(out.dtype)
            lse[rows, heads] = (top + torch.log(total)).view(-1, n).T
    return {"out": out, "lse": lse}


def _plain(s):
    return {"linear": _linear_plain, "rope": _rope_plain, "paged": _attention_plain,
            "prompt": _attention_plain}[s["case"]["op"]](s)


# ------------------------------------------------------------------------------------------------- calls


def _call(s):
    import mixture_experts_layer_gate_gb300 as moe
    case, op = s["case"], s["case"]["op"]
    if op == "linear":
        moe.linear(s["problem"], s["x"], s["w"], s["out"], s["ws"], bias=s["bias"], residual=s["residual"])
        return {"out": s["out"]}
    if op == "rope":
        n, m = case["Hq"] * case["D"], case["Hkv"] * case["D"]
        q, k, v = s["qkv"].split((n, m, m), dim=1)
        moe.qk_norm_rope(s["problem"], q, k, s["positions"], s["table"], s["q_out"], s["ws"], v=v,
                         k_cache=s["k_cache"], v_cache=s["v_cache"], slots=s["slots"], k_scale=s["k_scale"],
                         v_scale=s["v_scale"], q_weight=s["q_weight"], k_weight=s["k_weight"])
        return _rope_out(s, s["q_out"])
    if op == "prompt":
        moe.prompt_attention(s["problem"], s["q"], s["k"], s["v"], s["cu_q"], s["out"], s["ws"], lse=s["lse"])
    else:
        moe.paged_attention(s["problem"], s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["cu_q"], s["kv_len"],
                            s["out"], s["ws"], k_scale=s["k_scale"], v_scale=s["v_scale"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    return _call(state) if own else _plain(state)


# ------------------------------------------------------------------------------------ work and exact values


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
    op, b = case["op"], size[case["dtype"]]
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        moved = b * (M * K + N * K + N * case["bias"]) + size[case["out"]] * M * N * (1 + case["residual"])
        return {"bytes": moved, "flops": 2 * M * N * K}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if op == "rope":
        T, c = case["T"], size[case["cache"]]
        moved = T * D * (b * (2 * Hq + 2 * Hkv) + 2 * c * Hkv) + 8 * T + (8 * T * Hkv if c == 1 else 0)
        return {"bytes": moved, "flops": 8 * T * (Hq + Hkv) * D}
    new, past = _lengths(case)
    c = size[case.get("cache", case["dtype"])]
    keys = sum(new) + sum(past)
    seen = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    moved = 2 * b * sum(new) * Hq * D + 4 * sum(new) * Hq + keys * Hkv * (2 * D * c + (8 if c == 1 else 0))
    return {"bytes": moved, "flops": 4 * seen * Hq * D}


def _e4m3_64(v):
    """Nearest e4m3 value, ties to the even one, saturating, of 64-bit values."""
    size = v.abs()
    exponent = torch.frexp(size).exponent.clamp(min=-5).double() - 4.0
    step = torch.exp2(exponent)
    return torch.copysign((torch.round(size / step) * step).clamp(max=448.0), v)


def _exact_linear(s):
    v = s["x"].double() @ s["w"].double().T
    if s["bias"] is not None:
        v += s["bias"].double()
    act = s["case"]["act"]
    if act == "silu":
        v = v * torch.sigmoid(v)
    elif act == "gelu":
        v = v * torch.special.ndtr(v)
    elif act == "gelu_tanh":  # (1 + tanh z) / 2 = 1 / (1 + exp(-2 z))
        v = v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    elif act == "relu":
        v = v.clamp(min=0.0)
    return {"out": v if s["residual"] is None else v + s["residual"].double()}


def _exact_rope(s):
    case = s["case"]
    T, Hq, Hkv, D, rot, page = (case[n] for n in ("T", "Hq", "Hkv", "D", "rot", "page"))
    x = s["qkv"].double().view(T, Hq + 2 * Hkv, D)
    turn = torch.polar(torch.full((T, rot // 2), _magnitude(case), dtype=torch.float64, device=x.device),
                       torch.outer(s["positions"].double(), s["inv_freq"]))

    def head(h, weight):
        v = x[:, h]
        if weight is not None:
            v = weight.double() * v / torch.sqrt(torch.linalg.vecdot(v, v) / D + s["eps"])[:, None]
        front = v[:, :rot].reshape(T, 2, -1).transpose(1, 2) if case["layout"] == "half" else v[:, :rot].reshape(T, -1, 2)
        turned = torch.view_as_real(torch.view_as_complex(front.contiguous()) * turn)
        front = turned.transpose(1, 2) if case["layout"] == "half" else turned
        return torch.cat([front.reshape(T, rot), v[:, rot:]], dim=1)

    out = {"q": torch.cat([head(h, s["q_weight"]) for h in range(Hq)], dim=1)}
    slots = s["slots"].long()
    there = slots >= 0
    at = (slots[there] // page, slots[there] % page)
    for name in ("k", "v"):
        cache, scales = s[name + "_cache"].double(), s[name + "_scale"]
        if scales is not None:
            scales = scales.double()
        for h in range(Hkv):
            v = (head(Hq + h, s["k_weight"]) if name == "k" else x[:, Hq + Hkv + h])[there]
            if scales is not None:
                top = v.abs().amax(dim=1) / 448.0
                top = torch.where(top > 0, top, 1.0)
                scales[at[0], h, at[1]] = top
                v = _e4m3_64(v / top[:, None])
            cache[at[0], at[1], h] = v
        out[name + "_cache"] = cache
        if scales is not None:
            out[name + "_scale"] = scales
    return out


def _exact_attention(s):
    """Query head by query head, the rows in parts."""
    case = s["case"]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    out, lse = s["out"].double(), s["lse"].double()
    for b, (n, past) in enumerate(zip(s["new"], s["past"])):
        L, first = n + past, s["cu"][b]
        for h in range(Hkv):
            k, v = (_exact_keys(s, b, h, L, name) for name in ("k", "v"))
            for hq in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                for lo in range(0, n, 1024):
                    hi = min(n, lo + 1024)
                    q = s["q"][first + lo:first + hi, hq * D:(hq + 1) * D].double()
                    z = (q @ k[:past + hi].T) * s["scale"]
                    z = z.masked_fill(torch.ones_like(z, dtype=torch.bool).triu(past + lo + 1), -math.inf)
                    out[first + lo:first + hi, hq * D:(hq + 1) * D] = torch.softmax(z, dim=1) @ v[:past + hi]
                    lse[first + lo:first + hi, hq] = torch.logsumexp(z, dim=1)
    return {"out": out, "lse": lse}


def _exact_keys(s, b, h, L, name):
    case = s["case"]
    if case["op"] == "prompt":
        return s[name][s["cu"][b]:s["cu"][b + 1], h * case["D"]:(h + 1) * case["D"]].double()
    j = torch.arange(L, device=s["page_table"].device)
    page, row = s["page_table"][b].long()[j // case["page"]], j % case["page"]
    if s["k_scale"] is None:
        return s[name + "_cache"][page, row, h].double()
    codes = s[name + "_cache"].view(torch.uint8)[page, row, h].view(torch.float8_e4m3fn)
    return codes.double() * s[name + "_scale"][page, h, row].double()[:, None]


def exact(case, seed):
    """The outputs of run() from the definitions, in 64 bits."""
    s = prepare(case, seed)
    return {"linear": _exact_linear, "rope": _exact_rope, "paged": _exact_attention,
            "prompt": _exact_attention}[case["op"]](s)
