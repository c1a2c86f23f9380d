"""The pre-norm blocks of a decoder layer, each from the residual stream to what is added to it next.

AttentionBlock: residual add + RMS norm, the query, key and value projection, head
norms and rotation into a paged cache (KVCache), attention over it, the output
projection.  MoEBlock: residual add + RMS norm, router scores, the routed experts and a
shared expert in block-scaled 8-bit floating point (the DeepSeek-V3 block: every token
passes through its routed experts and one shared expert, both on the normed input).
DecoderLayer: one after the other.
"""
from __future__ import annotations

from . import binding as b


def _first_error(stream, *workspaces) -> int:
    found = 0
    for ws in workspaces:
        e = b.get_device_error(ws, stream) if ws is not None else 0
        if e:  # a call that timed out, perhaps after this error, leaves counters that are zero between calls
            b.run_on(stream, ws.zero_)
        found = found or e
    return found


class SharedExpert:
    """Weights of the shared expert: w13 e4m3 [2I, H] and w2 e4m3 [H, I] with a float32 scale per 128 x 128 block."""

    def __init__(self, w13, w13_scale, w2, w2_scale):
        self.w13, self.w13_scale, self.w2, self.w2_scale = w13, w13_scale, w2, w2_scale
        self.I = w2.shape[1]


class MoEBlock:
    """`block(x, residual)` -> (out, residual + x), both bf16 [T, H]; the next block adds out to the residual.

    `gate` takes problem()'s keywords (scoring, n_group, wdtype, ...).  Batches that
    moe_forward_few takes (FEW_MAX_TOKENS tokens up to H = 8192, fewer beyond) run
    there, others in moe_forward.  Calls
    of one block share its workspaces: order them on one stream, the given raw one or
    PyTorch's current one.  What a call allocates belongs to that stream.  With a
    stream other than the current one the block and the inputs have to be ready on it
    (wait_stream), and the outputs are once its work is; the memory of neither is reused
    before both streams are done with it.
    """

    def __init__(self, H, I, E, top_k, weights: b.Weights, norm_weight, router_weight, shared: SharedExpert | None,
                 max_tokens: int, device, router_bias=None, eps: float = 1e-6, **gate):
        self.H, self.eps = H, eps
        self.norm_weight, self.router_weight, self.router_bias = norm_weight, router_weight, router_bias
        self.shared, self.weights = shared, weights
        self.layer = b.MoELayer(H, I, E, top_k, weights, max_tokens, device, **gate)
        self.few_ws, self.kept, self.left = None, [], None  # (kept, left: workspace_of)
        for T in range(min(max_tokens, b.FEW_MAX_TOKENS), 0, -1):
            if b.few_workspace_size(self.layer.problem(T)):
                self.few_ws = b.alloc_few_workspace(self.layer.problem(T), device)
                break
        self.op_ws = b.alloc_op_workspace(device)

    def __call__(self, x, residual=None, stream=None):
        return b.run_on(stream, self._run, x, residual)

    def _run(self, x, residual):
        import torch
        T, H = x.shape
        dev = x.device
        new = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        y = new(T, H)
        total = new(T, H) if residual is not None else None
        codes = new(T, H, dtype=torch.uint8) if self.shared else None
        scales = new(T, -(-H // 128), dtype=torch.float32) if self.shared else None
        wdt = "f32" if self.norm_weight.dtype == torch.float32 else "bf16"
        b.add_rms_norm(b.norm_problem(T, H, weight_dtype=wdt, eps=self.eps, quant="block" if self.shared else "none"),
                       x, self.norm_weight, residual, total, y, codes, scales)
        p = self.layer.problem(T)
        logits = new(T, p.E, dtype=torch.float32)
        b.router_logits(b.router_problem(T, H, p.E), y, self.router_weight, logits, self.op_ws)
        out = new(T, H)
        few = b.few_workspace_size(p) if 0 < T <= b.FEW_MAX_TOKENS else 0
        if few:
            ws = b.workspace_of(self, "few_ws", few, lambda: b.alloc_few_workspace(p, dev))
            b.forward_few(p, self.weights, y, logits, self.router_bias, out, ws)
        else:
            self.layer(y, logits, self.router_bias, out)
        if self.shared:
            s = self.shared
            act = new(T, s.I, dtype=torch.uint8)
            act_scales = new(T, s.I // 128, dtype=torch.float32)
            b.gemm_fp8_block_swiglu(b.fp8_gemm_problem(T, s.I, H), codes, scales, s.w13, s.w13_scale, act, act_scales,
                                    self.op_ws)
            b.gemm_fp8_block(b.fp8_gemm_problem(T, H, s.I, accumulate=True), act, act_scales, s.w2, s.w2_scale, out,
                             self.op_ws)
        return out, total if total is not None else x

    def device_error(self, stream=None) -> int:
        """First error that a kernel of the block recorded (0: none), cleared; synchronises the stream.  Then
        the block can be used again."""
        return _first_error(stream, self.left, self.layer.left, self.op_ws, self.few_ws, self.layer.ws, *self.kept,
                            *self.layer.kept)


class KVCache:
    """Keys and values of num_pages pages of page_size tokens, Hkv heads of D values each: bf16, or e4m3 codes with a
    scale per token and head (cache_dtype="e4m3").  A head's tokens of a page are adjacent in memory.  What is not
    stored yet is never read."""

    def __init__(self, num_pages, page_size, Hkv, D, device, cache_dtype="bf16"):
        import torch
        if cache_dtype not in ("bf16", "e4m3"):
            raise ValueError("cache_dtype: 'bf16' or 'e4m3'")
        self.num_pages, self.page_size, self.Hkv, self.D, self.cache_dtype = num_pages, page_size, Hkv, D, cache_dtype
        dt = torch.float8_e4m3fn if cache_dtype == "e4m3" else torch.bfloat16
        self.k, self.v = (torch.empty((num_pages, Hkv, page_size, D), dtype=dt, device=device).transpose(1, 2)
                          for _ in range(2))
        self.k_scale = self.v_scale = None
        if cache_dtype == "e4m3":
            self.k_scale, self.v_scale = (torch.empty((num_pages, Hkv, page_size), dtype=torch.float32, device=device)
                                          for _ in range(2))

    @property
    def tensors(self):
        return self.k, self.v, self.k_scale, self.v_scale


class AttentionBlock:
    """`block(x, residual, positions, cu_q, max_q, ...)` -> (out, residual + x), both bf16 [T, H]; the next block adds
    out to the residual.

    Weights bf16: wqkv [(Hq + 2 Hkv) D, H] with an optional bias, wo [H, Hq D], norm_weight [H], and optionally
    q_norm, k_norm [D] (norms of each head).  turns: rope_table's of the rot (all D without it) rotated values.
    x holds the new tokens of some sequences, packed: sequence b's are rows cu_q[b] .. cu_q[b + 1] - 1 (int32), at
    most max_q of one, at positions (int32 [T]).  With a cache they are stored at slots (int32 [T], page * page_size +
    place; negative: a padded row) and attend kv_len[b] tokens through page_table; without one each sequence is a whole
    prompt.  Streams, graphs and workspaces as MoEBlock's.
    """

    def __init__(self, H, Hq, Hkv, D, wqkv, wo, norm_weight, turns, device, bias=None, q_norm=None, k_norm=None, rot=None,
                 layout="half", magnitude=1.0, scale=None, eps: float = 1e-6):
        self.H, self.Hq, self.Hkv, self.D, self.eps = H, Hq, Hkv, D, eps
        self.wqkv, self.wo, self.norm_weight, self.bias, self.turns = wqkv, wo, norm_weight, bias, turns
        self.q_norm, self.k_norm, self.scale = q_norm, k_norm, scale
        norms = [w for w in (q_norm, k_norm) if w is not None]
        self.rope = dict(rot=D if rot is None else rot, layout=layout, magnitude=magnitude, eps=eps,
                         weight_dtype="f32" if norms and str(norms[0].dtype) == "torch.float32" else "bf16")
        self.op_ws = b.alloc_op_workspace(device)
        self.attention_ws, self.kept, self.left = None, [], None  # (kept, left: workspace_of)

    def __call__(self, x, residual, positions, cu_q, max_q, cache: KVCache | None = None, slots=None, page_table=None,
                 kv_len=None, stream=None):
        return b.run_on(stream, self._run, x, residual, positions, cu_q, max_q, cache, slots, page_table, kv_len)

    def _run(self, x, residual, positions, cu_q, max_q, cache, slots, page_table, kv_len):
        import torch
        T, H = x.shape
        Hq, Hkv, D, dev = self.Hq, self.Hkv, self.D, x.device
        new = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device=dev)  # noqa: E731
        y, total = new(T, H), new(T, H) if residual is not None else None
        wdt = "f32" if self.norm_weight.dtype == torch.float32 else "bf16"
        b.add_rms_norm(b.norm_problem(T, H, weight_dtype=wdt, eps=self.eps), x, self.norm_weight, residual, total, y)
        width = (Hq + 2 * Hkv) * D
        qkv = new(T, width)
        b.linear(b.linear_problem(T, width, H), y, self.wqkv, qkv, self.op_ws, bias=self.bias)
        q, k, v = qkv.split((Hq * D, Hkv * D, Hkv * D), dim=1)
        if cache is not None:
            r = b.rope_problem(T, Hq, Hkv, D, cache_dtype=cache.cache_dtype, page_size=cache.page_size,
                               num_pages=cache.num_pages, **self.rope)
            b.qk_norm_rope(r, q, k, positions, self.turns, q, self.op_ws, v=v, k_cache=cache.k, v_cache=cache.v,
                           slots=slots, k_scale=cache.k_scale, v_scale=cache.v_scale, q_weight=self.q_norm,
                           k_weight=self.k_norm)
            p = b.attention_problem(T, cu_q.shape[0] - 1, Hq, Hkv, D, max_q, cache_dtype=cache.cache_dtype,
                                    page_size=cache.page_size, num_pages=cache.num_pages,
                                    max_pages=page_table.shape[1], scale=self.scale)
        else:
            b.qk_norm_rope(b.rope_problem(T, Hq, Hkv, D, **self.rope), q, k, positions, self.turns, q, self.op_ws,
                           k_out=k, q_weight=self.q_norm, k_weight=self.k_norm)
            p = b.attention_problem(T, cu_q.shape[0] - 1, Hq, Hkv, D, max_q, scale=self.scale)
        ws = b.workspace_of(self, "attention_ws", b.attention_workspace_size(p),
                            lambda: b.alloc_attention_workspace(p, dev))
        # (rows of no sequence are not written by the attention: they stay zero)
        o = torch.zeros((T, Hq * D), dtype=torch.bfloat16, device=dev)
        if cache is not None:
            b.paged_attention(p, q, cache.k, cache.v, page_table, cu_q, kv_len, o, ws, k_scale=cache.k_scale,
                              v_scale=cache.v_scale)
        else:
            b.prompt_attention(p, q, k, v, cu_q, o, ws)
        out = new(T, H)
        b.linear(b.linear_problem(T, H, Hq * D), o, self.wo, out, self.op_ws)
        return out, total if total is not None else x

    def device_error(self, stream=None) -> int:
        """First error that a kernel of the block recorded (0: none), cleared; synchronises the stream.  Then
        the block can be used again."""
        return _first_error(stream, self.left, self.op_ws, self.attention_ws, *self.kept)


class DecoderLayer:
    """`layer(x, residual, positions, cu_q, max_q, ...)` -> (out, residual): an AttentionBlock, then a MoEBlock; the
    arguments are AttentionBlock's."""

    def __init__(self, attention: AttentionBlock, moe: MoEBlock):
        self.attention, self.moe = attention, moe

    def __call__(self, x, residual, positions, cu_q, max_q, stream=None, **cache):
        out, total = self.attention(x, residual, positions, cu_q, max_q, stream=stream, **cache)
        return self.moe(out, total, stream=stream)

    def device_error(self, stream=None) -> int:
        return self.attention.device_error(stream) or self.moe.device_error(stream)
