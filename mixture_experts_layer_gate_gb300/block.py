"""One pre-norm MoE block of a decoder, from the residual stream to what is added to it next.

Residual add + RMS norm, router scores, the routed experts and a shared expert
in block-scaled 8-bit floating point (the DeepSeek-V3 block: every token passes
through its routed experts and one shared expert, both on the normed input).
"""
from __future__ import annotations

from . import binding as b


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
        self.few_ws, self.kept = None, []  # kept: workspaces that captured graphs use
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
        """First error that a kernel of the block recorded (0: none), cleared; synchronises the stream."""
        all_ws = (self.op_ws, self.few_ws, self.layer.ws, *self.kept, *self.layer.kept)
        found = [b.get_device_error(ws, stream) for ws in all_ws if ws is not None]
        return next((e for e in found if e), 0)
