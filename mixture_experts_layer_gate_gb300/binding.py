"""ctypes binding of the C ABI in include/moe.h.

Argument marshalling only: every function passes tensor device pointers, sizes
and the current CUDA stream to the library, which does all the work in its own
kernels.  PyTorch is used for device memory and streams.  If the shared library
has not been built, loading it raises (there is no fallback path).
"""
from __future__ import annotations

import ctypes
import os

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libmoe_gb300.so")

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
                4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE_BAD_INDEX", 6: "MOE_ERR_TIMEOUT"}
WDTYPES = {"bf16": 0, "fp8": 1, "int4": 2, "int8": 3, "int4_paired": 4}
ACT_SCALES = {"static": 0, "dynamic": 1}
SCORING = {"softmax": 0, "sigmoid": 1}

EXPORTED = ("moe_scratch_size", "moe_workspace_size", "moe_padded_capacity", "moe_gate_topk",
            "moe_align_permute", "moe_align_block_size", "moe_grouped_gemm_swiglu",
            "moe_grouped_gemm_down", "moe_unpermute_reduce", "moe_forward", "moe_get_device_error",
            "moe_status_string", "moe_get_plan", "moe_get_plan_for_sms", "moe_align_permute_noalloc",
            "moe_dynamic_scales", "moe_launch_count", "moe_set_tuning", "moe_repack_int4",
            "moe_add_rms_norm", "moe_router_logits", "moe_gemm_fp8_block", "moe_gemm_fp8_block_swiglu",
            "moe_few_workspace_size", "moe_forward_few", "moe_qk_norm_rope", "moe_linear",
            "moe_attention_workspace_size", "moe_paged_attention", "moe_prompt_attention")

DTYPES = {"bf16": 0, "f16": 1, "f32": 2}
QUANTS = {"none": 0, "block": 1, "token": 2}
OP_WORKSPACE_BYTES = 256 + 4096 + 4 * 8 * 16384
FEW_MAX_TOKENS = 8
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}
LAYOUTS = {"half": 0, "interleaved": 1}


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({status_string(status)})")


class Problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("top_k", ctypes.c_int32), ("scoring", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("routed_scaling_factor", ctypes.c_float),
                ("wdtype", ctypes.c_int32), ("group_size", ctypes.c_int32), ("act_scale", ctypes.c_int32)]

    @property
    def S(self) -> int:
        return self.T * self.top_k


class WeightsStruct(ctypes.Structure):
    _fields_ = [("w13", ctypes.c_void_p), ("w2", ctypes.c_void_p), ("w13_scale", ctypes.c_void_p),
                ("w2_scale", ctypes.c_void_p), ("a1_scale", ctypes.c_void_p),
                ("a2_scale", ctypes.c_void_p), ("w13_zero", ctypes.c_void_p), ("w2_zero", ctypes.c_void_p)]


class Plan(ctypes.Structure):
    _fields_ = [("bn_max_up", ctypes.c_int32), ("splits_up", ctypes.c_int32),
                ("stages_up", ctypes.c_int32), ("astages_up", ctypes.c_int32), ("smem_up", ctypes.c_int32),
                ("bn_max_down", ctypes.c_int32), ("splits_down", ctypes.c_int32),
                ("stages_down", ctypes.c_int32), ("astages_down", ctypes.c_int32),
                ("smem_down", ctypes.c_int32), ("num_sms", ctypes.c_int32),
                ("slot_kb_up", ctypes.c_int32), ("slot_kb_down", ctypes.c_int32),
                ("pair_up", ctypes.c_int32), ("pair_down", ctypes.c_int32),
                ("issuers_up", ctypes.c_int32), ("issuers_down", ctypes.c_int32),
                ("conv_groups_up", ctypes.c_int32), ("conv_groups_down", ctypes.c_int32),
                ("epi_warps_up", ctypes.c_int32), ("epi_warps_down", ctypes.c_int32),
                ("acc_bufs_up", ctypes.c_int32), ("acc_bufs_down", ctypes.c_int32)]


class Tuning(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("bn_max", "stages", "splits", "pair", "conv_groups", "slot_kb",
                                             "ksplit", "dual", "full_box", "w_stream", "unit_order",
                                             "epi_warps", "acc_bufs")]


class NormProblem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("quant", ctypes.c_int32), ("eps", ctypes.c_float)]


class RouterProblem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Fp8GemmProblem(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("accumulate", ctypes.c_int32)]


class KvStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)] + [(n, ctypes.c_int64) for n in (
                    "k_page_stride", "k_token_stride", "k_head_stride", "v_page_stride", "v_token_stride",
                    "v_head_stride")]


class LinearProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "dtype", "out_dtype", "activation")]


class RopeProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "Hq", "Hkv", "D", "rot", "interleaved", "dtype", "weight_dtype",
                                             "cache_dtype", "page_size", "num_pages")] + [
        ("eps", ctypes.c_float), ("magnitude", ctypes.c_float)]


class AttentionProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "B", "Hq", "Hkv", "D", "max_q", "dtype", "cache_dtype", "page_size",
                                             "num_pages", "max_pages")] + [("scale", ctypes.c_float)]


TUNING_KNOBS = tuple(n for n, _ in Tuning._fields_)

_lib = None


def load(path: str = LIB_PATH):
    """Loads the shared library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first (python -m mixture_experts_layer_gate_gb300.build)")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(Problem)
    vp, sz, i32, st = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int
    i64 = ctypes.c_int64
    sig = {
        "moe_scratch_size": (sz, [P]),
        "moe_workspace_size": (sz, [P]),
        "moe_padded_capacity": (sz, [P, i32]),
        "moe_gate_topk": (st, [P, vp, vp, vp, vp, vp]),
        "moe_align_permute": (st, [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "moe_align_block_size": (st, [P, vp, vp, i32, vp, vp, vp, vp]),
        "moe_align_permute_noalloc": (st, [P, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_grouped_gemm_swiglu": (st, [P, ctypes.POINTER(WeightsStruct), vp, vp, vp, vp, sz, vp]),
        "moe_grouped_gemm_down": (st, [P, ctypes.POINTER(WeightsStruct), vp, vp, vp, vp, sz, vp]),
        "moe_unpermute_reduce": (st, [P, vp, vp, vp, vp, vp, sz, vp]),
        "moe_forward": (st, [P, ctypes.POINTER(WeightsStruct), vp, vp, vp, vp, vp, sz, vp]),
        "moe_get_device_error": (st, [vp, vp]),
        "moe_status_string": (ctypes.c_char_p, [st]),
        "moe_get_plan": (st, [P, ctypes.POINTER(Plan)]),
        "moe_get_plan_for_sms": (st, [P, i32, ctypes.POINTER(Plan)]),
        "moe_dynamic_scales": (vp, [vp]),
        "moe_launch_count": (ctypes.c_uint64, []),
        "moe_set_tuning": (st, [ctypes.POINTER(Tuning)]),
        "moe_repack_int4": (st, [vp, vp, sz, vp]),
        "moe_add_rms_norm": (st, [ctypes.POINTER(NormProblem), vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp, vp]),
        "moe_router_logits": (st, [ctypes.POINTER(RouterProblem), vp, i64, vp, i64, vp, vp, sz, vp]),
        "moe_gemm_fp8_block": (st, [ctypes.POINTER(Fp8GemmProblem), vp, i64, vp, i64, vp, i64, vp, vp, i64, vp, sz,
                                    vp]),
        "moe_gemm_fp8_block_swiglu": (st, [ctypes.POINTER(Fp8GemmProblem), vp, i64, vp, i64, vp, i64, vp, vp, vp, vp,
                                           sz, vp]),
        "moe_few_workspace_size": (sz, [P]),
        "moe_forward_few": (st, [P, ctypes.POINTER(WeightsStruct), vp, vp, vp, vp, vp, sz, vp]),
        "moe_linear": (st, [ctypes.POINTER(LinearProblem), vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, sz, vp]),
        "moe_attention_workspace_size": (sz, [ctypes.POINTER(AttentionProblem)]),
        "moe_paged_attention": (st, [ctypes.POINTER(AttentionProblem), vp, i64, ctypes.POINTER(KvStruct), vp, i64, vp,
                                     vp, vp, i64, vp, vp, sz, vp]),
        "moe_prompt_attention": (st, [ctypes.POINTER(AttentionProblem), vp, i64, vp, i64, vp, i64, vp, vp, i64, vp, vp,
                                      sz, vp]),
        "moe_qk_norm_rope": (st, [ctypes.POINTER(RopeProblem), vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, i64, vp,
                                  i64, ctypes.POINTER(KvStruct), vp, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load().moe_status_string(int(status)).decode()
    except Exception:  # library missing: still report the code
        return STATUS_NAMES.get(status, str(status))


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


_raw_stream = None


def _stream(stream):
    """The given raw stream, or the current one of the current device."""
    global _raw_stream
    if stream is not None:
        return int(stream)
    if _raw_stream is None:
        import torch
        device, raw = getattr(torch._C, "_cuda_getDevice", None), getattr(torch._C, "_cuda_getCurrentRawStream", None)
        torch.cuda.current_stream()  # initialises CUDA
        if device is None or raw is None:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        else:  # 0.2 us a call instead of the stream object's 2.9 us
            _raw_stream = lambda: raw(device())  # noqa: E731
    return _raw_stream()


def run_on(stream, call, *args):
    """call(*args) with the given raw stream as PyTorch's current one (None: as it is), for calls that allocate: what
    they allocate then belongs to the stream that their kernels run on.  Tensors that cross streams are kept from
    reuse until both have done their work: the arguments (and what they hold as their `tensors`) on the given stream,
    the results on the caller's."""
    if stream is None or int(stream) == _stream(None):
        return call(*args)
    import torch
    caller = torch.cuda.current_stream()
    side = torch.cuda.ExternalStream(0 if int(stream) == 1 else int(stream))  # (1: cudaStreamLegacy, the default one)
    for arg in args:
        for t in getattr(arg, "tensors", (arg,)):
            if isinstance(t, torch.Tensor):
                t.record_stream(side)
    with torch.cuda.stream(side):
        results = call(*args)
    for t in results if isinstance(results, tuple) else (results,):
        t.record_stream(caller)
    return results


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoEError(status, where)


def problem(T, H, I, E, top_k, scoring="softmax", renormalize=True, n_group=0, topk_group=0,
            routed_scaling_factor=1.0, wdtype="bf16", group_size=128, act_scale="static") -> Problem:
    return Problem(int(T), int(H), int(I), int(E), int(top_k), SCORING[scoring], int(bool(renormalize)),
                   int(n_group), int(topk_group), float(routed_scaling_factor), WDTYPES[wdtype],
                   int(group_size), ACT_SCALES[act_scale])


class Weights:
    """Expert weights as the library reads them; keeps the tensors alive."""

    def __init__(self, w13, w2, w13_scale=None, w2_scale=None, a1_scale=None, a2_scale=None,
                 w13_zero=None, w2_zero=None):
        self.tensors = (w13, w2, w13_scale, w2_scale, a1_scale, a2_scale, w13_zero, w2_zero)
        self.struct = WeightsStruct(*[None if t is None else t.data_ptr() for t in self.tensors])


def scratch_size(p: Problem) -> int:
    return int(load().moe_scratch_size(ctypes.byref(p)))


def workspace_size(p: Problem) -> int:
    return int(load().moe_workspace_size(ctypes.byref(p)))


def padded_capacity(p: Problem, block: int) -> int:
    return int(load().moe_padded_capacity(ctypes.byref(p), int(block)))


def alloc_workspace(p: Problem, device, full: bool = True):
    """Zeroed workspace (the error header must start at zero)."""
    import torch
    n = workspace_size(p) if full else scratch_size(p)
    if n == 0:
        raise MoEError(1, "workspace size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def gate_topk(p: Problem, logits, bias, topk_ids, topk_w, stream=None):
    _check(load().moe_gate_topk(ctypes.byref(p), _ptr(logits), _ptr(bias), _ptr(topk_ids), _ptr(topk_w),
                                _stream(stream)), "moe_gate_topk")


def align_permute(p: Problem, topk_ids, x, a1_scale, counts, offsets, perm, inv, x_perm, ws, stream=None):
    _check(load().moe_align_permute(ctypes.byref(p), _ptr(topk_ids), _ptr(x), _ptr(a1_scale), _ptr(counts),
                                    _ptr(offsets), _ptr(perm), _ptr(inv), _ptr(x_perm), _ptr(ws),
                                    ws.numel(), _stream(stream)), "moe_align_permute")


def align_permute_noalloc(p: Problem, topk_ids, x, a1_scale, counts, offsets, perm, inv, x_perm, stream=None):
    """moe_align_permute for callers that cannot allocate: no workspace argument;
    the library's fixed device-side array holds the scratch (see include/moe.h)."""
    _check(load().moe_align_permute_noalloc(ctypes.byref(p), _ptr(topk_ids), _ptr(x), _ptr(a1_scale),
                                            _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv), _ptr(x_perm),
                                            _stream(stream)), "moe_align_permute_noalloc")


def align_block_size(p: Problem, offsets, perm, block, sorted_ids, block_expert, total_padded, stream=None):
    _check(load().moe_align_block_size(ctypes.byref(p), _ptr(offsets), _ptr(perm), int(block),
                                       _ptr(sorted_ids), _ptr(block_expert), _ptr(total_padded),
                                       _stream(stream)), "moe_align_block_size")


def grouped_gemm_swiglu(p: Problem, w: Weights, x_perm, offsets, act, ws, stream=None):
    _check(load().moe_grouped_gemm_swiglu(ctypes.byref(p), ctypes.byref(w.struct), _ptr(x_perm),
                                          _ptr(offsets), _ptr(act), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_grouped_gemm_swiglu")


def grouped_gemm_down(p: Problem, w: Weights, act, offsets, y_perm, ws, stream=None):
    _check(load().moe_grouped_gemm_down(ctypes.byref(p), ctypes.byref(w.struct), _ptr(act), _ptr(offsets),
                                        _ptr(y_perm), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_grouped_gemm_down")


def unpermute_reduce(p: Problem, y_perm, inv, topk_w, out, ws, stream=None):
    _check(load().moe_unpermute_reduce(ctypes.byref(p), _ptr(y_perm), _ptr(inv), _ptr(topk_w), _ptr(out),
                                       _ptr(ws), ws.numel(), _stream(stream)), "moe_unpermute_reduce")


def forward(p: Problem, w: Weights, x, logits, bias, out, ws, stream=None):
    _check(load().moe_forward(ctypes.byref(p), ctypes.byref(w.struct), _ptr(x), _ptr(logits), _ptr(bias),
                              _ptr(out), _ptr(ws), ws.numel(), _stream(stream)), "moe_forward")


def get_device_error(ws, stream=None) -> int:
    """Synchronises the stream; returns (and clears) the sticky device error code."""
    return int(load().moe_get_device_error(_ptr(ws), _stream(stream)))


def launch_count() -> int:
    """Kernel launches the library has issued in this process (graph captures once)."""
    return int(load().moe_launch_count())


def repack_int4(codes, out=None, stream=None):
    """int4 codes (uint8 tensor, packed order) -> a tensor of the same shape in the
    paired order of MOE_W_INT4_G128_PAIRED (moe_repack_int4); `out` may be
    `codes` itself (in place) but must not partly overlap it.  Returns the output
    tensor."""
    import torch
    if out is None:
        out = torch.empty_like(codes)
    if out.numel() != codes.numel() or codes.dtype != torch.uint8 or out.dtype != torch.uint8:
        raise ValueError("repack_int4: uint8 tensors of equal size")
    if not (codes.is_contiguous() and out.is_contiguous()):
        raise ValueError("repack_int4: contiguous tensors")
    _check(load().moe_repack_int4(_ptr(codes), _ptr(out), codes.numel(), _stream(stream)), "moe_repack_int4")
    return out


def dynamic_scales(ws):
    """The workspace's dynamic fp8 scales {a1, a2} as a float32 view [2] of ws."""
    import torch
    ptr = load().moe_dynamic_scales(_ptr(ws))
    if not ptr:
        raise MoEError(1, "moe_dynamic_scales")
    off = ptr - ws.data_ptr()
    return ws[off: off + 8].view(torch.float32)


def get_plan(p: Problem, num_sms: int | None = None) -> Plan:
    """Launch plan on the current device, or for `num_sms` SMs (no GPU needed)."""
    plan = Plan()
    if num_sms is None:
        _check(load().moe_get_plan(ctypes.byref(p), ctypes.byref(plan)), "moe_get_plan")
    else:
        _check(load().moe_get_plan_for_sms(ctypes.byref(p), int(num_sms), ctypes.byref(plan)),
               "moe_get_plan_for_sms")
    return plan


def set_tuning(**knobs):
    """Planner overrides (moe_set_tuning): keyword per knob, e.g. pair=0, dual=1;
    no keywords restores the planner's choices.  For tests and benchmarks."""
    unknown = set(knobs) - set(TUNING_KNOBS)
    if unknown:
        raise ValueError(f"unknown tuning knobs {sorted(unknown)}")
    if not knobs:
        _check(load().moe_set_tuning(None), "moe_set_tuning")
        return
    t = Tuning(*[int(knobs.get(n, -1)) for n in TUNING_KNOBS])
    _check(load().moe_set_tuning(ctypes.byref(t)), "moe_set_tuning")


class tuning:
    """Context manager: planner overrides inside the block, defaults after it."""

    def __init__(self, **knobs):
        self.knobs = knobs

    def __enter__(self):
        set_tuning(**self.knobs)
        return self

    def __exit__(self, *exc):
        set_tuning()


# ------------------------------------------------------- operators around the layer


def norm_problem(T, H, dtype="bf16", weight_dtype=None, eps=1e-6, quant="none") -> NormProblem:
    """T rows of H columns for add_rms_norm; quant: "none", "block" (a scale per 128 columns) or "token"."""
    return NormProblem(int(T), int(H), DTYPES[dtype], DTYPES[weight_dtype or dtype], QUANTS[quant], float(eps))


def router_problem(T, H, E, dtype="bf16") -> RouterProblem:
    return RouterProblem(int(T), int(H), int(E), DTYPES[dtype])


def fp8_gemm_problem(M, N, K, out_dtype="bf16", accumulate=False) -> Fp8GemmProblem:
    """M rows, N output columns, depth K; for gemm_fp8_block_swiglu the weight has 2N rows.  accumulate: the
    product is added to out."""
    return Fp8GemmProblem(int(M), int(N), int(K), DTYPES[out_dtype], int(bool(accumulate)))


def alloc_op_workspace(device):
    """Zeroed workspace (error header and scratch) for router_logits, linear, qk_norm_rope and the gemm_fp8_block calls
    of one stream."""
    import torch
    return torch.zeros(OP_WORKSPACE_BYTES, dtype=torch.uint8, device=device)


_ops = None


def _native():
    """The compiled entries of the operators below (csrc/binding.cpp): they check tensors against the problem."""
    global _ops
    if _ops is None:
        load()
        import torch  # noqa: F401  (its libraries first)
        try:
            from . import _ops as module
        except ImportError as e:
            raise RuntimeError("_ops.so is missing or does not fit this PyTorch: build it first "
                               "(python -m mixture_experts_layer_gate_gb300.build)") from e
        _ops = module
    return _ops


def add_rms_norm(n: NormProblem, x, weight, residual=None, residual_out=None, y=None, codes=None, scales=None,
                 stream=None):
    """moe_add_rms_norm.  x, residual, residual_out, y: [T, H] of n's dtype (rows may be strided; residual_out may
    be residual); weight [H]; codes [T, H] (uint8 or float8_e4m3fn) and scales (float32, [T, ceil(H / 128)] or
    [T]) exactly where n quantises."""
    _check((_ops or _native()).add_rms_norm(n, x, weight, residual, residual_out, y, codes, scales, stream),
           "moe_add_rms_norm")


def router_logits(r: RouterProblem, x, w, logits, ws, stream=None):
    """moe_router_logits: x [T, H] and w [E, H] (rows may be strided) -> logits float32 [T, E]."""
    _check((_ops or _native()).router_logits(r, x, w, logits, ws, stream), "moe_router_logits")


def gemm_fp8_block(g: Fp8GemmProblem, a, a_scale, w, w_scale, out, ws, stream=None):
    """moe_gemm_fp8_block: a [M, K], w [N, K] (uint8 or float8_e4m3fn), a_scale [M, ceil(K / 128)] and w_scale
    [ceil(N / 128), ceil(K / 128)] float32 -> out [M, N] of g's out_dtype."""
    _check((_ops or _native()).gemm_fp8_block(g, a, a_scale, w, w_scale, out, ws, stream), "moe_gemm_fp8_block")


def gemm_fp8_block_swiglu(g: Fp8GemmProblem, a, a_scale, w13, w13_scale, codes, scales, ws, stream=None):
    """moe_gemm_fp8_block_swiglu: a [M, K], w13 [2N, K] with their scales -> codes [M, N], scales [M, N / 128]."""
    _check((_ops or _native()).gemm_fp8_block_swiglu(g, a, a_scale, w13, w13_scale, codes, scales, ws, stream),
           "moe_gemm_fp8_block_swiglu")


def few_workspace_size(p: Problem) -> int:
    return int(load().moe_few_workspace_size(ctypes.byref(p)))


def alloc_few_workspace(p: Problem, device):
    """Zeroed workspace for forward_few."""
    import torch
    n = few_workspace_size(p)
    if n == 0:
        raise MoEError(2 if p.T > FEW_MAX_TOKENS else 1, "few workspace size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def forward_few(p: Problem, w: Weights, x, logits, bias, out, ws, stream=None):
    """moe_forward_few: the whole layer for at most FEW_MAX_TOKENS tokens in two launches."""
    _check((_ops or _native()).forward_few(p, w.struct, x, logits, bias, out, ws, stream), "moe_forward_few")


# ------------------------------------------------- the attention half of a block


def linear_problem(M, N, K, dtype="bf16", out_dtype=None, activation="none") -> LinearProblem:
    """M rows, N output columns, depth K; out (and residual) of out_dtype, dtype without it; activation: "none", "silu",
    "gelu", "gelu_tanh" or "relu"."""
    return LinearProblem(int(M), int(N), int(K), DTYPES[dtype], DTYPES[out_dtype or dtype], ACTIVATIONS[activation])


def linear(p: LinearProblem, x, w, out, ws, bias=None, residual=None, stream=None):
    """moe_linear: out = act(x w^T + bias) + residual; x [M, K] and w [N, K] (rows may be strided), bias [N] of p's
    dtype, residual [M, N] (may be out)."""
    _check((_ops or _native()).linear(p, x, w, out, ws, bias, residual, stream), "moe_linear")


def _cache_code(cache_dtype, dtype) -> int:
    """MOE_CACHE_SAME or MOE_CACHE_E4M3 of a cache of dtype's values or "e4m3"."""
    if cache_dtype == "e4m3":
        return 1
    if cache_dtype not in (None, dtype):
        raise ValueError(f"cache_dtype: {dtype!r} or 'e4m3'")
    return 0


def rope_problem(T, Hq, Hkv, D, rot=None, layout="half", dtype="bf16", weight_dtype=None, eps=1e-6, magnitude=1.0,
                 cache_dtype=None, page_size=0, num_pages=0) -> RopeProblem:
    """T tokens of Hq query and Hkv key and value heads of D values for qk_norm_rope; rot (all D without it) of them
    are rotated, as pairs (i, i + rot / 2) ("half") or (2 i, 2 i + 1) ("interleaved").  With page_size and num_pages
    keys and values go to a paged cache, of dtype's values or "e4m3"."""
    return RopeProblem(int(T), int(Hq), int(Hkv), int(D), int(D if rot is None else rot), LAYOUTS[layout],
                       DTYPES[dtype], DTYPES[weight_dtype or dtype], _cache_code(cache_dtype, dtype), int(page_size),
                       int(num_pages), float(eps), float(magnitude))


def rope_table(rot, theta=10000.0, factor=1.0, original=0, low=1.0, high=1.0, inv_freq=None, device=None):
    """The turns of qk_norm_rope (int64 [rot / 2], in 2^-64 of a turn a position): pair i turns theta^(-2 i / rot)
    radians a position (or inv_freq[i], float64), for a context stretched `factor` times as g f + (1 - g) f / factor.
    Without `original` g = 0: every frequency is divided.  With it, g goes from 0 for pairs of at most `low` turns over
    the `original` positions to 1 for those of `high` and more, in proportion to the turns; a model whose g is in
    proportion to the pair's index gives its own inv_freq."""
    import math

    import torch
    if rot < 0 or rot % 2 or not (factor > 0 and math.isfinite(factor)):
        raise ValueError("rope_table: an even rot and a positive factor")
    if inv_freq is None:
        freq = [float(theta) ** (-2.0 * i / rot) for i in range(rot // 2)]
    else:
        freq = [float(f) for f in inv_freq]
    if len(freq) != rot // 2 or not all(math.isfinite(f) for f in freq):
        raise ValueError("rope_table: rot / 2 finite frequencies")
    table = []
    for f in freq:
        keep = 0.0
        if factor == 1.0:
            keep = 1.0
        elif original:
            seen = original * f / (2.0 * math.pi)
            keep = min(1.0, max(0.0, (seen - low) / (high - low))) if high > low else float(seen >= high)
        turn = (keep * f + (1.0 - keep) * f / factor) / (2.0 * math.pi)
        whole = int((turn - math.floor(turn)) * 2.0 ** 64) % 2 ** 64
        table.append(whole - 2 ** 64 if whole >= 2 ** 63 else whole)
    return torch.tensor(table, dtype=torch.int64, device=device)


def qk_norm_rope(r: RopeProblem, q, k, positions, turns, q_out, ws, k_out=None, v=None, k_cache=None, v_cache=None,
                 slots=None, k_scale=None, v_scale=None, q_weight=None, k_weight=None, stream=None):
    """moe_qk_norm_rope.  q, q_out [T, Hq * D] and k, v, k_out [T, Hkv * D] of r's dtype (rows may be strided; outputs
    may be the inputs), positions int32 [T], turns of rope_table; weights [D] or None; k_cache, v_cache [num_pages,
    page_size, Hkv, D] of any order in memory with slots int32 [T], and for "e4m3" k_scale, v_scale float32 [num_pages,
    Hkv, page_size]."""
    _check((_ops or _native()).qk_norm_rope(r, q, k, v, positions, turns, q_weight, k_weight, q_out, k_out, k_cache,
                                            v_cache, k_scale, v_scale, slots, ws, stream), "moe_qk_norm_rope")


def attention_problem(T, B, Hq, Hkv, D, max_q, dtype="bf16", cache_dtype=None, page_size=0, num_pages=0, max_pages=0,
                      scale=None) -> AttentionProblem:
    """T rows of Hq query heads of D values, the new tokens of B sequences (max_q of one at most), against Hkv key and
    value heads.  For paged_attention with the cache's page_size, num_pages and type (dtype's values or "e4m3") and the
    page table's columns max_pages; scale: of the scores, 1 / sqrt(D) without it."""
    return AttentionProblem(int(T), int(B), int(Hq), int(Hkv), int(D), int(max_q), DTYPES[dtype],
                            _cache_code(cache_dtype, dtype), int(page_size), int(num_pages), int(max_pages),
                            float(D) ** -0.5 if scale is None else float(scale))


def attention_workspace_size(p: AttentionProblem) -> int:
    return int(load().moe_attention_workspace_size(ctypes.byref(p)))


def alloc_attention_workspace(p: AttentionProblem, device):
    """Zeroed workspace for the attention calls of one stream, of p and of problems with no longer heads and no more
    rows a key head (max_q * Hq / Hkv)."""
    import torch
    n = attention_workspace_size(p)
    if n == 0:
        raise MoEError(1, "attention workspace size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def paged_attention(p: AttentionProblem, q, k_cache, v_cache, page_table, cu_q, kv_len, out, ws, k_scale=None,
                    v_scale=None, lse=None, stream=None):
    """moe_paged_attention.  q, out [T, Hq * D] (rows may be strided); k_cache, v_cache [num_pages, page_size, Hkv, D] of
    any order in memory, for "e4m3" with k_scale, v_scale float32 [num_pages, Hkv, page_size]; page_table int32 [B,
    max_pages], cu_q int32 [B + 1], kv_len int32 [B]; lse float32 [T, Hq] or None."""
    _check((_ops or _native()).paged_attention(p, q, k_cache, v_cache, k_scale, v_scale, page_table, cu_q, kv_len, out,
                                               lse, ws, stream), "moe_paged_attention")


def prompt_attention(p: AttentionProblem, q, k, v, cu_q, out, ws, lse=None, stream=None):
    """moe_prompt_attention: q, out [T, Hq * D] and k, v [T, Hkv * D] (rows may be strided), cu_q int32 [B + 1], lse
    float32 [T, Hq] or None."""
    _check((_ops or _native()).prompt_attention(p, q, k, v, cu_q, out, lse, ws, stream), "moe_prompt_attention")


def workspace_of(owner, name: str, n: int, allocate):
    """A workspace of at least n bytes for a call: owner's attribute `name`, which allocate() replaces where it is too
    small.  One that a captured graph uses stays alive in owner.kept, and one whose zero fill is being captured
    serves that capture alone.  Of those that go owner.left keeps the error header, the first with an error if any."""
    import torch
    ws, capturing = getattr(owner, name), torch.cuda.is_current_stream_capturing()
    if ws is not None and n <= ws.numel():
        if capturing and not any(w is ws for w in owner.kept):
            owner.kept.append(ws)
        return ws
    new = allocate()
    if capturing:
        owner.kept.append(new)
        return new
    if ws is not None and not any(w is ws for w in owner.kept):
        header = ws[:256].clone()
        owner.left = header if owner.left is None else torch.where(owner.left.view(torch.int32)[0] != 0, owner.left, header)
        ws.record_stream(torch.cuda.current_stream())  # its calls may still run there
    setattr(owner, name, new)
    return new


class MoELayer:
    """Convenience wrapper: one problem shape (up to a token budget), its weights
    and a workspace; `__call__` runs moe_forward on the given raw stream or the current
    one, and allocates there what it needs."""

    def __init__(self, H, I, E, top_k, weights: Weights, max_tokens: int, device, **gate):
        self.shape = dict(H=H, I=I, E=E, top_k=top_k, **gate)
        self.weights = weights
        self.kept, self.left = [], None  # workspaces that captured graphs use; the error header of those outgrown
        self.ws = alloc_workspace(problem(max_tokens, H, I, E, top_k, **gate), device)

    def problem(self, T: int) -> Problem:
        return problem(T, **self.shape)

    def __call__(self, x, logits, bias=None, out=None, stream=None):
        return run_on(stream, self._run, x, logits, bias, out)

    def _run(self, x, logits, bias, out):
        import torch
        T = x.shape[0]
        if out is None:
            out = torch.empty((T, self.shape["H"]), dtype=torch.bfloat16, device=x.device)
        p = self.problem(T)
        ws = workspace_of(self, "ws", workspace_size(p), lambda: alloc_workspace(p, x.device))
        forward(p, self.weights, x, logits, bias, out, ws)
        return out
