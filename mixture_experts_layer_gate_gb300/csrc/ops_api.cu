// Host side of the operators around the layer declared in include/moe.h:
// argument checks and launches.
#include <cmath>

#include "../../include/moe.h"
#include "checks.h"
#include "common.cuh"
#include "kernels.h"

using namespace moe;

namespace {

struct FewLayout {
  size_t amax, act, total;
};

FewLayout few_layout(const moe_problem_t& p) {
  const size_t S = static_cast<size_t>(p.T) * p.top_k;
  FewLayout L;
  size_t o = kHeaderBytes;
  L.amax = o;
  o = align256(o + kFewMaxCtas * 4);
  L.act = o;
  o = align256(o + S * p.I * 4);
  L.total = o;
  return L;
}

bool few_fits(const moe_problem_t& p) {
  const long long values = static_cast<long long>(p.T) * (p.H + 32);
  const bool int4 = p.wdtype == MOE_W_INT4_G128 || p.wdtype == MOE_W_INT4_G128_PAIRED;
  return p.T <= kFewMaxTokens && values <= kFewMaxTokenValues && (!int4 || values + p.H / 8 <= kFewMaxInt4Values);
}

moe_status_t check_fp8_gemm(const moe_fp8_gemm_t* g, const void* a, int64_t a_stride, const float* a_scale,
                            int64_t a_scale_stride, const void* w, int64_t w_stride, const float* w_scale) {
  const int64_t kb = (static_cast<int64_t>(g->K) + 127) / 128;
  if (!rows_ok(a, a_stride, g->K, 16) || a_stride % 16 != 0) return MOE_ERR_INVALID_ARG;
  if (!rows_ok(w, w_stride, g->K, 16) || w_stride % 16 != 0) return MOE_ERR_INVALID_ARG;
  if (!rows_ok(a_scale, a_scale_stride, kb, 4) || w_scale == nullptr || !aligned(w_scale, 4))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status_t validate_fp8_gemm(const moe_fp8_gemm_t* g) {
  if (g == nullptr || g->M < 0 || g->N < 0 || g->K < 16 || g->K % 16 != 0) return MOE_ERR_INVALID_ARG;
  if (g->accumulate != 0 && g->accumulate != 1) return MOE_ERR_INVALID_ARG;
  if (g->M > (1 << 22) || g->N > (1 << 22)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_add_rms_norm(const moe_norm_t* n, const void* x, int64_t x_stride, const void* residual,
                              int64_t residual_stride, const void* weight, void* residual_out,
                              int64_t residual_out_stride, void* y, int64_t y_stride, void* codes,
                              float* scales, moe_stream_t stream) {
  if (n == nullptr || n->T < 0 || n->H < 1 || !is_dtype(n->dtype)) return MOE_ERR_INVALID_ARG;
  if (n->weight_dtype != n->dtype && n->weight_dtype != MOE_T_F32) return MOE_ERR_INVALID_ARG;
  if (n->quant < MOE_QUANT_NONE || n->quant > MOE_QUANT_TOKEN) return MOE_ERR_INVALID_ARG;
  if (!(n->eps >= 0.f) || !std::isfinite(n->eps)) return MOE_ERR_INVALID_ARG;
  if (n->H > 16384 || n->T > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  if (n->T == 0) return MOE_OK;
  const size_t b = size_of(n->dtype), wb = size_of(n->weight_dtype);
  if (!rows_ok(x, x_stride, n->H, b) || weight == nullptr || !aligned(weight, wb)) return MOE_ERR_INVALID_ARG;
  if (residual != nullptr && !rows_ok(residual, residual_stride, n->H, b)) return MOE_ERR_INVALID_ARG;
  if (residual_out != nullptr && (residual == nullptr || !rows_ok(residual_out, residual_out_stride, n->H, b)))
    return MOE_ERR_INVALID_ARG;
  if (residual_out != nullptr && residual_out == residual && residual_out_stride != residual_stride)
    return MOE_ERR_INVALID_ARG;
  if (y != nullptr && !rows_ok(y, y_stride, n->H, b)) return MOE_ERR_INVALID_ARG;
  const bool quant = n->quant != MOE_QUANT_NONE;
  if (quant != (codes != nullptr) || quant != (scales != nullptr) || !aligned(scales, 4)) return MOE_ERR_INVALID_ARG;
  if (y == nullptr && residual_out == nullptr && !quant) return MOE_ERR_INVALID_ARG;
  NormArgs a;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.residual_out = residual_out;
  a.y = y;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.residual_out_stride = residual_out_stride;
  a.y_stride = y_stride;
  a.T = n->T;
  a.H = n->H;
  a.quant = n->quant;
  a.eps = n->eps;
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return MOE_ERR_CUDA;
  a.sms = di.sms;
  auto wide = [&](const void* p, int64_t stride) {
    return p == nullptr || (aligned(p, 16) && stride * static_cast<int64_t>(b) % 16 == 0);
  };
  a.vec = n->H % 8 == 0 && wide(x, x_stride) && wide(residual, residual_stride) &&
          wide(residual_out, residual_out_stride) && wide(y, y_stride) && aligned(weight, 16) && aligned(codes, 8);
  return cuda_status(
      launch_add_rms_norm(a, n->dtype, n->weight_dtype == MOE_T_F32, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_router_logits(const moe_router_t* r, const void* x, int64_t x_stride, const void* w,
                               int64_t w_stride, float* logits, void* ws, size_t ws_bytes,
                               moe_stream_t stream) {
  if (r == nullptr || r->T < 0 || r->H < 8 || r->H % 8 != 0 || r->E < 1) return MOE_ERR_INVALID_ARG;
  if (r->dtype != MOE_T_BF16 && r->dtype != MOE_T_F16) return MOE_ERR_INVALID_ARG;
  if (r->E > 1024 || r->T > (1 << 22)) return MOE_ERR_UNSUPPORTED;
  MOE_TRY(check_header(ws, ws_bytes));
  if (r->T == 0) return MOE_OK;
  if (!rows_ok(x, x_stride, r->H, 16) || x_stride % 8 != 0 || !rows_ok(w, w_stride, r->H, 16) || w_stride % 8 != 0)
    return MOE_ERR_INVALID_ARG;
  if (logits == nullptr || !aligned(logits, 4)) return MOE_ERR_INVALID_ARG;
  RouterArgs a;
  a.x = x;
  a.w = w;
  a.logits = logits;
  a.x_stride = x_stride;
  a.w_stride = w_stride;
  a.T = r->T;
  a.H = r->H;
  a.E = r->E;
  a.dtype = r->dtype;
  a.err = static_cast<uint32_t*>(ws);
  return cuda_status(launch_router(a, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_gemm_fp8_block(const moe_fp8_gemm_t* g, const void* a, int64_t a_stride, const float* a_scale,
                                int64_t a_scale_stride, const void* w, int64_t w_stride, const float* w_scale,
                                void* out, int64_t out_stride, void* ws, size_t ws_bytes, moe_stream_t stream) {
  MOE_TRY(validate_fp8_gemm(g));
  if (!is_dtype(g->out_dtype)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_header(ws, ws_bytes));
  if (g->M == 0 || g->N == 0) return MOE_OK;
  MOE_TRY(check_fp8_gemm(g, a, a_stride, a_scale, a_scale_stride, w, w_stride, w_scale));
  if (!rows_ok(out, out_stride, g->N, size_of(g->out_dtype))) return MOE_ERR_INVALID_ARG;
  Fp8GemmArgs f = {};
  f.a = static_cast<const uint8_t*>(a);
  f.w = static_cast<const uint8_t*>(w);
  f.a_scale = a_scale;
  f.w_scale = w_scale;
  f.out = out;
  f.a_stride = a_stride;
  f.a_scale_stride = a_scale_stride;
  f.w_stride = w_stride;
  f.out_stride = out_stride;
  f.M = g->M;
  f.N = g->N;
  f.K = g->K;
  f.out_dtype = g->out_dtype;
  f.accumulate = g->accumulate;
  f.err = static_cast<uint32_t*>(ws);
  return cuda_status(launch_fp8_block(f, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_gemm_fp8_block_swiglu(const moe_fp8_gemm_t* g, const void* a, int64_t a_stride,
                                       const float* a_scale, int64_t a_scale_stride, const void* w13,
                                       int64_t w13_stride, const float* w13_scale, void* codes, float* scales,
                                       void* ws, size_t ws_bytes, moe_stream_t stream) {
  MOE_TRY(validate_fp8_gemm(g));
  if (g->N % 128 != 0 || g->accumulate != 0) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_header(ws, ws_bytes));
  if (g->M == 0 || g->N == 0) return MOE_OK;
  MOE_TRY(check_fp8_gemm(g, a, a_stride, a_scale, a_scale_stride, w13, w13_stride, w13_scale));
  if (codes == nullptr || !aligned(codes, 16) || scales == nullptr || !aligned(scales, 4)) return MOE_ERR_INVALID_ARG;
  Fp8GemmArgs f = {};
  f.a = static_cast<const uint8_t*>(a);
  f.w = static_cast<const uint8_t*>(w13);
  f.a_scale = a_scale;
  f.w_scale = w13_scale;
  f.codes = static_cast<uint8_t*>(codes);
  f.scales = scales;
  if (g->M <= 8 && static_cast<size_t>(g->N) / 128 * 4 <= kFewTicketBytes &&
      ws_bytes >= kHeaderBytes + fp8_few_scratch(g->M, g->N)) {
    uint8_t* scratch = static_cast<uint8_t*>(ws) + kHeaderBytes;
    f.tickets = reinterpret_cast<uint32_t*>(scratch);
    f.act = reinterpret_cast<float*>(scratch + kFewTicketBytes);
  }
  f.a_stride = a_stride;
  f.a_scale_stride = a_scale_stride;
  f.w_stride = w13_stride;
  f.M = g->M;
  f.N = g->N;
  f.K = g->K;
  f.err = static_cast<uint32_t*>(ws);
  return cuda_status(launch_fp8_block(f, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_few_workspace_size(const moe_problem_t* p) {
  if (validate_problem(p) != MOE_OK || !few_fits(*p)) return 0;
  return few_layout(*p).total;
}

moe_status_t moe_forward_few(const moe_problem_t* p, const moe_weights_t* w, const void* x, const float* logits,
                             const float* bias, void* out, void* ws, size_t ws_bytes, moe_stream_t stream) {
  MOE_TRY(validate_problem(p));
  if (!few_fits(*p)) return MOE_ERR_UNSUPPORTED;
  MOE_TRY(validate_weights(p, w));
  const FewLayout L = few_layout(*p);
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  if (p->T == 0) return MOE_OK;
  if (!x || !logits || !out || !aligned(x, 16) || !aligned(out, 16) || !aligned(logits, 4) ||
      (bias && !aligned(bias, 4)) || !aligned(w->w13_scale, 4) || !aligned(w->w2_scale, 4) ||
      !aligned(w->w13_zero, 4) || !aligned(w->w2_zero, 4))
    return MOE_ERR_INVALID_ARG;
  uint8_t* base = static_cast<uint8_t*>(ws);
  GateArgs g;
  g.logits = logits;
  g.bias = p->scoring == MOE_SCORE_SIGMOID ? bias : nullptr;
  g.ids = nullptr;  // the kernels keep them to themselves
  g.w = nullptr;
  g.T = p->T;
  g.E = p->E;
  g.k = p->top_k;
  g.sigmoid = p->scoring == MOE_SCORE_SIGMOID;
  g.renormalize = p->renormalize;
  g.n_group = p->n_group;
  g.topk_group = p->topk_group;
  g.scale = p->routed_scaling_factor;
  FewArgs a;
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.w13 = w->w13;
  a.w2 = w->w2;
  a.w13_scale = w->w13_scale;
  a.w2_scale = w->w2_scale;
  a.w13_zero = static_cast<const uint8_t*>(w->w13_zero);
  a.w2_zero = static_cast<const uint8_t*>(w->w2_zero);
  a.a1 = w->a1_scale;
  a.a2 = w->a2_scale;
  a.act = reinterpret_cast<uint16_t*>(base + L.act);
  a.amax = reinterpret_cast<float*>(base + L.amax);
  a.err = reinterpret_cast<uint32_t*>(base);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.T = p->T;
  a.H = p->H;
  a.I = p->I;
  a.E = p->E;
  a.k = p->top_k;
  a.wkind = p->wdtype == MOE_W_FP8_E4M3 ? kW_FP8
            : p->wdtype == MOE_W_INT8_G128 ? kW_INT8
            : p->wdtype == MOE_W_BF16      ? kW_BF16
                                           : kW_INT4;
  a.paired = p->wdtype == MOE_W_INT4_G128_PAIRED;
  return cuda_status(launch_few(g, a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
