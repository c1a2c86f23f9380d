// Host side of the attention half's operators declared in include/moe.h: argument
// checks and launches.
#include <cmath>

#include "../../include/moe.h"
#include "checks.h"
#include "common.cuh"
#include "kernels.h"

using namespace moe;

namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool page_size_ok(int n) { return n >= 16 && n <= 1024 && (n & (n - 1)) == 0; }
int shift_of(int n) {
  int s = 0;
  while ((1 << s) < n) ++s;
  return s;
}

// The cache's pointers and strides; of one page, token or head the stride is not used.
moe_status_t check_cache(const moe_kv_t* c, int cache_dtype, int Hkv, int D, int page_size, int num_pages, KvCache* out) {
  if (c == nullptr || cache_dtype < MOE_CACHE_SAME || cache_dtype > MOE_CACHE_E4M3) return MOE_ERR_INVALID_ARG;
  if (!page_size_ok(page_size) || num_pages < 1) return MOE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(num_pages) * page_size > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  const bool e4m3 = cache_dtype == MOE_CACHE_E4M3;
  const int64_t unit = e4m3 ? 16 : 8;
  if (D % unit != 0 || !aligned(c->k, 16) || !aligned(c->v, 16) || c->k == nullptr || c->v == nullptr)
    return MOE_ERR_INVALID_ARG;
  const int64_t strides[2][3] = {{c->k_page_stride, c->k_token_stride, c->k_head_stride},
                                 {c->v_page_stride, c->v_token_stride, c->v_head_stride}};
  const int64_t counts[3] = {num_pages, page_size, Hkv};
  for (const auto& s : strides)
    for (int i = 0; i < 3; ++i)
      if (counts[i] > 1 && (s[i] < D || s[i] % unit != 0 || s[i] > (1ll << 37))) return MOE_ERR_INVALID_ARG;
  if (e4m3 != (c->k_scale != nullptr) || e4m3 != (c->v_scale != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(c->k_scale, 16) || !aligned(c->v_scale, 16)) return MOE_ERR_INVALID_ARG;
  auto used = [&](int i, int64_t s) { return counts[i] > 1 ? s : static_cast<int64_t>(unit); };
  *out = {static_cast<uint8_t*>(c->k),  static_cast<uint8_t*>(c->v),  c->k_scale,
          c->v_scale,                   used(0, c->k_page_stride),    used(1, c->k_token_stride),
          used(2, c->k_head_stride),    used(0, c->v_page_stride),    used(1, c->v_token_stride),
          used(2, c->v_head_stride)};
  return MOE_OK;
}

bool half_dtype(int d) { return d == MOE_T_BF16 || d == MOE_T_F16; }

// 16-byte aligned rows of 16-bit values
bool wide_rows(const void* p, int64_t stride, int64_t cols) { return rows_ok(p, stride, cols, 16) && stride % 8 == 0; }

moe_status_t validate_attention(const moe_attention_t* p) {
  if (p == nullptr || p->T < 0 || p->B < 0 || p->Hq < 1 || p->Hkv < 1 || p->Hq % p->Hkv != 0) return MOE_ERR_INVALID_ARG;
  if (p->D < 8 || p->D % 8 != 0 || p->max_q < 1 || !half_dtype(p->dtype)) return MOE_ERR_INVALID_ARG;
  if (p->cache_dtype < MOE_CACHE_SAME || p->cache_dtype > MOE_CACHE_E4M3) return MOE_ERR_INVALID_ARG;
  if (!(p->scale > 0.f) || !std::isfinite(p->scale * kLog2e)) return MOE_ERR_INVALID_ARG;
  if (p->D > 128 || p->Hq > 4096 || p->B > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(p->T) * p->Hq > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool few_rows(const moe_attention_t& p) { return static_cast<int64_t>(p.max_q) * (p.Hq / p.Hkv) <= kAttnFewRows; }

size_t attention_workspace(const moe_attention_t& p) {
  return kHeaderBytes + kAttnTicketBytes +
         2 * kAttnMaxCtas * attn_piece_bytes(few_rows(p) ? kAttnFewRows : kAttnRows, p.D);
}

moe_status_t check_attention(const moe_attention_t* p, const void* q, int64_t q_stride, const int32_t* cu_q,
                             const void* out, int64_t out_stride, const float* lse, const void* ws, size_t ws_bytes) {
  MOE_TRY(check_header(ws, ws_bytes));
  if (ws_bytes < attention_workspace(*p)) return MOE_ERR_WORKSPACE;
  if (p->B == 0 || p->T == 0) return MOE_OK;
  const int64_t nq = static_cast<int64_t>(p->Hq) * p->D;
  if (!wide_rows(q, q_stride, nq) || !wide_rows(out, out_stride, nq)) return MOE_ERR_INVALID_ARG;
  if (cu_q == nullptr || !aligned(cu_q, 4) || !aligned(lse, 4)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status_t attend(const moe_attention_t* p, AttnArgs& a, const void* q, int64_t q_stride, const int32_t* cu_q,
                    void* out, int64_t out_stride, float* lse, void* ws, moe_stream_t stream) {
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return MOE_ERR_CUDA;
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.q = static_cast<const uint16_t*>(q);
  a.cu_q = cu_q;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.err = reinterpret_cast<uint32_t*>(base);
  a.tickets = reinterpret_cast<uint32_t*>(base + kHeaderBytes);
  a.partial = reinterpret_cast<float*>(base + kHeaderBytes + kAttnTicketBytes);
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.T = p->T;
  a.B = p->B;
  a.Hq = p->Hq;
  a.Hkv = p->Hkv;
  a.D = p->D;
  a.G = p->Hq / p->Hkv;
  a.f16 = p->dtype == MOE_T_F16;
  a.scale_log2 = p->scale * kLog2e;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(few_rows(*p) ? launch_attention_few(a, p->max_q * a.G, di.sms, s) : launch_attention(a, di.sms, s));
}

}  // namespace

extern "C" {

moe_status_t moe_qk_norm_rope(const moe_rope_t* r, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                              const void* v, int64_t v_stride, const int32_t* positions, const uint64_t* turns,
                              const void* q_weight, const void* k_weight, void* q_out, int64_t q_out_stride,
                              void* k_out, int64_t k_out_stride, const moe_kv_t* cache, const int32_t* slots, void* ws,
                              size_t ws_bytes, moe_stream_t stream) {
  if (r == nullptr || r->T < 0 || r->Hq < 1 || r->Hkv < 1 || r->D < 8 || r->D % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (r->rot < 0 || r->rot > r->D || r->rot % 2 != 0) return MOE_ERR_INVALID_ARG;
  if (r->interleaved != 0 && r->interleaved != 1) return MOE_ERR_INVALID_ARG;
  if (!half_dtype(r->dtype) || (r->weight_dtype != r->dtype && r->weight_dtype != MOE_T_F32)) return MOE_ERR_INVALID_ARG;
  if (!(r->eps >= 0.f) || !std::isfinite(r->eps) || !std::isfinite(r->magnitude)) return MOE_ERR_INVALID_ARG;
  if (r->D > 256 || r->Hq > 4096 || r->Hkv > 4096 || r->T > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  MOE_TRY(check_header(ws, ws_bytes));
  RopeArgs a = {};
  if (cache != nullptr) {
    MOE_TRY(check_cache(cache, r->cache_dtype, r->Hkv, r->D, r->page_size, r->num_pages, &a.cache));
  } else if (r->page_size != 0 || k_out == nullptr) {
    return MOE_ERR_INVALID_ARG;
  }
  if (r->T == 0) return MOE_OK;
  const int64_t nq = static_cast<int64_t>(r->Hq) * r->D, nk = static_cast<int64_t>(r->Hkv) * r->D;
  if (!wide_rows(q, q_stride, nq) || !wide_rows(k, k_stride, nk) || !wide_rows(q_out, q_out_stride, nq))
    return MOE_ERR_INVALID_ARG;
  if (k_out != nullptr && !wide_rows(k_out, k_out_stride, nk)) return MOE_ERR_INVALID_ARG;
  if ((q_out == q && q_out_stride != q_stride) || (k_out == k && k_out_stride != k_stride)) return MOE_ERR_INVALID_ARG;
  if (cache != nullptr && (!wide_rows(v, v_stride, nk) || slots == nullptr || !aligned(slots, 4)))
    return MOE_ERR_INVALID_ARG;
  if (r->rot > 0 && (positions == nullptr || !aligned(positions, 4) || turns == nullptr || !aligned(turns, 8)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16)) return MOE_ERR_INVALID_ARG;
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return MOE_ERR_CUDA;
  a.q = q;
  a.k = k;
  a.v = v;
  a.positions = positions;
  a.turns = turns;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.q_out = q_out;
  a.k_out = k_out;
  a.slots = slots;
  a.err = static_cast<uint32_t*>(ws);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.capacity = static_cast<int64_t>(r->num_pages) * r->page_size;
  a.T = r->T;
  a.Hq = r->Hq;
  a.Hkv = r->Hkv;
  a.D = r->D;
  a.rot = r->rot;
  a.interleaved = r->interleaved;
  a.weight_f32 = r->weight_dtype == MOE_T_F32;
  a.e4m3 = cache != nullptr && r->cache_dtype == MOE_CACHE_E4M3;
  a.page_shift = cache != nullptr ? shift_of(r->page_size) : 0;
  a.sms = di.sms;
  a.eps = r->eps;
  a.magnitude = r->magnitude;
  return cuda_status(launch_rope(a, r->dtype, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_linear(const moe_linear_t* l, const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                        const void* bias, const void* residual, int64_t residual_stride, void* out, int64_t out_stride,
                        void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (l == nullptr || l->M < 0 || l->N < 0 || l->K < 8 || l->K % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (!half_dtype(l->dtype) || !is_dtype(l->out_dtype)) return MOE_ERR_INVALID_ARG;
  if (l->activation < MOE_ACT_NONE || l->activation > MOE_ACT_RELU) return MOE_ERR_INVALID_ARG;
  if (l->M > (1 << 22) || l->N > (1 << 22) || l->K > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  MOE_TRY(check_header(ws, ws_bytes));
  if (l->M == 0 || l->N == 0) return MOE_OK;
  if (!wide_rows(x, x_stride, l->K) || !wide_rows(w, w_stride, l->K) || !aligned(bias, 2)) return MOE_ERR_INVALID_ARG;
  const size_t b = size_of(l->out_dtype);
  if (!rows_ok(out, out_stride, l->N, b)) return MOE_ERR_INVALID_ARG;
  if (residual != nullptr && !rows_ok(residual, residual_stride, l->N, b)) return MOE_ERR_INVALID_ARG;
  if (residual == out && residual_stride != out_stride) return MOE_ERR_INVALID_ARG;
  LinearArgs a = {};
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.residual = residual;
  a.out = out;
  a.x_stride = x_stride;
  a.w_stride = w_stride;
  a.residual_stride = residual_stride;
  a.out_stride = out_stride;
  a.M = l->M;
  a.N = l->N;
  a.K = l->K;
  a.f16 = l->dtype == MOE_T_F16;
  a.out_dtype = l->out_dtype;
  a.act = l->activation;
  a.err = static_cast<uint32_t*>(ws);
  return cuda_status(launch_linear(a, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_paged_attention(const moe_attention_t* p, const void* q, int64_t q_stride, const moe_kv_t* cache,
                                 const int32_t* page_table, int64_t table_stride, const int32_t* cu_q,
                                 const int32_t* kv_len, void* out, int64_t out_stride, float* lse, void* ws,
                                 size_t ws_bytes, moe_stream_t stream) {
  MOE_TRY(validate_attention(p));
  AttnArgs a = {};
  MOE_TRY(check_cache(cache, p->cache_dtype, p->Hkv, p->D, p->page_size, p->num_pages, &a.kv));
  if (p->max_pages < 1) return MOE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(p->max_pages) * p->page_size > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  MOE_TRY(check_attention(p, q, q_stride, cu_q, out, out_stride, lse, ws, ws_bytes));
  if (p->B == 0 || p->T == 0) return MOE_OK;
  if (page_table == nullptr || !aligned(page_table, 4) || (p->B > 1 && table_stride < p->max_pages) ||
      kv_len == nullptr || !aligned(kv_len, 4))
    return MOE_ERR_INVALID_ARG;
  a.page_table = page_table;
  a.table_stride = table_stride;
  a.kv_len = kv_len;
  a.page_shift = shift_of(p->page_size);
  a.num_pages = p->num_pages;
  a.max_len = p->max_pages * p->page_size;
  a.e4m3 = p->cache_dtype == MOE_CACHE_E4M3;
  return attend(p, a, q, q_stride, cu_q, out, out_stride, lse, ws, stream);
}

moe_status_t moe_prompt_attention(const moe_attention_t* p, const void* q, int64_t q_stride, const void* k,
                                  int64_t k_stride, const void* v, int64_t v_stride, const int32_t* cu_q, void* out,
                                  int64_t out_stride, float* lse, void* ws, size_t ws_bytes, moe_stream_t stream) {
  MOE_TRY(validate_attention(p));
  if (p->cache_dtype != MOE_CACHE_SAME || p->page_size != 0 || p->num_pages != 0 || p->max_pages != 0)
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_attention(p, q, q_stride, cu_q, out, out_stride, lse, ws, ws_bytes));
  if (p->B == 0 || p->T == 0) return MOE_OK;
  const int64_t nk = static_cast<int64_t>(p->Hkv) * p->D;
  if (!wide_rows(k, k_stride, nk) || !wide_rows(v, v_stride, nk)) return MOE_ERR_INVALID_ARG;
  AttnArgs a = {};
  a.kv.k = static_cast<uint8_t*>(const_cast<void*>(k));
  a.kv.v = static_cast<uint8_t*>(const_cast<void*>(v));
  a.kv.k_token = k_stride;
  a.kv.v_token = v_stride;
  a.kv.k_head = a.kv.v_head = p->D;
  a.num_pages = 1;
  return attend(p, a, q, q_stride, cu_q, out, out_stride, lse, ws, stream);
}

size_t moe_attention_workspace_size(const moe_attention_t* p) {
  return validate_attention(p) == MOE_OK ? attention_workspace(*p) : 0;
}

}  // extern "C"
