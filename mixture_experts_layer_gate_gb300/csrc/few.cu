// The MoE layer for a few tokens (moe_forward_few): one warp per output value,
// after the gate kernel.
//   act[t, j, i] = silu(w13[e, i] . x[t]) (w13[e, I + i] . x[t]), e = ids[t, j]
//   out[t, h]    = sum_j w[t, j] (w2[e, h] . act[t, j])
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

__device__ __forceinline__ float e4m3_f32(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}
__device__ __forceinline__ float quantised(float v, float scale) {
  return e4m3_f32(static_cast<uint8_t>(f32x2_to_e4m3x2(__fdiv_rn(v, scale), 0.f))) * scale;
}

// value of weight k of a row (scale of fp8 rows left to the caller)
__device__ float weight_at(const FewArgs& a, const void* w, const void* scale, const uint8_t* zero, int64_t row,
                           int K, int k) {
  if (a.wkind == kW_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[row * K + k]);
  const uint8_t* b = static_cast<const uint8_t*>(w);
  if (a.wkind == kW_FP8) return e4m3_f32(b[row * K + k]);
  const int64_t g = row * (K / 128) + k / 128;
  int c;
  if (a.wkind == kW_INT8) {
    c = b[row * K + k];
    if (zero == nullptr) c = static_cast<int8_t>(c);
  } else {
    const uint32_t word = reinterpret_cast<const uint32_t*>(b)[(row * K + k) / 8];
    const int j = k % 8;
    c = (word >> (4 * (a.paired ? (j >> 1) + 4 * (j & 1) : j))) & 15;
    if (zero == nullptr) c = (c ^ 8) - 8;
  }
  if (zero != nullptr) c -= zero[g];
  return static_cast<float>(c) * __half2float(static_cast<const __half*>(scale)[g]);
}

__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(256) few_up_kernel(FewArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (at >= static_cast<int64_t>(a.T) * a.k * a.I) return;
  const int slot = static_cast<int>(at / a.I), i = static_cast<int>(at % a.I), t = slot / a.k;
  const int64_t e = a.ids[slot], r0 = e * 2 * a.I + i, r1 = r0 + a.I;
  float a1 = 1.f;
  if (a.wkind == kW_FP8) {
    if (a.a1 != nullptr) {
      a1 = a.a1[0];
    } else {
      float m = 0.f;
      for (int j = lane; j < a.T * a.H; j += 32) m = fmaxf(m, fabsf(__bfloat162float(a.x[j])));
      m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
      a1 = m > 0.f ? __fdiv_rn(m, 448.0f) : 1.0f;
    }
  }
  float g = 0.f, u = 0.f;
  for (int k = lane; k < a.H; k += 32) {
    float xv = __bfloat162float(a.x[static_cast<int64_t>(t) * a.H + k]);
    if (a.wkind == kW_FP8) xv = quantised(xv, a1);
    g = fmaf(weight_at(a, a.w13, a.w13_scale, a.w13_zero, r0, a.H, k), xv, g);
    u = fmaf(weight_at(a, a.w13, a.w13_scale, a.w13_zero, r1, a.H, k), xv, u);
  }
  g = warp_sum(g);
  u = warp_sum(u);
  if (lane == 0) {
    if (a.wkind == kW_FP8) {
      g *= static_cast<const float*>(a.w13_scale)[e];
      u *= static_cast<const float*>(a.w13_scale)[e];
    }
    const float v = __fdiv_rn(g, 1.0f + expf(-g)) * u;
    a.act[at] = v;
    if (a.wkind == kW_FP8 && a.a2 == nullptr) atomicMax(a.amax, __float_as_uint(fabsf(v)));
  }
}

__global__ void __launch_bounds__(256) few_down_kernel(FewArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (at >= static_cast<int64_t>(a.T) * a.H) return;
  const int t = static_cast<int>(at / a.H), h = static_cast<int>(at % a.H);
  float a2 = 1.f;
  if (a.wkind == kW_FP8) {
    const float m = a.a2 != nullptr ? 0.f : __uint_as_float(*a.amax);
    a2 = a.a2 != nullptr ? a.a2[0] : (m > 0.f ? __fdiv_rn(m, 448.0f) : 1.0f);
  }
  float total = 0.f;
  for (int j = 0; j < a.k; ++j) {
    const int slot = t * a.k + j;
    const int64_t e = a.ids[slot], row = e * a.H + h;
    float y = 0.f;
    for (int k = lane; k < a.I; k += 32) {
      float v = a.act[static_cast<int64_t>(slot) * a.I + k];
      if (a.wkind == kW_FP8) v = quantised(v, a2);
      y = fmaf(weight_at(a, a.w2, a.w2_scale, a.w2_zero, row, a.I, k), v, y);
    }
    if (a.wkind == kW_FP8) y *= static_cast<const float*>(a.w2_scale)[e];
    total = fmaf(a.topk_w[slot], y, total);
  }
  total = warp_sum(total);
  if (lane == 0) a.out[at] = __float2bfloat16_rn(total);
}

}  // namespace

cudaError_t launch_few(const GateArgs& g, const FewArgs& a, cudaStream_t s) {
  cudaError_t err = launch_gate(g, s);
  if (err != cudaSuccess) return err;
  err = cudaMemsetAsync(a.amax, 0, sizeof(uint32_t), s);
  if (err != cudaSuccess) return err;
  const int64_t up = static_cast<int64_t>(a.T) * a.k * a.I, down = static_cast<int64_t>(a.T) * a.H;
  err = launch_pdl(few_up_kernel, dim3(static_cast<unsigned>((up + 7) / 8)), dim3(256), 0, s, a);
  if (err != cudaSuccess) return err;
  return launch_pdl(few_down_kernel, dim3(static_cast<unsigned>((down + 7) / 8)), dim3(256), 0, s, a);
}

}  // namespace moe
