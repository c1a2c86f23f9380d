// Router scores (moe_router_logits): logits[t, e] = sum_h x[t, h] w[e, h], in
// float.  One warp per token and expert, 16-byte loads along H, a shuffle sum.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

template <typename T2>
__device__ __forceinline__ float2 pair_f32(uint32_t v);
template <>
__device__ __forceinline__ float2 pair_f32<__nv_bfloat162>(uint32_t v) {
  return make_float2(bf16_lo(v), bf16_hi(v));
}
template <>
__device__ __forceinline__ float2 pair_f32<__half2>(uint32_t v) {
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}

template <typename T2>
__global__ void __launch_bounds__(256) router_dot_kernel(RouterArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (at >= static_cast<int64_t>(a.T) * a.E) return;
  const int64_t t = at / a.E, e = at % a.E;
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + t * a.x_stride);
  const uint4* w = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.w) + e * a.w_stride);
  float sum = 0.f;
  for (int i = lane; i < a.H / 8; i += 32) {
    const uint4 u = x[i], v = w[i];
    const uint32_t p[4] = {u.x, u.y, u.z, u.w}, q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = pair_f32<T2>(p[j]), g = pair_f32<T2>(q[j]);
      sum = fmaf(f.x, g.x, sum);
      sum = fmaf(f.y, g.y, sum);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) a.logits[at] = sum;
}

}  // namespace

cudaError_t launch_router(const RouterArgs& a, cudaStream_t s) {
  const int64_t n = static_cast<int64_t>(a.T) * a.E;
  const dim3 grid(static_cast<unsigned>((n + 7) / 8));
  if (a.dtype == 0) return launch_pdl(router_dot_kernel<__nv_bfloat162>, grid, dim3(256), 0, s, a);
  return launch_pdl(router_dot_kernel<__half2>, grid, dim3(256), 0, s, a);
}

}  // namespace moe
