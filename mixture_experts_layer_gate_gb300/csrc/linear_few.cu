// moe_linear for at most 8 rows of x (decode): bound by the rate at which the
// weights stream in, so no tile of 128 rows: a warp multiplies 16 weight rows with
// all rows of x (the 8 columns of mma.sync m16n8k16) over its part of K, straight
// from global memory to registers.  K is permuted inside 32 values so that the 16
// adjacent bytes a lane loads are its fragment: lane (g, c) holds k = 8 c .. 8 c + 7 of
// weight rows g and g + 8 and of row g of x, words 0 and 1 for one product, 2 and 3 for
// the next.  The warps' sums are joined through shared memory in a fixed order.  N =
// 6144, K = 4096 in a graph, the weights from memory: one row 9.2 us = 5.5 TB/s, eight
// 9.9; two CTAs an SM instead of three 11.1, six or eight steps ahead instead of four
// 9.9 and 14 (their registers).  Sixteen rows took 15 us, the tensor cores' tiles 12.4.
#include "common.cuh"
#include "kernels.h"
#include "stream.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kAhead = 4;  // steps of 32 k whose loads are in flight

__device__ __forceinline__ uint4 load_weights(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case 1: return v / (1.0f + expf(-v));
    case 2: return gelu(v);
    case 3: return v / (1.0f + expf(-v * fmaf(v * v, 0.044715f * 1.5957691216057308f, 1.5957691216057308f)));
    case 4: return v < 0.f ? 0.f : v;
    default: return v;
  }
}

__device__ __forceinline__ float value_at(const void* p, int64_t i, int dtype) {
  return dtype == 2   ? static_cast<const float*>(p)[i]
         : dtype == 1 ? __half2float(static_cast<const __half*>(p)[i])
                      : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

template <bool F16>
__global__ void __launch_bounds__(kThreads, 3) linear_few_kernel(const LinearArgs a) {
  __shared__ float red[kWarps][16][9];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int n0 = blockIdx.x * 16;
  const int steps = (a.K + 31) / 32;
  const uint16_t* w0 = static_cast<const uint16_t*>(a.w) + static_cast<int64_t>(min(n0 + g, a.N - 1)) * a.w_stride;
  const uint16_t* w1 = static_cast<const uint16_t*>(a.w) + static_cast<int64_t>(min(n0 + g + 8, a.N - 1)) * a.w_stride;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + static_cast<int64_t>(min(g, a.M - 1)) * a.x_stride;
  float acc[4] = {}, sum[4] = {};
  int run = 0;
  const uint4 none = make_uint4(0, 0, 0, 0);
  uint4 p[kAhead], q[kAhead];
  pdl_wait();
  pdl_trigger();
  auto fetch = [&](int s, uint4& u, uint4& v) {
    const int k = s * 32 + c * 8;
    const bool there = s < steps && k < a.K;
    u = there ? load_weights(reinterpret_cast<const uint4*>(w0 + k)) : none;
    v = there ? load_weights(reinterpret_cast<const uint4*>(w1 + k)) : none;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(warp + i * kWarps, p[i], q[i]);
  for (int s0 = warp; s0 < steps; s0 += kWarps * kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int s = s0 + i * kWarps, k = s * 32 + c * 8;
      const uint4 u = p[i], v = q[i];
      const bool there = s < steps && k < a.K;
      // (rows of x past M, and k past K, multiply nothing)
      const uint4 b = there && g < a.M ? *reinterpret_cast<const uint4*>(x + k) : none;
      mma16816<F16>(acc, u.x, v.x, u.y, v.y, b.x, b.y);
      mma16816<F16>(acc, u.z, v.z, u.w, v.w, b.z, b.w);
      fetch(s + kWarps * kAhead, p[i], q[i]);
    }
    if (++run == kLinearRun / (32 * kAhead)) {  // (a tensor core's sum is joined in float)
      run = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sum[e] += acc[e];
        acc[e] = 0.f;
      }
    }
  }
  red[warp][g][2 * c] = sum[0] + acc[0];
  red[warp][g][2 * c + 1] = sum[1] + acc[1];
  red[warp][g + 8][2 * c] = sum[2] + acc[2];
  red[warp][g + 8][2 * c + 1] = sum[3] + acc[3];
  __syncthreads();
  const int n = n0 + (tid & 15), m = tid >> 4;
  if (m < a.M && n < a.N) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += red[i][tid & 15][m];
    if (a.bias != nullptr) v += value_at(a.bias, n, F16 ? 1 : 0);
    v = activate(v, a.act);
    if (a.residual != nullptr) v += value_at(a.residual, m * a.residual_stride + n, a.out_dtype);
    const int64_t at = m * a.out_stride + n;
    if (a.out_dtype == 2) static_cast<float*>(a.out)[at] = v;
    else if (a.out_dtype == 1) static_cast<__half*>(a.out)[at] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
  }
}

}  // namespace

cudaError_t launch_linear_few(const LinearArgs& a, cudaStream_t s) {
  const dim3 grid((a.N + 15) / 16), block(kThreads);
  return a.f16 ? launch_pdl(linear_few_kernel<true>, grid, block, 0, s, a)
               : launch_pdl(linear_few_kernel<false>, grid, block, 0, s, a);
}

}  // namespace moe
