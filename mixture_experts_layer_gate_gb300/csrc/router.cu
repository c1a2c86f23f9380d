// Router scores (moe_router_logits): logits[t, e] = sum_h x[t, h] w[e, h], in
// float.  A batch goes through the dense kernel with 16-bit operands (bound by
// the reads of x and the tiles' repeated reads through L2: T = 4096, H = 7168,
// 256 experts 20 us, of which x is 8.6 us of DRAM time).  Up to 4 tokens, where
// only latency counts, a CTA takes an expert: all of its row is in flight at
// once, and the threads' sums are joined in a fixed order (T = 1, H = 7168, 256
// experts: 1.8 us in a graph; 2 and 4 tokens see launch_router).
#include "dense.cuh"

namespace moe {
namespace {

constexpr int kFewTokens = 4;
constexpr int kFewThreads = 128;

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

template <typename T2, int T>
__global__ void __launch_bounds__(kFewThreads) router_few_kernel(RouterArgs a) {
  __shared__ float part[kFewThreads / 32][T];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t e = blockIdx.x;
  const uint4* w = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.w) + e * a.w_stride);
  const int nvec = a.H / 8;
  pdl_wait();
  pdl_trigger();
  float sum[T] = {};
  for (int i0 = tid; i0 < nvec; i0 += 8 * kFewThreads) {
    uint4 q[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) q[u] = i0 + u * kFewThreads < nvec ? w[i0 + u * kFewThreads] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + t * a.x_stride);
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = i0 + u * kFewThreads < nvec ? x[i0 + u * kFewThreads] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint32_t p[4] = {q[u].x, q[u].y, q[u].z, q[u].w}, r[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = pair_f32<T2>(p[j]), g = pair_f32<T2>(r[j]);
          sum[t] = fmaf(f.x, g.x, sum[t]);
          sum[t] = fmaf(f.y, g.y, sum[t]);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum[t] += __shfl_xor_sync(0xffffffffu, sum[t], o);
    if (lane == 0) part[warp][t] = sum[t];
  }
  __syncthreads();
  if (tid < T) {
    float s = part[0][tid];
#pragma unroll
    for (int i = 1; i < kFewThreads / 32; ++i) s += part[i][tid];
    a.logits[static_cast<int64_t>(tid) * a.E + e] = s;
  }
}

template <typename T2>
cudaError_t launch_few(const RouterArgs& a, cudaStream_t s) {
  switch (a.T) {
    case 1: return launch_pdl(router_few_kernel<T2, 1>, dim3(a.E), dim3(kFewThreads), 0, s, a);
    case 2: return launch_pdl(router_few_kernel<T2, 2>, dim3(a.E), dim3(kFewThreads), 0, s, a);
    case 3: return launch_pdl(router_few_kernel<T2, 3>, dim3(a.E), dim3(kFewThreads), 0, s, a);
    default: return launch_pdl(router_few_kernel<T2, kFewTokens>, dim3(a.E), dim3(kFewThreads), 0, s, a);
  }
}

}  // namespace

cudaError_t launch_router(const RouterArgs& a, cudaStream_t s) {
  // the few-token kernel reads the tokens once per expert: T = 1, 2, 4 of 256 experts
  // 1.8, 2.5, 4.1 us against 5.2 us, but 4 of 1024 experts 7.8 against 6.8
  if (a.T <= kFewTokens && a.T * a.E <= 2048) return a.dtype == 0 ? launch_few<__nv_bfloat162>(a, s) : launch_few<__half2>(a, s);
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  dense::Params p = {};
  p.out = a.logits;
  p.err = a.err;
  p.out_stride = a.E;
  p.M = a.T;
  p.N = a.E;
  p.KB = (a.H + 63) / 64;
  p.group = 16;
  p.out_dtype = 2;
  p.fmt = a.dtype == 0 ? 1 : 0;
  p.vec = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.E % 4 == 0;
  const dense::Choice c = dense::choose(a.T, a.E, p.KB, false, false, di.sms);
  p.P = c.P;
  return dense::plan_and_launch<dense::kHalf>(p, c.bn, c.pair, false, a.x, a.x_stride, a.w, a.w_stride, a.E, a.H, di.sms,
                                              s);
}

}  // namespace moe
