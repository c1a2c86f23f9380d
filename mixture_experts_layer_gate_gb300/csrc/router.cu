// Router scores (moe_router_logits): logits[t, e] = sum_h x[t, h] w[e, h], in
// float.  A batch goes through the dense kernel with 16-bit operands (bound by
// the reads of x and the tiles' repeated reads through L2: T = 4096, H = 7168,
// 256 experts 20 us, of which x is 8.6 us of DRAM time).  Up to 8 tokens, where
// only latency counts, a CTA takes an expert, 128 threads a token, and the threads'
// sums are joined in a fixed order (T = 1, H = 7168, 256 experts: 2.0 us in a graph, 2
// tokens 2.2, 4 tokens 2.9, 8 tokens 4.4).
#include "dense.cuh"

namespace moe {
namespace {

constexpr int kFewTokens = 8;
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

// Threads kFewThreads t .. take token t; the weight row that they share comes from
// L2 once a CTA.  At most TMAX tokens: bounded to a CTA of one or two tokens the
// kernel is faster than bounded to eight (H = 7168, 256 experts: one token 2.0 and
// 2.5 us, two 2.2 and 2.6, in a graph), to four it is not (2.9 both), with about 32
// registers a thread in each, so that the sixteen loads are not all in flight at once.
template <typename T2, int TMAX>
__global__ void __launch_bounds__(kFewThreads * TMAX) router_few_kernel(RouterArgs a) {
  __shared__ float part[TMAX][kFewThreads / 32];
  const int token = threadIdx.x / kFewThreads, tid = threadIdx.x % kFewThreads, warp = tid >> 5, lane = tid & 31;
  const int64_t e = blockIdx.x;
  const uint4* w = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.w) + e * a.w_stride);
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + token * a.x_stride);
  const int nvec = a.H / 8;
  pdl_wait();
  pdl_trigger();
  float sum = 0.f;
  for (int i0 = tid; i0 < nvec; i0 += 8 * kFewThreads) {
    uint4 q[8], v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) q[u] = i0 + u * kFewThreads < nvec ? w[i0 + u * kFewThreads] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = i0 + u * kFewThreads < nvec ? x[i0 + u * kFewThreads] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t p[4] = {q[u].x, q[u].y, q[u].z, q[u].w}, r[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = pair_f32<T2>(p[j]), g = pair_f32<T2>(r[j]);
        sum = fmaf(f.x, g.x, sum);
        sum = fmaf(f.y, g.y, sum);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) part[token][warp] = sum;
  __syncthreads();
  if (tid == 0) {
    float s = part[token][0];
#pragma unroll
    for (int i = 1; i < kFewThreads / 32; ++i) s += part[token][i];
    a.logits[static_cast<int64_t>(token) * a.E + e] = s;
  }
}

template <typename T2>
cudaError_t launch_few(const RouterArgs& a, cudaStream_t s) {
  const dim3 grid(a.E), block(kFewThreads * a.T);
  if (a.T == 1) return launch_pdl(router_few_kernel<T2, 1>, grid, block, 0, s, a);
  if (a.T == 2) return launch_pdl(router_few_kernel<T2, 2>, grid, block, 0, s, a);
  return launch_pdl(router_few_kernel<T2, kFewTokens>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_router(const RouterArgs& a, cudaStream_t s) {
  // the few-token kernel reads the tokens once per expert, so its time grows with T * E
  // (few / dense, in a graph): H = 7168, 256 experts, 8 tokens 4.3 / 5.2 us; H = 4096,
  // 512 experts, 4 tokens 4.1 / 4.8, 5 tokens 5.1 / 4.8; 1024 experts, 2 tokens 4.1 /
  // 5.4, 4 tokens 6.5 / 5.4; 8 experts, 8 tokens 2.6 / 4.2
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
