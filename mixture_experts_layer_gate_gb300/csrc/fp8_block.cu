// Product of e4m3 operands with a scale per block of 128 (moe_gemm_fp8_block,
// moe_gemm_fp8_block_swiglu): out[m, n] = sum_b a_scale[m, b] w_scale[n / 128, b]
// sum_{k in b} a[m, k] w[n, k].
//
// 16 rows x 128 columns per CTA (gate and up columns together for SwiGLU, so a
// row's quantisation block is whole), operands of 32 k at a time in shared
// memory as floats.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kTileM = 16, kTileN = 128, kTileK = 32;

__device__ __forceinline__ float e4m3_f32(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(__half(h));
}

// SETS = 2: columns [n0, n0 + 128) of the gate and of the up half.
template <int SETS>
__global__ void __launch_bounds__(256) fp8_block_kernel(Fp8GemmArgs g) {
  __shared__ float sa[kTileM][kTileK + 1];
  __shared__ float sw[SETS][kTileN][kTileK + 1];
  __shared__ float amax[2][8];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, col = tid % kTileN, half = tid / kTileN;  // rows half * 8 ..
  const int n0 = blockIdx.x * kTileN, m0 = blockIdx.y * kTileM;
  const int KB = (g.K + 127) / 128;
  float acc[SETS][8] = {};
  for (int b = 0; b < KB; ++b) {
    float part[SETS][8] = {};
    for (int k0 = b * 128; k0 < min(g.K, b * 128 + 128); k0 += kTileK) {
      __syncthreads();
      for (int i = tid; i < kTileM * kTileK; i += 256) {
        const int m = m0 + i / kTileK, k = k0 + i % kTileK;
        sa[i / kTileK][i % kTileK] = (m < g.M && k < g.K) ? e4m3_f32(g.a[m * g.a_stride + k]) : 0.f;
      }
      for (int s = 0; s < SETS; ++s)
        for (int i = tid; i < kTileN * kTileK; i += 256) {
          const int n = n0 + i / kTileK, k = k0 + i % kTileK;
          sw[s][i / kTileK][i % kTileK] =
              (n < g.N && k < g.K) ? e4m3_f32(g.w[(static_cast<int64_t>(s) * g.N + n) * g.w_stride + k]) : 0.f;
        }
      __syncthreads();
      for (int k = 0; k < kTileK; ++k)
#pragma unroll
        for (int s = 0; s < SETS; ++s) {
          const float wv = sw[s][col][k];
#pragma unroll
          for (int i = 0; i < 8; ++i) part[s][i] = fmaf(sa[half * 8 + i][k], wv, part[s][i]);
        }
    }
#pragma unroll
    for (int s = 0; s < SETS; ++s) {
      const float ws = n0 + col < g.N ? g.w_scale[static_cast<int64_t>((s * g.N + n0 + col) / 128) * KB + b] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int m = m0 + half * 8 + i;
        const float as = m < g.M ? g.a_scale[m * g.a_scale_stride + b] : 0.f;
        acc[s][i] = fmaf(part[s][i], as * ws, acc[s][i]);
      }
    }
  }
  if (SETS == 1) {
    if (n0 + col >= g.N) return;
    for (int i = 0; i < 8; ++i) {
      const int m = m0 + half * 8 + i;
      if (m >= g.M) break;
      const int64_t at = m * g.out_stride + n0 + col;
      float v = acc[0][i];
      if (g.out_dtype == 0) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(g.out) + at;
        *o = __float2bfloat16_rn(g.accumulate ? v + __bfloat162float(*o) : v);
      } else if (g.out_dtype == 1) {
        __half* o = static_cast<__half*>(g.out) + at;
        *o = __float2half_rn(g.accumulate ? v + __half2float(*o) : v);
      } else {
        float* o = static_cast<float*>(g.out) + at;
        *o = g.accumulate ? v + *o : v;
      }
    }
    return;
  }
  for (int i = 0; i < 8; ++i) {
    const float h = acc[0][i];
    const float v = __fdiv_rn(h, 1.0f + expf(-h)) * acc[SETS - 1][i];
    float m = fabsf(v);
    for (int o = 16; o > 0; o >>= 1) {
      const float p = __shfl_xor_sync(0xffffffffu, m, o);
      m = (m > p || m != m) ? m : p;
    }
    __syncthreads();
    if (tid % 32 == 0) amax[half][(tid / 32) % 4] = m;
    __syncthreads();
    m = amax[half][0];
    for (int j = 1; j < 4; ++j) {
      const float p = amax[half][j];
      m = (m > p || m != m) ? m : p;
    }
    const float scale = m == 0.f ? 1.0f : __fdiv_rn(m, 448.0f);
    const int row = m0 + half * 8 + i;
    if (row < g.M) {
      if (col == 0) g.scales[static_cast<int64_t>(row) * (g.N / 128) + blockIdx.x] = scale;
      g.codes[static_cast<int64_t>(row) * g.N + n0 + col] =
          static_cast<uint8_t>(f32x2_to_e4m3x2(__fdiv_rn(v, scale), 0.f));
    }
  }
}

}  // namespace

cudaError_t launch_fp8_block(const Fp8GemmArgs& g, cudaStream_t s) {
  const dim3 grid((g.N + kTileN - 1) / kTileN, (g.M + kTileM - 1) / kTileM);
  if (g.codes != nullptr) return launch_pdl(fp8_block_kernel<2>, grid, dim3(256), 0, s, g);
  return launch_pdl(fp8_block_kernel<1>, grid, dim3(256), 0, s, g);
}

}  // namespace moe
