// The block-scaled 8-bit product for at most 8 rows of activations (decode):
// bound by the rate at which the weights stream in, so no tile of 128 rows, but
// the rings and mma.sync of the few-token layer (stream.cuh): a warp multiplies
// 16 weight rows with all activation rows (the 8 columns) by m16n8k16 on e4m3
// turned into f16 (exact), and joins each k-step's product, times its block's
// scales, to its sums in registers.
//
// SwiGLU: a CTA takes 16 gate rows and the 16 up rows that go with them, its
// warps each a part of K.  A quantisation block of 128 columns is 8 CTAs' work:
// each leaves its values (float) in scratch and counts itself, and the last of
// the eight takes the block's maxima and writes scales and codes (the same
// whichever is last).  A cluster of eight that exchanged the maxima through
// distributed shared memory took 13.6 us for one row, K = 7168, N = 2048 (such
// clusters start late and did not all fit with 16 warps a CTA).
// Else a CTA goes through blocks of 16 rows.
//
// In a graph, the weights in L2 / from memory (as many copies in turn as L2 does not
// hold): SwiGLU, K = 7168, N = 2048 (29 MB) one row 9.5 / 10.7 us, 2.7 TB/s, eight rows
// 10.2 / 10.8, the general kernel 13 (in L2); K = 2048, N = 7168 (14.7 MB) one row 4.1 /
// 4.5 us, 3.3 TB/s, eight rows 5.2 / 5.8, the general kernel 7 (16 rows, in L2): the
// stream, not the products, sets the time, and of it the start of the loads and the
// join at the end are half.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "stream.cuh"

namespace moe {
namespace {

// Warps of a CTA: one CTA an SM with SwiGLU, whose units are few, else two or three.
template <bool SWIGLU>
constexpr int kFewWarps = SWIGLU ? 16 : 8;
constexpr int kStage = 2048 + 32;  // 4 loads of 16 bytes a lane, and two weight scales
constexpr int kMaxFewDepth = 8;
template <bool SWIGLU>
constexpr int kFewSmem = SWIGLU ? 200 * 1024 : 110 * 1024;
constexpr int kThirdSmem = 73 * 1024;  // of three CTAs an SM
template <bool SWIGLU>
constexpr int kRed = kFewWarps<SWIGLU> * (SWIGLU ? 32 : 16) * 8 * 4;  // the warps' sums

__host__ __device__ constexpr int code_stride(int K) { return (K + 127) / 128 * 128 + 64; }

__device__ __forceinline__ void cp_async16_if(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16u : 0u) : "memory");
}
__device__ __forceinline__ float max_nan(float a, float b) { return (a > b || a != a) ? a : b; }

// SWIGLU: a step is 64 k of 16 gate and 16 up rows; else 128 k of 16 rows.
template <bool SWIGLU>
__global__ void __launch_bounds__(32 * kFewWarps<SWIGLU>, SWIGLU ? 1 : 2) fp8_few_kernel(Fp8GemmArgs p, int depth) {
  extern __shared__ __align__(128) uint8_t fp8_few_smem[];
  __shared__ bool last;
  constexpr int kWarps = kFewWarps<SWIGLU>, kThreads = 32 * kWarps;
  constexpr int STEP = SWIGLU ? 64 : 128, SETS = SWIGLU ? 2 : 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int KB = (p.K + 127) / 128, stride = code_stride(p.K);
  float* red = reinterpret_cast<float*>(fp8_few_smem);                   // [warp][set, row][8]
  float* as = red + kRed<SWIGLU> / 4;                                            // [block][8] activation scales
  uint8_t* codes = reinterpret_cast<uint8_t*>(as + KB * 8);              // [row][stride]
  const uint32_t rings = smem_u32(codes) + static_cast<uint32_t>((p.M * stride + 127) / 128 * 128);
  const uint32_t ring = rings + static_cast<uint32_t>(warp * depth * kStage);
  const uint32_t iend = ring + static_cast<uint32_t>(depth * kStage);
  const int units = SWIGLU ? p.N / 16 : (p.N + 15) / 16;
  const int nsteps = (p.K + STEP - 1) / STEP;
  const int s0 = nsteps * warp / kWarps, s1 = nsteps * (warp + 1) / kWarps;
  pdl_wait();
  pdl_trigger();

  int iu = blockIdx.x, is = s0;
  uint32_t idst = ring;
  auto issue = [&] {
    if (iu < units && s0 < s1) {
      const int64_t n0 = static_cast<int64_t>(iu) * 16;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // SWIGLU: gate rows g and g + 8, up rows g and g + 8; else rows g and g +
        // 8 of the step's first 64 k and of its second
        const int64_t n = n0 + g + 8 * (q & 1);
        const int64_t row = n + (SWIGLU && q >= 2 ? p.N : 0);
        const int k = is * STEP + t4 * 16 + (SWIGLU ? 0 : 64 * (q >> 1));
        const bool there = k < p.K && n < p.N;
        cp_async16_if(idst + static_cast<uint32_t>(q * 512 + lane * 16), there ? p.w + row * p.w_stride + k : p.w, there);
      }
      if (lane < SETS)
        cp_async4(idst + 2048 + lane * 4, p.w_scale + ((n0 + static_cast<int64_t>(lane) * p.N) / 128) * KB + is * STEP / 128);
      if (++is == s1) {
        is = s0;
        iu += gridDim.x;
      }
    }
    cp_async_commit();
    idst += kStage;
    if (idst >= iend) idst = ring;
  };
  // the activations, as the oldest group of copies (N = 2048, K = 7168, one row 5.1 us,
  // eight 6.9; with loads through registers after the first weights 6.3 and 8.9)
  for (int i = tid; i < p.M * (stride / 16); i += kThreads) {
    const int m = i / (stride / 16), k = (i - m * (stride / 16)) * 16;
    const bool there = k < p.K;
    cp_async16_if(smem_u32(codes) + static_cast<uint32_t>(m * stride + k), there ? p.a + m * p.a_stride + k : p.a, there);
  }
  for (int i = tid; i < KB * 8; i += kThreads)
    cp_async4(smem_u32(as) + static_cast<uint32_t>(i * 4),
              p.a_scale + static_cast<int64_t>(min(i & 7, p.M - 1)) * p.a_scale_stride + (i >> 3));
  cp_async_commit();
  for (int i = 0; i < depth - 1; ++i) issue();
  cp_async_wait(depth - 1);
  __syncthreads();

  uint32_t src = ring;
  // (columns past the last row repeat it; nobody reads their sums)
  const uint32_t mine = smem_u32(codes) + static_cast<uint32_t>(min(g, p.M - 1) * stride + t4 * 16);
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    float acc[SETS][4] = {};
    for (int s = s0; s < s1; ++s) {
      __syncwarp();
      issue();
      cp_async_wait(depth - 1);
      __syncwarp();
      float part[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {  // SWIGLU: gate and up of the same k; else two runs of k
        const uint4 wa = lds128(src + static_cast<uint32_t>(2 * u * 512 + lane * 16));
        const uint4 wb = lds128(src + static_cast<uint32_t>((2 * u + 1) * 512 + lane * 16));
        const uint4 b = lds128(mine + static_cast<uint32_t>(s * STEP + (SWIGLU ? 0 : 64 * u)));
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t a0 = e4m3x2_f16x2(word(wa, m) & 0xFFFFu), a2 = e4m3x2_f16x2(word(wa, m) >> 16);
          const uint32_t a1 = e4m3x2_f16x2(word(wb, m) & 0xFFFFu), a3 = e4m3x2_f16x2(word(wb, m) >> 16);
          const uint32_t b0 = e4m3x2_f16x2(word(b, m) & 0xFFFFu), b1 = e4m3x2_f16x2(word(b, m) >> 16);
          if (m == 0) mma16816_first<true>(part[u], a0, a1, a2, a3, b0, b1);
          else mma16816<true>(part[u], a0, a1, a2, a3, b0, b1);
        }
      }
      const float2 sa = *reinterpret_cast<const float2*>(as + (s * STEP / 128) * 8 + 2 * t4);
      const uint2 sw = lds64(src + 2048);
      const float w0 = __uint_as_float(sw.x), w1 = SWIGLU ? __uint_as_float(sw.y) : w0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float f = j & 1 ? sa.y : sa.x;
        if (SWIGLU) {
          acc[0][j] = fmaf(part[0][j], f * w0, acc[0][j]);
          acc[SETS - 1][j] = fmaf(part[1][j], f * w1, acc[SETS - 1][j]);
        } else {
          acc[0][j] = fmaf(part[0][j] + part[1][j], f * w0, acc[0][j]);
        }
      }
      src += kStage;
      if (src >= iend) src = ring;
    }
#pragma unroll
    for (int y = 0; y < SETS; ++y)
#pragma unroll
      for (int j = 0; j < 4; j += 2)
        *reinterpret_cast<float2*>(red + ((warp * SETS + y) * 16 + g + 4 * j) * 8 + 2 * t4) =
            make_float2(acc[y][j], acc[y][j + 1]);
    __syncthreads();
    if (!SWIGLU) {
      if (tid < 128) {
        const int row = tid & 15, t = tid >> 4;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += red[(w * 16 + row) * 8 + t];
        const int n = unit * 16 + row;
        if (t < p.M && n < p.N) {
          const int64_t at = t * p.out_stride + n;
          if (p.out_dtype == 0) {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at;
            *o = __float2bfloat16_rn(p.accumulate ? v + __bfloat162float(*o) : v);
          } else if (p.out_dtype == 1) {
            __half* o = static_cast<__half*>(p.out) + at;
            *o = __float2half_rn(p.accumulate ? v + __half2float(*o) : v);
          } else {
            float* o = static_cast<float*>(p.out) + at;
            *o = p.accumulate ? v + *o : v;
          }
        }
      }
      __syncthreads();
      continue;
    }
    // SWIGLU: thread (row of the 16, activation row)
    if (tid < 128) {
      const int i = tid & 15, t = tid >> 4;
      float gate = 0.f, up = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        gate += red[((w * SETS) * 16 + i) * 8 + t];
        up += red[((w * SETS + SETS - 1) * 16 + i) * 8 + t];
      }
      // (the fast exponential's error grows with |gate|; here the full one costs nothing)
      if (t < p.M) __stcg(p.act + static_cast<int64_t>(t) * p.N + unit * 16 + i, __fdiv_rn(gate, 1.0f + expf(-gate)) * up);
      __threadfence();
    }
    __syncthreads();
    if (tid == 0) {
      last = atomicAdd(p.tickets + unit / 8, 1u) == 7u;
      if (last) p.tickets[unit / 8] = 0;  // for the next call
    }
    __syncthreads();
    if (last) {
      // warp t: row t of the block, four columns a lane
      __threadfence();
      if (warp < p.M) {
        const int64_t n0 = static_cast<int64_t>(unit / 8) * 128;
        const float4 v = __ldcg(reinterpret_cast<const float4*>(p.act + static_cast<int64_t>(warp) * p.N + n0) + lane);
        float m = max_nan(max_nan(fabsf(v.x), fabsf(v.y)), max_nan(fabsf(v.z), fabsf(v.w)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float whole = __fdiv_rn(m, 448.0f), scale = whole == 0.f ? 1.0f : whole;
        if (lane == 0) p.scales[static_cast<int64_t>(warp) * (p.N / 128) + unit / 8] = scale;
        reinterpret_cast<uint32_t*>(p.codes + static_cast<int64_t>(warp) * p.N + n0)[lane] =
            f32x2_to_e4m3x2(__fdiv_rn(v.x, scale), __fdiv_rn(v.y, scale)) |
            (static_cast<uint32_t>(f32x2_to_e4m3x2(__fdiv_rn(v.z, scale), __fdiv_rn(v.w, scale))) << 16);
      }
    }
    __syncthreads();
  }
}

// smem before the rings
template <bool SWIGLU>
int fixed_bytes(const Fp8GemmArgs& p) {
  return kRed<SWIGLU> + (p.K + 127) / 128 * 32 + (p.M * code_stride(p.K) + 127) / 128 * 128;
}
template <bool SWIGLU>
int depth_of(const Fp8GemmArgs& p, int smem = kFewSmem<SWIGLU>) {
  return std::min(kMaxFewDepth, (smem - fixed_bytes<SWIGLU>(p)) / (kFewWarps<SWIGLU> * kStage));
}

template <bool SWIGLU>
cudaError_t launch(const Fp8GemmArgs& p, int depth, int grid, cudaStream_t s) {
  static int configured[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64 || configured[dev] == 0) {
    err = cudaFuncSetAttribute(fp8_few_kernel<SWIGLU>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem<SWIGLU>);
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  const size_t smem = static_cast<size_t>(fixed_bytes<SWIGLU>(p)) + static_cast<size_t>(depth) * kFewWarps<SWIGLU> * kStage;
  return launch_pdl(fp8_few_kernel<SWIGLU>, dim3(grid), dim3(32 * kFewWarps<SWIGLU>), smem, s, p, depth);
}

}  // namespace

size_t fp8_few_scratch(int M, int N) { return kFewTicketBytes + static_cast<size_t>(M) * N * 4; }

// At most 8 rows whose codes leave room for a ring of two stages a warp, and
// with SwiGLU scratch for them and a ticket for each block.
bool fp8_few_fits(const Fp8GemmArgs& p) {
  if (p.M > 8 || p.K > 65536) return false;
  return p.codes != nullptr ? p.tickets != nullptr && depth_of<true>(p) >= 2 : depth_of<false>(p) >= 2;
}

cudaError_t launch_fp8_few(const Fp8GemmArgs& p, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  if (p.codes != nullptr) return launch<true>(p, depth_of<true>(p), std::min(p.N / 16, di.sms), s);
  const int units = (p.N + 15) / 16;
  const int third = depth_of<false>(p, kThirdSmem);
  // Three CTAs an SM where that takes an SM's units in better balance, or nearly as
  // good: 3 / 2 CTAs, one row, weights from memory, N x K = 7168 x 2048 (3 / 4 units an
  // SM) 4.5 / 5.7 us, 14336 x 4096 (6 / 6) 12.0 / 13.1, 16384 x 7168 (9 / 8) 23.4 / 24.3,
  // 9000 x 1104 (6 / 4) 5.4 / 4.7
  const int on3 = 3 * ((units + 3 * di.sms - 1) / (3 * di.sms)), on2 = 2 * ((units + 2 * di.sms - 1) / (2 * di.sms));
  if (units > 2 * di.sms && 4 * on3 <= 5 * on2 && third >= 3)
    return launch<false>(p, third, std::min(units, 3 * di.sms), s);
  return launch<false>(p, depth_of<false>(p), std::min(units, 2 * di.sms), s);
}

}  // namespace moe
