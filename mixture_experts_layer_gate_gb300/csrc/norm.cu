// Residual add + RMS norm with an optional 8-bit copy of the result
// (moe_add_rms_norm): s = x + residual, v = s * weight * rsqrt(mean(s^2) + eps),
// and per block of 128 columns or per row scale = max |v| / 448, code =
// e4m3(v / scale).
//
// One pass over the data: a row's sums stay in registers between the mean, the
// norm and the quantisation, so every input is read and every output written
// once.  Bound by memory.  A row is held by TPR threads (a multiple of 32), 8
// columns of it per thread and chunk, CH chunks; rows of up to 1024 columns share
// a CTA of 256 threads, longer ones have a CTA of their own size, and the
// CTAs of a large batch go through its rows with the weight in registers and the
// next row's loads in flight.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kNormThreads = 256;      // rows of one warp
// a row of a whole CTA: at most 1024 threads of one chunk or 512 of two or four
__host__ __device__ constexpr int wide_threads(int ch) { return ch == 1 ? 1024 : 512; }

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  return static_cast<float>(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  return static_cast<T>(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

// Column of element j of this thread's chunk c.  VEC: 8 adjacent columns per
// lane (16-byte pieces, 16 lanes hold a quantisation block).  Else 32 adjacent
// columns per warp and element (a row that is not 16-byte aligned: each load
// of a warp is still one contiguous run, elements 0-3 and 4-7 hold a block each).
template <bool VEC>
__device__ __forceinline__ int column(int c, int j, int tpr, int tr) {
  const int base = c * tpr * 8;
  return VEC ? base + tr * 8 + j : base + (tr & ~31) * 8 + j * 32 + (tr & 31);
}

// Eight elements as they are stored, until they are used.
template <typename T>
struct alignas(16) Raw {
  T u[8];
};

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int c, int tpr, int tr, int H, Raw<T>& r) {
  if (VEC) {
    const int i = column<true>(c, 0, tpr, tr);
    constexpr int n = sizeof(T) * 8 / 16;
#pragma unroll
    for (int k = 0; k < n; ++k)
      reinterpret_cast<uint4*>(r.u)[k] =
          i < H ? reinterpret_cast<const uint4*>(row + i)[k] : make_uint4(0, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = column<false>(c, j, tpr, tr);
      r.u[j] = i < H ? row[i] : from_f32<T>(0.f);
    }
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, int c, int tpr, int tr, int H, const float (&v)[8]) {
  if (VEC) {
    const int i = column<true>(c, 0, tpr, tr);
    if (i < H) {
      alignas(16) T u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = from_f32<T>(v[j]);
      constexpr int n = sizeof(T) * 8 / 16;
#pragma unroll
      for (int k = 0; k < n; ++k) reinterpret_cast<uint4*>(row + i)[k] = reinterpret_cast<uint4*>(u)[k];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = column<false>(c, j, tpr, tr);
      if (i < H) row[i] = from_f32<T>(v[j]);
    }
  }
}

struct Add {
  static __device__ __forceinline__ float f(float a, float b) { return a + b; }
};
// NaN wins, so that a row with one gets a NaN scale
struct MaxNan {
  static __device__ __forceinline__ float f(float a, float b) {
    return (a > b || a != a) ? a : b;
  }
};

// Reduction over the threads of a row, the same on all of them; `part` holds a
// float per warp of the CTA.  Every thread of the CTA calls it.
template <typename Op, bool WIDE>
__device__ __forceinline__ float row_reduce(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = Op::f(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (WIDE) {  // the CTA's one row
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();  // the previous reduction's partial results have been read
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[lane < warps ? lane : 0];
    if (lane >= warps) v = 0.f;  // (no sum and no magnitude is below it)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = Op::f(v, __shfl_xor_sync(0xffffffffu, v, o));
  }
  return v;
}

// v / scale to within the quotient's last bits: by the reciprocal, unless that
// would overflow (an IEEE division per value took a third of the kernel's time).
struct Quotient {
  float scale, r;
  __device__ __forceinline__ explicit Quotient(float s) {
    scale = s;
    r = s < 1e-37f ? 0.f : __fdiv_rn(1.0f, s);
  }
  __device__ __forceinline__ float operator()(float v) const { return r == 0.f && scale < 1.f ? __fdiv_rn(v, scale) : v * r; }
};

__device__ __forceinline__ float scale_of(float amax) {
  // 1 for a block of zeros, or of values so small that the scale would be zero; a
  // NaN (or infinite) maximum stays one
  const float s = __fdiv_rn(amax, 448.0f);
  return s == 0.f ? 1.0f : s;
}

template <typename T, typename W, bool VEC, bool WIDE, int CH>
__global__ void __launch_bounds__(WIDE ? wide_threads(CH) : kNormThreads, WIDE && CH == 2 ? 2 : 1)
    add_rms_norm_kernel(NormArgs a) {
  // (where a CTA takes one row, registers for another's loads would cost occupancy)
  constexpr bool kLoop = WIDE && CH == 2;
  __shared__ float part[32];
  const int TPR = WIDE ? blockDim.x : 32;
  const int tr = WIDE ? threadIdx.x : threadIdx.x & 31;
  const int per = WIDE ? 1 : kNormThreads / 32;  // rows of a CTA
  const int step = gridDim.x * per, H = a.H;
  int t = static_cast<int>(blockIdx.x) * per + (WIDE ? 0 : threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  if (t >= a.T) return;  // (a whole warp; a CTA of one row has one)
  const T* x = static_cast<const T*>(a.x);
  const T* residual = static_cast<const T*>(a.residual);
  Raw<T> xr[CH], rr[CH];
  Raw<W> wr[CH];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < CH; ++c) load8<T, VEC>(x + row * a.x_stride, c, TPR, tr, H, xr[c]);
    if (residual != nullptr) {
#pragma unroll
      for (int c = 0; c < CH; ++c) load8<T, VEC>(residual + row * a.residual_stride, c, TPR, tr, H, rr[c]);
    }
  };
  fetch(t);
#pragma unroll
  for (int c = 0; c < CH; ++c) load8<W, VEC>(static_cast<const W*>(a.weight), c, TPR, tr, H, wr[c]);
  for (; t < a.T; t += kLoop ? step : a.T) {
    const int64_t tt = t;
    float s[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[c][j] = to_f32(xr[c].u[j]) + (residual != nullptr ? to_f32(rr[c].u[j]) : 0.f);
    if (kLoop && t + step < a.T) fetch(t + step);  // the next row's loads run while this row is finished
    if (a.residual_out != nullptr) {
      T* o = static_cast<T*>(a.residual_out) + tt * a.residual_out_stride;
#pragma unroll
      for (int c = 0; c < CH; ++c) store8<T, VEC>(o, c, TPR, tr, H, s[c]);
    }
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(s[c][j], s[c][j], sum);
    sum = row_reduce<Add, WIDE>(sum, part);
    const float r = rsqrtf(sum / static_cast<float>(a.H) + a.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[c][j] = s[c][j] * r * to_f32(wr[c].u[j]);
    if (a.y != nullptr) {
      T* o = static_cast<T*>(a.y) + tt * a.y_stride;
#pragma unroll
      for (int c = 0; c < CH; ++c) store8<T, VEC>(o, c, TPR, tr, H, s[c]);
    }
    if (a.quant == 0) continue;

    float row_scale = 0.f;
    if (a.quant == 2) {
      float m = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = MaxNan::f(m, fabsf(s[c][j]));
      row_scale = scale_of(row_reduce<MaxNan, WIDE>(m, part));
      if (tr == 0) a.scales[t] = row_scale;
    }
    const int nb = (a.H + 127) / 128;
    uint8_t* codes = a.codes + tt * a.H;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float lo = row_scale, hi = row_scale;  // scales of elements 0-3 and 4-7
      if (a.quant == 1) {
        float m0 = 0.f, m1 = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          m0 = MaxNan::f(m0, fabsf(s[c][j]));
          m1 = MaxNan::f(m1, fabsf(s[c][4 + j]));
        }
        if (VEC) {
          m0 = MaxNan::f(m0, m1);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) m0 = MaxNan::f(m0, __shfl_xor_sync(0xffffffffu, m0, o));
          m1 = m0;
        } else {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            m0 = MaxNan::f(m0, __shfl_xor_sync(0xffffffffu, m0, o));
            m1 = MaxNan::f(m1, __shfl_xor_sync(0xffffffffu, m1, o));
          }
        }
        lo = scale_of(m0);
        hi = scale_of(m1);
        const int i0 = column<VEC>(c, 0, TPR, tr), i1 = column<VEC>(c, 4, TPR, tr);
        if (VEC ? tr % 16 == 0 : tr % 32 == 0) {
          if (i0 < H) a.scales[tt * nb + i0 / 128] = lo;
          if (!VEC && i1 < H) a.scales[tt * nb + i1 / 128] = hi;
        }
      }
      const Quotient qlo(lo), qhi(VEC ? lo : hi);
      uint16_t q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Quotient& d = j < 2 ? qlo : qhi;
        q[j] = f32x2_to_e4m3x2(d(s[c][2 * j]), d(s[c][2 * j + 1]));
      }
      if (VEC) {
        const int i = column<true>(c, 0, TPR, tr);
        if (i < H)
          *reinterpret_cast<uint2*>(codes + i) =
              make_uint2(q[0] | (static_cast<uint32_t>(q[1]) << 16), q[2] | (static_cast<uint32_t>(q[3]) << 16));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = column<false>(c, j, TPR, tr);
          if (i < H) codes[i] = static_cast<uint8_t>(q[j / 2] >> (8 * (j & 1)));
        }
      }
    }
  }
}

template <typename T, typename W, bool VEC, int CH>
cudaError_t launch_warp(const NormArgs& a, cudaStream_t s) {
  constexpr int R = kNormThreads / 32;
  return launch_pdl(add_rms_norm_kernel<T, W, VEC, false, CH>, dim3((a.T + R - 1) / R), dim3(kNormThreads), 0, s, a);
}
template <typename T, typename W, bool VEC, int CH>
cudaError_t launch_wide(const NormArgs& a, cudaStream_t s) {
  const int chunks = (a.H + 7) / 8, threads = ((chunks + CH - 1) / CH + 31) / 32 * 32;
  const int grid = CH == 2 ? std::min(a.T, std::max(1, 1024 / threads) * a.sms) : a.T;  // (as many as registers let live)
  return launch_pdl(add_rms_norm_kernel<T, W, VEC, true, CH>, dim3(grid), dim3(threads), 0, s, a);
}

// A warp a row up to 1024 columns.  Beyond, a CTA a row: with one chunk a thread
// while the SMs hold all rows at once (the latency of a row counts), else with two,
// going through the rows with the next one's loads in flight; four for rows of over
// 8192 columns.  In a graph, f16 / bf16, block codes and (without a residual) y only:
//   one chunk / two, H = 1536: 608 rows 2.5 / 3.0 us and 1.7 / 1.9, 4096 rows 12.1 /
//   12.9 and 5.6 / 5.4; H = 4096: 456 rows 3.6 / 4.4 and 2.2 / 2.5, 608 rows 5.2 /
//   4.6 and 3.1 / 2.5; H = 7168: 152 rows 2.7 / 3.3 and 1.9 / 2.0, 304 rows 4.9 / 4.1
//   and 3.2 / 2.5.
// Rows that are not 16-byte aligned take one chunk whatever their number: two take
// twice as many small loads to start (H = 2571: 333 rows 4.1 / 7.4 us and 2.4 / 3.7,
// 4096 rows 30 / 53 and 17 / 22; H = 7167: 4096 rows 103 / 119).  Of long rows for y
// alone two would be faster (H = 7167: 4096 rows 60 / 49).
// T = 4096, H = 7168, residual and block codes, event times with 4 us of launch: two
// chunks, two CTAs an SM 50 us, three 61 (spills), one chunk 52, four chunks 85 (14
// warps an SM); without the next row's loads in flight 54.  H = 4096: four CTAs an SM
// 31 us, two 37.
template <typename T, typename W, bool VEC>
cudaError_t launch_shape(const NormArgs& a, cudaStream_t s) {
  const int chunks = (a.H + 7) / 8;
  if (chunks <= 32) return launch_warp<T, W, VEC, 1>(a, s);
  if (chunks <= 64) return launch_warp<T, W, VEC, 2>(a, s);
  if (chunks <= 128) return launch_warp<T, W, VEC, 4>(a, s);
  if (chunks > 1024) return launch_wide<T, W, VEC, 4>(a, s);
  if constexpr (VEC) {
    const int rows = 1536 / ((chunks + 31) / 32 * 32);  // of one chunk a thread that an SM holds
    if (a.T > rows * a.sms) return launch_wide<T, W, VEC, 2>(a, s);
  }
  return launch_wide<T, W, VEC, 1>(a, s);
}

template <typename T, typename W>
cudaError_t launch_vec(const NormArgs& a, cudaStream_t s) {
  return a.vec ? launch_shape<T, W, true>(a, s) : launch_shape<T, W, false>(a, s);
}

template <typename T>
cudaError_t launch_weight(const NormArgs& a, int weight_f32, cudaStream_t s) {
  return weight_f32 ? launch_vec<T, float>(a, s) : launch_vec<T, T>(a, s);
}

}  // namespace

cudaError_t launch_add_rms_norm(const NormArgs& a, int dtype, int weight_f32, cudaStream_t s) {
  if (dtype == 0) return launch_weight<__nv_bfloat16>(a, weight_f32, s);
  if (dtype == 1) return launch_weight<__half>(a, weight_f32, s);
  return launch_vec<float, float>(a, s);
}

}  // namespace moe
