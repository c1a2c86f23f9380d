// Residual add + RMS norm with an optional 8-bit copy of the result
// (moe_add_rms_norm): s = x + residual, v = s * weight * rsqrt(mean(s^2) + eps),
// and per block of 128 columns or per row scale = max |v| / 448, code =
// e4m3(v / scale).
//
// One pass over the data: a row's sums stay in registers between the mean, the
// norm and the quantisation, so every input is read and every output written
// once.  Bound by memory.  A row is held by TPR threads, 8 columns of it per
// thread and chunk, CH chunks, and a CTA of 256 threads holds 256 / TPR rows.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kNormThreads = 256;

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

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int c, int tpr, int tr, int H, float (&v)[8]) {
  if (VEC) {
    const int i = column<true>(c, 0, tpr, tr);
    if (i < H) {
      alignas(16) T u[8];
      constexpr int n = sizeof(T) * 8 / 16;
#pragma unroll
      for (int k = 0; k < n; ++k) reinterpret_cast<uint4*>(u)[k] = reinterpret_cast<const uint4*>(row + i)[k];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = to_f32(u[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = column<false>(c, j, tpr, tr);
      v[j] = i < H ? to_f32(row[i]) : 0.f;
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
template <typename Op, int TPR>
__device__ __forceinline__ float row_reduce(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = Op::f(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    constexpr int W = TPR / 32;
    __syncthreads();  // the previous reduction's partial results have been read
    if ((threadIdx.x & 31) == 0) part[warp] = v;
    __syncthreads();
    const int w0 = warp / W * W;
    v = part[w0];
#pragma unroll
    for (int i = 1; i < W; ++i) v = Op::f(v, part[w0 + i]);
  }
  return v;
}

__device__ __forceinline__ float scale_of(float amax) {
  // 1 for a block of zeros; a NaN (or infinite) maximum stays one
  return amax == 0.f ? 1.0f : __fdiv_rn(amax, 448.0f);
}

template <typename T, typename W, bool VEC, int TPR, int CH>
__global__ void __launch_bounds__(kNormThreads) add_rms_norm_kernel(NormArgs a) {
  constexpr int R = kNormThreads / TPR;
  __shared__ float part[kNormThreads / 32];
  const int tr = threadIdx.x % TPR;
  const int t = blockIdx.x * R + threadIdx.x / TPR;
  const bool live = t < a.T;
  const int64_t tt = live ? t : 0;
  const int H = live ? a.H : 0;  // a thread without a row reads and writes nothing
  pdl_wait();
  pdl_trigger();
  float s[CH][8];
  const T* x = static_cast<const T*>(a.x) + tt * a.x_stride;
#pragma unroll
  for (int c = 0; c < CH; ++c) load8<T, VEC>(x, c, TPR, tr, H, s[c]);
  if (a.residual != nullptr) {
    const T* r = static_cast<const T*>(a.residual) + tt * a.residual_stride;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float v[8];
      load8<T, VEC>(r, c, TPR, tr, H, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[c][j] += v[j];
    }
    if (a.residual_out != nullptr) {
      T* o = static_cast<T*>(a.residual_out) + tt * a.residual_out_stride;
#pragma unroll
      for (int c = 0; c < CH; ++c) store8<T, VEC>(o, c, TPR, tr, H, s[c]);
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(s[c][j], s[c][j], sum);
  sum = row_reduce<Add, TPR>(sum, part);
  const float r = rsqrtf(sum / static_cast<float>(a.H) + a.eps);
  const W* w = static_cast<const W*>(a.weight);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float v[8];
    load8<W, VEC>(w, c, TPR, tr, H, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[c][j] = s[c][j] * r * v[j];
  }
  if (a.y != nullptr) {
    T* o = static_cast<T*>(a.y) + tt * a.y_stride;
#pragma unroll
    for (int c = 0; c < CH; ++c) store8<T, VEC>(o, c, TPR, tr, H, s[c]);
  }
  if (a.quant == 0) return;

  float row_scale = 0.f;
  if (a.quant == 2) {
    float m = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = MaxNan::f(m, fabsf(s[c][j]));
    row_scale = scale_of(row_reduce<MaxNan, TPR>(m, part));
    if (live && tr == 0) a.scales[t] = row_scale;
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
    uint16_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float d = j < 2 ? lo : hi;
      q[j] = f32x2_to_e4m3x2(__fdiv_rn(s[c][2 * j], d), __fdiv_rn(s[c][2 * j + 1], d));
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

template <typename T, typename W, bool VEC, int TPR, int CH>
cudaError_t launch_one(const NormArgs& a, cudaStream_t s) {
  constexpr int R = kNormThreads / TPR;
  return launch_pdl(add_rms_norm_kernel<T, W, VEC, TPR, CH>, dim3((a.T + R - 1) / R), dim3(kNormThreads), 0, s, a);
}

// The fewest threads per row that hold it in at most 4 chunks of 8 columns per
// thread (8 beyond 8192 columns), so that short rows share a CTA.
template <typename T, typename W, bool VEC>
cudaError_t launch_shape(const NormArgs& a, cudaStream_t s) {
  const int chunks = (a.H + 7) / 8;
  if (chunks <= 32) return launch_one<T, W, VEC, 32, 1>(a, s);
  if (chunks <= 64) return launch_one<T, W, VEC, 32, 2>(a, s);
  if (chunks <= 128) return launch_one<T, W, VEC, 32, 4>(a, s);
  if (chunks <= 256) return launch_one<T, W, VEC, 64, 4>(a, s);
  if (chunks <= 512) return launch_one<T, W, VEC, 256, 2>(a, s);
  if (chunks <= 1024) return launch_one<T, W, VEC, 256, 4>(a, s);
  return launch_one<T, W, VEC, 256, 8>(a, s);
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
