// Norms of the query and key heads, the rotation of their positions and the
// write of new keys and values into the paged cache (moe_qk_norm_rope), in one
// pass: every value is read once and written once (the keys' norm, rotation and
// 8-bit scale all come from registers).  Bound by memory.
//
// A head is held by LANES lanes of a warp, 8 values (16 bytes) each, so its mean
// and its largest value are a few shuffles; a CTA takes heads of one token, whose
// angles it computes once.  An angle is a fraction of a turn in 64 bits,
// position * turns mod 2^64, which is exact, where position * frequency in float
// is off by 0.06 radians at position 10^6.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 128;  // D <= 256

template <typename T>
__device__ __forceinline__ float2 two_f32(uint32_t v);
template <>
__device__ __forceinline__ float2 two_f32<__nv_bfloat16>(uint32_t v) {
  return make_float2(bf16_lo(v), bf16_hi(v));
}
template <>
__device__ __forceinline__ float2 two_f32<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}
template <typename T>
__device__ __forceinline__ uint32_t two_from(float a, float b);
template <>
__device__ __forceinline__ uint32_t two_from<__nv_bfloat16>(float a, float b) {
  return pack_bf16x2(a, b);
}
template <>
__device__ __forceinline__ uint32_t two_from<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = two_f32<T>(w[j]);
    x[2 * j] = f.x;
    x[2 * j + 1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(two_from<T>(x[0], x[1]), two_from<T>(x[2], x[3]), two_from<T>(x[4], x[5]), two_from<T>(x[6], x[7]));
}

// NaN wins, so that a head with one gets a NaN scale
__device__ __forceinline__ float max_nan(float a, float b) { return (a > b || a != a) ? a : b; }

template <typename T, int LANES>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  constexpr int kHeads = kRopeThreads / LANES;  // of a pass
  __shared__ float2 turn[kMaxPairs];            // cos and sin, times the magnitude
  __shared__ float spare[kRopeThreads / 32][32 * 9];
  const int tid = threadIdx.x, lane = tid & 31, in_head = tid & (LANES - 1);
  const int pairs = a.rot >> 1, chunks = a.D >> 3, heads = a.Hq + 2 * a.Hkv;
  const int64_t t = blockIdx.x;
  const bool mine = in_head < chunks;
  const int e0 = in_head * 8;  // this lane's values
  auto source = [&](int h) {   // of head h: queries, keys, values
    const T* p = h < a.Hq            ? static_cast<const T*>(a.q) + t * a.q_stride + static_cast<int64_t>(h) * a.D
                 : h < a.Hq + a.Hkv ? static_cast<const T*>(a.k) + t * a.k_stride + static_cast<int64_t>(h - a.Hq) * a.D
                                    : static_cast<const T*>(a.v) + t * a.v_stride +
                                          static_cast<int64_t>(h - a.Hq - a.Hkv) * a.D;
    return reinterpret_cast<const uint4*>(p + e0);
  };
  // without a cache the value heads are nobody's
  const int last = a.cache.k != nullptr ? heads : a.Hq + a.Hkv;
  const int step = kHeads * gridDim.y;
  int h = blockIdx.y * kHeads + tid / LANES;
  pdl_wait();
  pdl_trigger();
  uint4 next = mine && h < last ? *source(h) : make_uint4(0, 0, 0, 0);
  int64_t slot = -1;
  if (a.cache.k != nullptr) {
    slot = a.slots[t];
    if (slot >= a.capacity) {
      if (tid == 0 && blockIdx.y == 0) record_error(a.err, kErrBadIndex, static_cast<uint32_t>(t));
      slot = -1;
    }
  }
  if (tid < pairs) {
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(a.positions[t])) * a.turns[tid];
    // the upper half as a signed fraction of a turn: within 2^-26 of a turn
    const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    turn[tid] = make_float2(c * a.magnitude, s * a.magnitude);
  }
  __syncthreads();

  // (every lane of a warp goes through the same number of passes)
  for (int h0 = blockIdx.y * kHeads; h0 < last; h0 += step, h += step) {
    const uint4 raw = next;
    next = mine && h + step < last ? *source(h + step) : make_uint4(0, 0, 0, 0);
    const bool live = mine && h < last, value = h >= a.Hq + a.Hkv, query = h < a.Hq;
    const void* weight = value ? nullptr : query ? a.q_weight : a.k_weight;
    float x[8];
    unpack8<T>(raw, x);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (weight != nullptr && mine) {
      const float r = 1.0f / sqrtf(sum / static_cast<float>(a.D) + a.eps);
      float w[8];
      if (a.weight_f32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(weight) + e0);
        const float4 u = p[0], v = p[1];
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
      } else {
        unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(weight) + e0), w);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
    }
    if (a.interleaved) {
      if (!value) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (e0 + 2 * j < a.rot) {
            const float2 f = turn[e0 / 2 + j];
            const float u = x[2 * j], v = x[2 * j + 1];
            x[2 * j] = fmaf(u, f.x, -v * f.y);
            x[2 * j + 1] = fmaf(v, f.x, u * f.y);
          }
        }
      }
    } else if (pairs > 0) {
      // the other half's values, from the lane that holds them (whole chunks), or
      // through shared memory where the halves do not begin at a chunk
      float y[8];
      const bool front = e0 < pairs;
      if ((pairs & 7) == 0) {
        const int from = lane + (front ? pairs / 8 : -(pairs / 8));
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = __shfl_sync(0xffffffffu, x[j], from & 31);
      } else {
        float* buf = spare[tid >> 5];
#pragma unroll
        for (int j = 0; j < 8; ++j) buf[lane * 9 + j] = x[j];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = e0 + j, other = e < pairs ? e + pairs : e < a.rot ? e - pairs : e;
          y[j] = buf[((lane & ~(LANES - 1)) + (other >> 3)) * 9 + (other & 7)];
        }
        __syncwarp();
      }
      if (!value && mine) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = e0 + j;
          if (e < a.rot) {
            const bool first = e < pairs;
            const float2 f = turn[first ? e : e - pairs];
            x[j] = fmaf(x[j], f.x, first ? -y[j] * f.y : y[j] * f.y);
          }
        }
      }
    }
    if (query) {
      if (live)
        *reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + t * a.q_out_stride + static_cast<int64_t>(h) * a.D + e0) =
            pack8<T>(x);
      continue;
    }
    const int hk = value ? h - a.Hq - a.Hkv : h - a.Hq;
    if (live && !value && a.k_out != nullptr)
      *reinterpret_cast<uint4*>(static_cast<T*>(a.k_out) + t * a.k_out_stride + static_cast<int64_t>(hk) * a.D + e0) =
          pack8<T>(x);
    if (slot < 0) continue;
    const int64_t page = slot >> a.page_shift, place = slot & ((1 << a.page_shift) - 1);
    const KvCache& c = a.cache;
    const int64_t at = (value ? page * c.v_page + place * c.v_token + hk * c.v_head
                              : page * c.k_page + place * c.k_token + hk * c.k_head) + e0;
    uint8_t* to = value ? c.v : c.k;
    if (!a.e4m3) {
      if (live) *reinterpret_cast<uint4*>(to + 2 * at) = pack8<T>(x);
      continue;
    }
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max_nan(amax, fabsf(x[j]));
    // only the lanes of this head: others of the warp may have left the pass for a query
    const uint32_t group = LANES == 32 ? 0xffffffffu : ((1u << (LANES & 31)) - 1u) << (lane & ~(LANES - 1));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(group, amax, o));
    float scale = __fdiv_rn(amax, 448.0f);
    if (scale == 0.f) scale = 1.0f;
    if (!live) continue;
    if (in_head == 0)
      (value ? c.v_scale : c.k_scale)[((page * a.Hkv + hk) << a.page_shift) + place] = scale;
    uint32_t code[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) code[j] = f32x2_to_e4m3x2(__fdiv_rn(x[2 * j], scale), __fdiv_rn(x[2 * j + 1], scale));
    *reinterpret_cast<uint2*>(to + at) = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
  }
}

template <typename T, int LANES>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  // a token's heads in one CTA, or over several where the tokens leave SMs idle
  constexpr int kHeads = kRopeThreads / LANES;
  const int passes = (a.Hq + (a.cache.k != nullptr ? 2 : 1) * a.Hkv + kHeads - 1) / kHeads;
  const int spread = std::max(1, std::min(passes, 2 * a.sms / a.T));
  return launch_pdl(rope_kernel<T, LANES>, dim3(a.T, spread), dim3(kRopeThreads), 0, s, a);
}

template <typename T>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  if (a.D <= 64) return launch<T, 8>(a, s);
  if (a.D <= 128) return launch<T, 16>(a, s);
  return launch<T, 32>(a, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t s) {
  return dtype == 0 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // namespace moe
