// Norms of the query and key heads, the rotation of their positions and the
// write of new keys and values into the paged cache (moe_qk_norm_rope), in one
// pass: every value is read once and written once (the keys' norm, rotation and
// 8-bit scale all come from registers).  Bound by memory.
//
// A head is held by LANES lanes of a warp, 8 values (16 bytes) each, so its mean
// and its largest value are a few shuffles; a warp takes some of a token's heads,
// kAhead loads at a time, and computes the token's angles once, each lane some pairs,
// handed on by shuffles (no shared memory, no barrier).  An angle is a fraction of a
// turn in 64 bits, position * turns mod 2^64, which is exact, where position *
// frequency in float is off by 0.06 radians at position 10^6.
//
// In a graph, 32 query and 8 key heads of 128, bf16: 4096 tokens 31 us = 3.3 TB/s (58%
// of the issue slots, latency in the rest), 16384 94 us = 4.3 TB/s; a CTA a token, with
// a barrier for its angles, 48 and 150.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kAhead = 4;        // loads of a lane in flight
constexpr int kWarpsPerSm = 48;  // asked for; 24 of them run at a time (80 registers)

// (eight values of a head are four pairs of floats)
template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& r, uint64_t (&x)[4]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      x[j] = pack2(f.x, f.y);
    } else {
      x[j] = pack2(bf16_lo(w[j]), bf16_hi(w[j]));
    }
  }
}
template <bool F16>
__device__ __forceinline__ uint4 pack8(const uint64_t (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (F16) {
      const __half2 h = __floats2half2_rn(lo2(x[j]), hi2(x[j]));
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      w[j] = pack_bf16x2(lo2(x[j]), hi2(x[j]));
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// NaN wins, so that a head with one gets a NaN scale
__device__ __forceinline__ float max_nan(float a, float b) { return (a > b || a != a) ? a : b; }

// A head's values as e4m3 codes with its scale; of the lanes of one head.
template <int LANES>
__device__ __forceinline__ void store_codes(const uint64_t (&x)[4], uint8_t* to, float* scale_to, int lane, bool live, bool first) {
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) amax = max_nan(amax, max_nan(fabsf(lo2(x[j])), fabsf(hi2(x[j]))));
  // only the lanes of this head: others of the warp may have a query
  const uint32_t members = LANES == 32 ? 0xffffffffu : ((1u << (LANES & 31)) - 1u) << (lane & ~(LANES - 1));
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(members, amax, o));
  float scale = __fdiv_rn(amax, 448.0f);
  if (scale == 0.f) scale = 1.0f;
  if (!live) return;
  if (first) *scale_to = scale;
  uint32_t code[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) code[j] = f32x2_to_e4m3x2(__fdiv_rn(lo2(x[j]), scale), __fdiv_rn(hi2(x[j]), scale));
  *reinterpret_cast<uint2*>(to) = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
}

template <bool F16, int LANES, bool NORM, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_kernel(const RopeArgs a, const int groups) {
  constexpr int kHeads = 32 / LANES;  // of a pass
  constexpr int kPairs = LANES / 8;   // pairs whose angle a lane computes (D <= 8 LANES has 4 LANES pairs at most)
  __shared__ float spare[kRopeThreads / 32][32 * 9];
  const int lane = threadIdx.x & 31, in_head = lane & (LANES - 1);
  const int pairs = a.rot >> 1, chunks = a.D >> 3, D = a.D;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = unit / groups;
  if (t >= a.T) return;
  const int group = static_cast<int>(unit - t * groups);
  const bool mine = in_head < chunks;
  const int e0 = in_head * 8;  // this lane's values
  const int turned = a.Hq + a.Hkv, step = kHeads * groups;
  const int h_first = group * kHeads + lane / LANES;
  // this lane's place in the token's rows (heads times D fit 32 bits)
  const uint16_t* of_q = static_cast<const uint16_t*>(a.q) + t * a.q_stride + e0;
  const uint16_t* of_k = static_cast<const uint16_t*>(a.k) + t * a.k_stride + e0 - a.Hq * D;
  pdl_wait();
  pdl_trigger();
  uint4 raw[kAhead];
  auto fetch = [&](int h) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i, h += step)
      raw[i] = mine && h < turned ? *reinterpret_cast<const uint4*>((h < a.Hq ? of_q : of_k) + h * D) : make_uint4(0, 0, 0, 0);
  };
  fetch(h_first);
  int64_t slot = -1;
  if (a.cache.k != nullptr) {
    slot = a.slots[t];
    if (slot >= a.capacity) {
      if (lane == 0 && group == 0) record_error(a.err, kErrBadIndex, static_cast<uint32_t>(t));
      slot = -1;
    }
  }
  // the slot's keys and values, in bytes, and its place among the scales
  const KvCache& cache = a.cache;
  const int64_t page = slot < 0 ? 0 : slot >> a.page_shift, place = slot < 0 ? 0 : slot & ((1 << a.page_shift) - 1);
  const int size = a.e4m3 ? 1 : 2;
  const int64_t scale_at = ((page * a.Hkv) << a.page_shift) + place;
  // cos and sin of this lane's values' pairs, times the magnitude
  uint64_t co[4], si[4];
  if (pairs > 0) {
    const uint64_t position = static_cast<uint64_t>(static_cast<int64_t>(a.positions[t]));
    float c[kPairs], s[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int q = lane * kPairs + i;
      const uint64_t phase = q < pairs ? position * a.turns[q] : 0;
      // the upper half as a signed fraction of a turn: within 2^-26 of a turn
      sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &s[i], &c[i]);
      c[i] *= a.magnitude;
      s[i] *= a.magnitude;
    }
    float co8[8], si8[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = e0 + j, q = INTERLEAVED ? e >> 1 : e < pairs ? e : e - pairs;
      const int from = (q / kPairs) & 31;
      co8[j] = si8[j] = 0.f;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float u = __shfl_sync(0xffffffffu, c[i], from), v = __shfl_sync(0xffffffffu, s[i], from);
        if (q % kPairs == i) {
          co8[j] = u;
          si8[j] = v;
        }
      }
      if (INTERLEAVED ? (e & 1) == 0 : e < pairs) si8[j] = -si8[j];  // of the first of a pair
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      co[j] = pack2(co8[2 * j], co8[2 * j + 1]);
      si[j] = pack2(si8[2 * j], si8[2 * j + 1]);
    }
  }
  const float per_d = 1.0f / static_cast<float>(D);
  uint16_t* to_q = static_cast<uint16_t*>(a.q_out) + t * a.q_out_stride + e0;
  uint16_t* to_k = a.k_out != nullptr ? static_cast<uint16_t*>(a.k_out) + t * a.k_out_stride + e0 - a.Hq * D : nullptr;
  uint8_t* slot_k = cache.k + size * (page * cache.k_page + place * cache.k_token + e0);

  // ---- queries and keys (every lane of a warp goes through the same number of passes)
  int h = h_first;
  for (int h0 = group * kHeads; h0 < turned; h0 += kAhead * step) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i, h += step) {
      if (h0 + i * step >= turned) break;
      const bool live = mine && h < turned, query = h < a.Hq;
      uint64_t x[4];
      unpack8<F16>(raw[i], x);
      if (NORM) {
        const void* weight = query ? a.q_weight : a.k_weight;
        uint64_t sum2 = mul2(x[0], x[0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) sum2 = fma2(x[j], x[j], sum2);
        float sum = lo2(sum2) + hi2(sum2);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (weight != nullptr && mine) {
          const float r = rsqrtf(fmaf(sum, per_d, a.eps));
          uint64_t w[4];
          if (a.weight_f32) {
            const ulonglong2* p = reinterpret_cast<const ulonglong2*>(static_cast<const float*>(weight) + e0);
            w[0] = p[0].x, w[1] = p[0].y, w[2] = p[1].x, w[3] = p[1].y;
          } else {
            unpack8<F16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(weight) + e0), w);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = mul2(mul2(x[j], pack2(r, r)), w[j]);
        }
      }
      if (pairs > 0) {
        uint64_t y[4];  // the other of each value's pair
        if (INTERLEAVED) {
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = pack2(hi2(x[j]), lo2(x[j]));
        } else if ((pairs & 7) == 0) {
          // from the lane that holds the other half's chunk
          const int from = lane + (e0 < pairs ? pairs / 8 : -(pairs / 8));
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = __shfl_sync(0xffffffffu, x[j], from & 31);
        } else {
          // through shared memory where the halves do not begin at a chunk
          float* buf = spare[threadIdx.x >> 5];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            buf[lane * 9 + 2 * j] = lo2(x[j]);
            buf[lane * 9 + 2 * j + 1] = hi2(x[j]);
          }
          __syncwarp();
          float z[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int e = e0 + j, other = e < pairs ? e + pairs : e < a.rot ? e - pairs : e;
            z[j] = buf[((lane & ~(LANES - 1)) + (other >> 3)) * 9 + (other & 7)];
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = pack2(z[2 * j], z[2 * j + 1]);
          __syncwarp();
        }
        uint64_t z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = fma2(x[j], co[j], mul2(y[j], si[j]));
        if (e0 + 8 <= a.rot) {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = z[j];
        } else {  // the end of the rotated part
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[j] = pack2(e0 + 2 * j < a.rot ? lo2(z[j]) : lo2(x[j]), e0 + 2 * j + 1 < a.rot ? hi2(z[j]) : hi2(x[j]));
        }
      }
      if (query) {
        if (live) *reinterpret_cast<uint4*>(to_q + h * D) = pack8<F16>(x);
        continue;
      }
      if (live && to_k != nullptr) *reinterpret_cast<uint4*>(to_k + h * D) = pack8<F16>(x);
      if (slot < 0) continue;
      uint8_t* to = slot_k + size * (h - a.Hq) * cache.k_head;
      if (a.e4m3)
        store_codes<LANES>(x, to, cache.k_scale + scale_at + (static_cast<int64_t>(h - a.Hq) << a.page_shift), lane, live, in_head == 0);
      else if (live)
        *reinterpret_cast<uint4*>(to) = pack8<F16>(x);
    }
    fetch(h);
  }

  // ---- values
  if (slot < 0) return;
  const uint16_t* of_v = static_cast<const uint16_t*>(a.v) + t * a.v_stride + e0;
  uint8_t* slot_v = cache.v + size * (page * cache.v_page + place * cache.v_token + e0);
  for (h = h_first; h - lane / LANES < a.Hkv; h += 2 * step) {
    uint4 v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      v[i] = mine && h + i * step < a.Hkv ? *reinterpret_cast<const uint4*>(of_v + (h + i * step) * D) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool live = mine && h + i * step < a.Hkv;
      uint8_t* to = slot_v + size * (h + i * step) * cache.v_head;
      if (a.e4m3) {
        uint64_t x[4];
        unpack8<F16>(v[i], x);
        store_codes<LANES>(x, to, cache.v_scale + scale_at + (static_cast<int64_t>(h + i * step) << a.page_shift), lane, live, in_head == 0);
      } else if (live) {
        *reinterpret_cast<uint4*>(to) = v[i];
      }
    }
  }
}

template <bool F16, int LANES, bool NORM, bool INTERLEAVED>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  // A token's heads by one warp, or by several where there are fewer tokens than
  // kWarpsPerSm warps an SM.
  constexpr int kHeads = 32 / LANES;
  const int passes = (a.Hq + a.Hkv + kHeads - 1) / kHeads;
  const int groups = std::max(1, std::min(passes, (kWarpsPerSm * a.sms + a.T - 1) / a.T));
  const int64_t ctas = (static_cast<int64_t>(a.T) * groups + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  return launch_pdl(rope_kernel<F16, LANES, NORM, INTERLEAVED>, dim3(static_cast<unsigned>(ctas)), dim3(kRopeThreads), 0, s, a, groups);
}

template <bool F16, int LANES>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  const bool norm = a.q_weight != nullptr || a.k_weight != nullptr;
  if (norm) return a.interleaved ? launch<F16, LANES, true, true>(a, s) : launch<F16, LANES, true, false>(a, s);
  return a.interleaved ? launch<F16, LANES, false, true>(a, s) : launch<F16, LANES, false, false>(a, s);
}

template <bool F16>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  if (a.D <= 64) return launch<F16, 8>(a, s);
  if (a.D <= 128) return launch<F16, 16>(a, s);
  return launch<F16, 32>(a, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t s) {
  return dtype == 0 ? launch<false>(a, s) : launch<true>(a, s);
}

}  // namespace moe
