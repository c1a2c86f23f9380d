// The MoE layer for a few tokens (moe_forward_few), in two launches.
//   up:   act[t, j, i] = silu(w13[e, i] . x[t]) (w13[e, I + i] . x[t]), e = ids[t, j]
//   down: out[t, h]    = sum_j w[t, j] (w2[e, h] . act[t, j])
// With at most 8 tokens the chosen experts' weights are read once and nothing
// else is large, so the layer is bound by the rate at which the weights stream
// in (int4: nearly by the integer work that unpacks them, see convert()).
// Measured in a graph: Mixtral bf16, 8 tokens 386 us = 6.6 TB/s, one token 106 us;
// DeepSeek-V3 int4, one token 59 us for 182 MB (the first kernel 4.9 TB/s, the
// second 3.1 TB/s), 8 tokens 312 us; Qwen2 fp8, one token 43 us.
//
// Every warp streams its own part of the weights through a private ring in
// shared memory (cp.async, 16 bytes a lane; a lane reads back what it copied
// itself) and multiplies 16 weight rows at a time with all tokens by
// mma.sync m16n8k16: the 8 columns are the tokens, and a weight is converted
// once for all of them.  The order of K inside a step is free as long as both
// operands agree, so a lane's 16 contiguous bytes of a weight row are its
// fragment, and the tokens are stored in the order that the weight format's
// lanes unpack (fragment order, frag_pos()).
//
// up: a CTA takes 16 gate rows and the 16 matching up rows of one expert, its 16
// warps each a part of K; the sums are joined in warp order.  Every CTA runs the
// gate for itself (one warp per token).  down: a CTA takes 16 rows of H and its
// warps the chosen experts' K axes laid end to end, so the weighted sum over
// experts needs no second pass.  The activations pass between the two in 32
// bits, but not as a float: as a bf16 and the bf16 of what that left over (two MMAs
// and no conversion; together within 2^-16 of the value, where out is rounded to
// 2^-8 in the end), or for fp8 as the format's codes.
#include <float.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "stream.cuh"

namespace moe {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxTopK = 32;
constexpr int kMaxSlots = kFewMaxTokens * kMaxTopK;
constexpr int kMaxDepth = 8;

// K per lane load of 16 bytes by four lanes, 16-byte slices of a token's
// fragment per load, and loads per step of the second kernel (one in the first).
// A step lies within one scale group of 128 (int4, int8).
template <int FMT>
struct Fmt;
template <>
struct Fmt<kW_BF16> {
  static constexpr int KC = 32, NS = 1, DOWN = 2;
};
template <>
struct Fmt<kW_FP8> {
  static constexpr int KC = 64, NS = 2, DOWN = 2;
};
template <>
struct Fmt<kW_INT8> {
  static constexpr int KC = 64, NS = 2, DOWN = 2;
};
template <>
struct Fmt<kW_INT4> {
  static constexpr int KC = 128, NS = 4, DOWN = 1;
};
template <int FMT>
constexpr bool kGrouped = FMT == kW_INT4 || FMT == kW_INT8;

// bytes of k weights of one row
template <int FMT>
__host__ __device__ constexpr int64_t row_bytes(int64_t k) {
  return FMT == kW_BF16 ? 2 * k : FMT == kW_INT4 ? k / 2 : k;
}

// Position of element k in fragment order: steps of KC, in a step slices of 8
// elements for each of four lanes.  int4 in the packed order unpacks a word's
// codes as the pairs (0, 4), (1, 5), (2, 6), (3, 7).
template <int FMT>
__device__ __forceinline__ int frag_pos(int k, int packed) {
  constexpr int KC = Fmt<FMT>::KC;
  const int r = k % KC, t = r / (KC / 4), q = r % (KC / 4), p = q & 7;
  const int pos = (FMT == kW_INT4 && packed) ? (p < 4 ? 2 * p : 2 * p - 7) : p;
  return k - r + (q >> 3) * 32 + t * 8 + pos;
}

// What a lane needs to turn codes into integers: flip is xored into the codes
// (signed ones become offset ones), then the offset is subtracted (one per row:
// the zero point, or the sign's offset).
struct Offset {
  uint32_t flip;
  uint32_t pair;   // int4: bf16x2 of 128 + offset
  float magic;     // int8: 2^23 + offset
  float plus;      // int4: 128 + offset
};

// The A registers (one row) of MMA m of a 16-byte load.
//   int4: a nibble in the low bits of the bf16 128.0 is 128 + code: a pair is a
//     shift and a masked xor; the 128 and the offset are taken off the pair
//     (SUB, exact), or by the caller off the product: sum (128 + c - p) x =
//     sum (128 + c) x - p sum x, a multiply-add per group of 128 instead of a
//     subtraction per pair (0.9 operations a code instead of 1.4)
//   int8: a byte in the low bits of the float 2^23 is 2^23 + code
//   fp8: the converter's f16 pairs
template <int FMT, bool SUB>
__device__ __forceinline__ void convert(const uint4& w, int m, const Offset& o, uint32_t& lo, uint32_t& hi) {
  if (FMT == kW_BF16) {
    lo = word(w, 2 * m);
    hi = word(w, 2 * m + 1);
  } else if (FMT == kW_FP8) {
    lo = e4m3x2_f16x2(word(w, m) & 0xFFFFu);
    hi = e4m3x2_f16x2(word(w, m) >> 16);
  } else if (FMT == kW_INT8) {
    const uint32_t v = word(w, m) ^ o.flip;
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = __uint_as_float(__byte_perm(v, 0x4B000000u, 0x7540u + i)) - o.magic;
    lo = pack_bf16x2(f[0], f[1]);
    hi = pack_bf16x2(f[2], f[3]);
  } else {
    const uint32_t v = word(w, m >> 1) >> (8 * (m & 1));
    lo = (v & 0x000F000Fu) ^ o.flip;
    hi = ((v >> 4) & 0x000F000Fu) ^ o.flip;
    if (SUB) {
      const __nv_bfloat162 off = *reinterpret_cast<const __nv_bfloat162*>(&o.pair);
      __nv_bfloat162 pa = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&lo), off);
      __nv_bfloat162 pb = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&hi), off);
      lo = *reinterpret_cast<uint32_t*>(&pa);
      hi = *reinterpret_cast<uint32_t*>(&pb);
    }
  }
}

// Where a row's group lies in the 4-byte words that are copied for it: index =
// (row * groups + group) modulo 4.  Rows of a tile are 16 r + g (+ 8, + I) with
// every other term a multiple of 4 groups, so index = g * groups + group for all
// the rows of a lane.
struct Place {
  uint32_t half;   // byte selector of the scale
  uint32_t shift;  // of the zero point
  __device__ __forceinline__ explicit Place(uint32_t index) {
    half = (index & 1u) ? 0x4432u : 0x4410u;
    shift = 8u * (index & 3u);
  }
};

// Scale and offset of one row's group.
template <int FMT>
__device__ __forceinline__ void group_of(uint32_t sword, uint32_t zword, const Place& at, bool zero, float& scale, Offset& o) {
  scale = __half2float(__ushort_as_half(static_cast<uint16_t>(__byte_perm(sword, 0u, at.half))));
  if (FMT == kW_INT4) {
    o.flip = zero ? 0x43004300u : 0x43084308u;
    o.pair = 0x43084308u;
    o.plus = 136.0f;
    if (zero) {
      const uint32_t z = (zword >> at.shift) & 255u;
      o.pair = 0x43004300u | z | (z << 16);
      o.plus = static_cast<float>(128u + z);
    }
  } else {
    o.flip = zero ? 0u : 0x80808080u;
    o.magic = 8388736.0f;
    if (zero) o.magic = static_cast<float>(8388608u + ((zword >> at.shift) & 255u));
  }
}

// What the chosen experts are, in shared memory: the distinct ones in ascending
// order, and for each which of the tokens' slots chose it.
struct Routing {
  int count;
  int32_t ids[kMaxSlots];              // per slot
  float w[kMaxSlots];                  // per slot
  uint32_t seen[32];                   // bit per expert
  int before[32];                      // chosen experts before each word's
  int16_t expert[kMaxSlots];
  uint8_t tokens[kMaxSlots];           // bit per token
  uint8_t slot[kMaxSlots][kFewMaxTokens];
  int most;                            // tokens of the expert with the most
};
// per chosen expert and token: the weight of the sum, 0 where the token did not choose it
typedef float (*Weights)[kFewMaxTokens];

// From r.ids (-1: no expert) and r.w; every thread of the CTA.  weight: null where it is not needed.
__device__ __forceinline__ void build_routing(Routing& r, const FewArgs& a, Weights weight) {
  const int S = a.T * a.k;
  if (threadIdx.x == 0) r.most = 1;
  for (int i = threadIdx.x; i < 32; i += kThreads) r.seen[i] = 0;
  if (weight != nullptr)
    for (int i = threadIdx.x; i < S * kFewMaxTokens; i += kThreads) (&weight[0][0])[i] = 0.f;
  for (int i = threadIdx.x; i < (S + 3) / 4; i += kThreads) reinterpret_cast<uint32_t*>(r.tokens)[i] = 0;
  __syncthreads();
  for (int s = threadIdx.x; s < S; s += kThreads)
    if (r.ids[s] >= 0) atomicOr(&r.seen[r.ids[s] >> 5], 1u << (r.ids[s] & 31));
  __syncthreads();
  if (threadIdx.x < 32) {
    const int n = __popc(r.seen[threadIdx.x]);
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (static_cast<int>(threadIdx.x) >= o) sum += v;
    }
    r.before[threadIdx.x] = sum - n;
    if (threadIdx.x == 31) r.count = sum;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < S; s += kThreads) {
    const int e = r.ids[s], t = s / a.k;
    if (e < 0) continue;
    const int at = r.before[e >> 5] + __popc(r.seen[e >> 5] & ((1u << (e & 31)) - 1u));
    r.expert[at] = static_cast<int16_t>(e);
    r.slot[at][t] = static_cast<uint8_t>(s);
    if (weight != nullptr) weight[at][t] = r.w[s];
    atomicOr(reinterpret_cast<uint32_t*>(r.tokens) + (at >> 2), 1u << (8 * (at & 3) + t));
  }
  __syncthreads();
  if (weight != nullptr) {  // (only the second kernel's ring goes by it)
    if (threadIdx.x < r.count) atomicMax(&r.most, __popc(r.tokens[threadIdx.x]));
    __syncthreads();
  }
}

__device__ __forceinline__ float block_max(float v, float* part) {
  v = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));  // v >= 0
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
  for (int i = 1; i < kWarps; ++i) v = fmaxf(v, part[i]);
  return v;
}

// 1 for zeros, and for values so small that the scale would be zero
__device__ __forceinline__ float act_scale_of(float amax) {
  const float s = __fdiv_rn(amax, 448.0f);
  return s == 0.f ? 1.0f : s;
}

// e4m3 of two values as the f16 pair that they stand for
__device__ __forceinline__ uint32_t quantised_f16x2(float a, float b) { return e4m3x2_f16x2(f32x2_to_e4m3x2(a, b)); }

constexpr size_t kRoutingBytes = (sizeof(Routing) + 127) / 128 * 128;
static_assert(kMaxSlots <= 256, "slots in a byte");
constexpr size_t kDownRedBytes = 2 * kWarps * 128 * 4;
constexpr size_t kWeightBytes = sizeof(float) * kMaxSlots * kFewMaxTokens;
// a warp's sums of 32 rows and 8 tokens; the up half starts in other banks
constexpr int kRedHalf = 16 * 8 + 16, kRedWarp = 2 * 16 * 8 + 16;
constexpr size_t kRedBytes = static_cast<size_t>(kWarps) * kRedWarp * 4;
// row stride of a token in shared memory: 64 bytes over a multiple of 128, so
// that the lanes of two tokens read different banks
__host__ __device__ constexpr int token_stride(int H) { return 2 * H + 64; }

template <int FMT>
constexpr int up_stage() {
  return 4 * 512 + (kGrouped<FMT> ? 256 : 0);
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// A float's order as an unsigned one (-0 as +0); 0, below every number, for NaN,
// which is never chosen.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return v != v ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The k best of the warp's keys (32 strided experts per register, 0: out of the
// running), ties to the lower expert: lane j returns the j-th expert, -1 where
// fewer were in the running.  A lane keeps the best of its own; a round is two warp
// reductions, after which the winner's lane looks for its next.
template <int EPL>
__device__ __forceinline__ int best_k(uint32_t (&key)[EPL], int k, int lane) {
  int mine = 0;
  uint32_t top = 0, at = 0;
  auto look = [&] {
    top = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) top = max(top, key[i]);
#pragma unroll
    for (int i = EPL - 1; i >= 0; --i)
      if (key[i] == top) at = static_cast<uint32_t>(lane + 32 * i);
  };
  look();
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, top);
    const uint32_t best = __reduce_min_sync(0xffffffffu, top == m && m != 0 ? at : 0xffffffffu);
    if (lane == j) mine = static_cast<int>(best);
    if (top == m && at == best) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (best == static_cast<uint32_t>(lane + 32 * i)) key[i] = 0;
      look();
    }
  }
  return mine;
}

// The gate of one token by one warp: moe_gate_topk's rule (gate_token.cuh), with
// reductions by the warp's integer unit, because here a single token's latency
// counts (DeepSeek-V3 gate of one token: 2 us against 8).  scratch: 32 * EPL floats.
template <int EPL>
__device__ __forceinline__ void gate_one(const GateArgs& a, int t, int lane, float* scratch, int32_t* ids, float* w) {
  const float* row = a.logits + static_cast<size_t>(t) * a.E;
  float val[EPL], bias[EPL];
  uint32_t key[EPL];
  float top = -FLT_MAX;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {  // (every load before the first use: their latencies overlap)
    const int e = lane + 32 * i;
    val[i] = e < a.E ? row[e] : -INFINITY;
    bias[i] = a.bias != nullptr && e < a.E ? a.bias[e] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    float l = val[i];
    if (l != l) l = -INFINITY;  // a NaN logit is read as -inf
    val[i] = l;
    top = fmaxf(top, l);
  }
  float inv_z = 1.0f;
  if (!a.sigmoid) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      key[i] = ordered(val[i]);
      val[i] = lane + 32 * i < a.E ? expf(val[i] - top) : 0.f;
      z += val[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    inv_z = 1.0f / z;
  } else {
    const bool raw = a.n_group == 0 && a.bias == nullptr;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      const float s = 1.0f / (1.0f + expf(-val[i]));
      const float kk = raw ? val[i] : s + bias[i];
      key[i] = ordered(kk);
      val[i] = s;
      if (a.n_group > 0 && e < a.E) scratch[e] = kk == kk ? kk : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (lane + 32 * i >= a.E) key[i] = 0;
  if (a.n_group > 0) {
    // a group's two largest keys, by `per` lanes a group
    __syncwarp();
    const int gs = a.E / a.n_group;
    const int shift = 31 - __clz(32 / a.n_group), per = 1 << shift;
    const int g = lane >> shift, p = lane & (per - 1);
    float m1 = -INFINITY, m2 = -INFINITY;
    if (g < a.n_group)
      for (int j = p; j < gs; j += per) {
        const float v = scratch[g * gs + j];
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
    for (int o = per / 2; o > 0; o >>= 1) {
      const float b1 = __shfl_xor_sync(0xffffffffu, m1, o), b2 = __shfl_xor_sync(0xffffffffu, m2, o);
      m2 = fmaxf(fminf(m1, b1), fmaxf(m2, b2));
      m1 = fmaxf(m1, b1);
    }
    const float score = gs >= 2 ? m1 + m2 : m1;
    // lane g takes group g's score
    const float mine = __shfl_sync(0xffffffffu, score, (lane * per) & 31);
    uint32_t gkey[1] = {lane < a.n_group ? ordered(mine) : 0u};
    const int picked = best_k<1>(gkey, a.topk_group, lane);
    const uint32_t allowed = __reduce_or_sync(0xffffffffu, lane < a.topk_group && picked >= 0 ? 1u << (picked & 31) : 0u);
    const float inv_gs = 1.0f / static_cast<float>(gs);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      // (e + 0.5) / gs is at least 1 / 2048 from every integer: its float is on the same side
      const int e = lane + 32 * i, eg = static_cast<int>((static_cast<float>(e) + 0.5f) * inv_gs);
      if (e < a.E && !(allowed >> (eg & 31) & 1u)) key[i] = 0;
    }
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) scratch[lane + 32 * i] = val[i];
  const int id = best_k<EPL>(key, a.k, lane);
  __syncwarp();
  float v = 0.f;
  if (lane < a.k && id >= 0) v = scratch[id] * inv_z;
  float total = v;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane < a.k) {
    const float inv = a.renormalize ? (total > 0.f ? 1.0f / total : 0.f) : 1.0f;
    ids[t * a.k + lane] = id;
    w[t * a.k + lane] = (v * inv) * a.scale;
  }
}

// The gate (warps 0 .. T - 1, one token each), while the other warps run
// `meanwhile`; then the routing tables.
template <int EPL, typename Fn>
__device__ __forceinline__ void route(const GateArgs& gate, const FewArgs& a, Routing& r, Weights weight, float* scratch,
                                      Fn&& meanwhile) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < a.T) {
    gate_one<EPL>(gate, warp, lane, scratch + warp * (32 * EPL), r.ids, r.w);
    // (a NaN bias can leave the gate without a choice)
    if (blockIdx.x == 0 && lane < a.k && r.ids[warp * a.k + lane] < 0)
      record_error(a.err, kErrBadIndex, static_cast<uint32_t>(warp * a.k + lane));
  } else {
    meanwhile();
  }
  build_routing(r, a, weight);
}

// Part of K of warp w, as step w' of kWarps: where 16 does not divide the steps
// the longer parts are spread over the SM's four sub-partitions.
__device__ __forceinline__ int part_of(int warp) { return (warp & ~3) + ((warp + (warp >> 2)) & 3); }

// ------------------------------------------------------------------- up

template <int FMT, int EPL>
__global__ void __launch_bounds__(kThreads, 1) few_up_kernel(GateArgs gate, FewArgs a, int depth, int reds) {
  extern __shared__ __align__(128) uint8_t few_smem[];
  using F = Fmt<FMT>;
  constexpr bool kCorrect = FMT == kW_INT4;  // offsets are taken off the products
  Routing& r = *reinterpret_cast<Routing*>(few_smem);
  float* red = reinterpret_cast<float*>(few_smem + kRoutingBytes);  // [reds][warp][gate, up][16 rows][token]
  float* xsum = red + reds * (kRedBytes / 4);                       // int4: [group][token] sums of x
  uint8_t* xs = reinterpret_cast<uint8_t*>(xsum) + (kCorrect ? a.H / 128 * 32 : 0);
  const int xstride = token_stride(a.H);
  uint8_t* rings = xs + (static_cast<size_t>(a.T) * xstride + 127) / 128 * 128;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  // While the kernel before still runs: what the gate reads towards L2 (a hint
  // only: nothing is read before the wait)
  if (blockIdx.x == 0) {
    for (int i = tid * 32; i < a.T * a.E; i += kThreads * 32) prefetch_l2(gate.logits + i);
    if (gate.bias != nullptr)
      for (int i = tid * 32; i < a.E; i += kThreads * 32) prefetch_l2(gate.bias + i);
    for (int i = tid * 64; i < a.T * a.H; i += kThreads * 64) prefetch_l2(a.x + i);
  }
  pdl_wait();
  pdl_trigger();

  // tokens into shared memory in fragment order; fp8: as codes of x / a1
  const uint4* xg = reinterpret_cast<const uint4*>(a.x);
  const int nvec = a.T * a.H / 8;
  auto stage = [&](int t0, int n, float a1) {
    for (int c = tid - t0; c - lane < a.H / 8; c += n) {
      const bool live = c < a.H / 8;
      const int k = c * 8;
#pragma unroll 1
      for (int t0 = 0; t0 < a.T; t0 += 4) {
        uint4 vs[4];  // four tokens' loads in flight
#pragma unroll
        for (int u = 0; u < 4; ++u)
          vs[u] = live && t0 + u < a.T ? xg[static_cast<size_t>(t0 + u) * (a.H / 8) + c] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int t = t0 + u;
          if (t >= a.T) break;
          uint4 v = vs[u];
          if (kCorrect) {  // a group of 128 is 16 adjacent lanes
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += bf16_lo(word(v, j)) + bf16_hi(word(v, j));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (live && (lane & 15) == 0) xsum[k / 128 * 8 + t] = sum;
          }
          if (FMT == kW_FP8) {
            uint32_t q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              q[j] = quantised_f16x2(__fdiv_rn(bf16_lo(word(v, j)), a1), __fdiv_rn(bf16_hi(word(v, j)), a1));
            v = make_uint4(q[0], q[1], q[2], q[3]);
          } else if (FMT == kW_INT4 && !a.paired) {
            v = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                           __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
          }
          if (live) *reinterpret_cast<uint4*>(xs + static_cast<size_t>(t) * xstride + 2 * frag_pos<FMT>(k, 0)) = v;
        }
      }
    }
  };
  const bool dynamic = FMT == kW_FP8 && a.a1 == nullptr;
  float a1 = FMT == kW_FP8 && !dynamic ? a.a1[0] : 1.f;
  if (kCorrect) {
    for (int i = tid; i < a.H / 128 * 8; i += kThreads)
      if ((i & 7) >= a.T) xsum[i] = 0.f;
  }
  route<EPL>(gate, a, r, nullptr, reinterpret_cast<float*>(rings), [&] {
    if (!dynamic) stage(32 * a.T, kThreads - 32 * a.T, a1);
  });
  if (dynamic) {
    float m = 0.f;
    for (int i = tid; i < nvec; i += kThreads) {
      const uint4 v = xg[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(fabsf(bf16_lo(word(v, j))), fabsf(bf16_hi(word(v, j)))));
    }
    a1 = act_scale_of(block_max(m, red));
    stage(0, kThreads, a1);
    __syncthreads();
  }

  constexpr int STEP = F::KC;  // K of a step
  constexpr int kStage = up_stage<FMT>();
  const int tiles = a.I / 16, count = r.count;
  const int nsteps = a.H / STEP;
  const int part_no = part_of(warp);
  const int s0 = nsteps * part_no / kWarps, s1 = nsteps * (part_no + 1) / kWarps;
  const uint32_t ring = smem_u32(rings) + static_cast<uint32_t>(warp * depth * kStage);
  const int64_t rb = row_bytes<FMT>(a.H), to8 = 8 * rb, to_up = a.I * rb;
  const int G = a.H / 128;
  const bool zero = a.w13_zero != nullptr;
  const uint8_t* w13 = static_cast<const uint8_t*>(a.w13);

  // issue side: its unit (expert ix, tile it), step is, pointers of the step
  int ix = static_cast<int>(blockIdx.x) / tiles, it = static_cast<int>(blockIdx.x) % tiles, is = s0;
  uint32_t idst = ring + lane * 16;
  const uint32_t wpos = static_cast<uint32_t>(2048 - lane * 16 + (lane & 7) * 16 + (lane >> 3) * 4);
  const uint32_t iend = ring + static_cast<uint32_t>(depth * kStage);
  const uint8_t* isrc = nullptr;
  // addresses of row `lane`'s scale and zero point (16 gate rows, 16 up rows)
  uint64_t isc = 0, izp = 0;
  auto start_unit = [&] {
    const int64_t row = static_cast<int64_t>(r.expert[ix]) * 2 * a.I + it * 16;
    isrc = w13 + (row + g) * rb + row_bytes<FMT>(static_cast<int64_t>(s0) * STEP) + t4 * 16;
    if (kGrouped<FMT>) {
      const int64_t at = (row + (lane & 15) + static_cast<int64_t>(lane >> 4) * a.I) * G + s0 * STEP / 128;
      isc = reinterpret_cast<uint64_t>(a.w13_scale) + 2 * at;
      izp = reinterpret_cast<uint64_t>(a.w13_zero) + at;
    }
    is = s0;
  };
  bool more = ix < count && s0 < s1;
  if (more) start_unit();
  auto issue = [&] {
    if (more) {
      cp_async16(idst, isrc);  // gate rows g and g + 8, up rows g and g + 8
      cp_async16(idst + 512, isrc + to8);
      cp_async16(idst + 1024, isrc + to_up);
      cp_async16(idst + 1536, isrc + to_up + to8);
      if (kGrouped<FMT>) {
        // the 4-byte words that hold row `lane`'s scale and zero point
        cp_async4(idst + wpos, reinterpret_cast<const void*>(isc & ~3ull));
        if (zero) cp_async4(idst + wpos + 128, reinterpret_cast<const void*>(izp & ~3ull));
        if (STEP == 128 || (is & 1)) {
          isc += 2;
          izp += 1;
        }
      }
      isrc += 64;
      if (++is == s1) {
        it += gridDim.x;
        while (it >= tiles) {
          it -= tiles;
          ++ix;
        }
        more = ix < count;
        if (more) start_unit();
      }
    }
    cp_async_commit();
    idst += kStage;
    if (idst >= iend) idst -= static_cast<uint32_t>(depth * kStage);
  };
  for (int i = 0; i < depth - 1; ++i) issue();

  uint32_t src = ring;
  float amax = 0.f;
  int buf = 0;
  int x = static_cast<int>(blockIdx.x) / tiles, tile = static_cast<int>(blockIdx.x) % tiles;
  // (columns past the last token repeat it; nobody reads their sums)
  const uint8_t* xlane = xs + static_cast<size_t>(min(g, a.T - 1)) * xstride + t4 * 16;
  while (x < count) {
    const int i0 = tile * 16;
    float acc[2][4] = {};
    for (int s = s0; s < s1; ++s) {
      __syncwarp();
      issue();
      cp_async_wait(depth - 1);
      __syncwarp();
      float sc[4];
      Offset off[4] = {};
      float part[2][4];
      const int group = s * STEP / 128;
      if (kGrouped<FMT>) {
        const uint4 sw = lds128(src + 2048 + g * 16);  // rows g, g + 8 (gate), g, g + 8 (up)
        uint4 zw = make_uint4(0, 0, 0, 0);
        if (zero) zw = lds128(src + 2176 + g * 16);
        const Place at(static_cast<uint32_t>(g * G + group));
#pragma unroll
        for (int q = 0; q < 4; ++q) group_of<FMT>(word(sw, q), word(zw, q), at, zero, sc[q], off[q]);
      }
      uint4 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = lds128(src + static_cast<uint32_t>(q * 512 + lane * 16));
#pragma unroll
      for (int n = 0; n < F::NS; ++n) {
        const uint4 b = *reinterpret_cast<const uint4*>(xlane + 2 * s * F::KC + n * 64);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int m = 2 * n + h;
          const uint32_t b0 = h ? b.z : b.x, b1 = h ? b.w : b.y;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t r0, r1, r2, r3;
            convert<FMT, !kCorrect>(w[2 * y], m, off[2 * y], r0, r2);
            convert<FMT, !kCorrect>(w[2 * y + 1], m, off[2 * y + 1], r1, r3);
            if (kGrouped<FMT> && m == 0) mma16816_first<false>(part[y], r0, r1, r2, r3, b0, b1);
            else mma16816<FMT == kW_FP8>(kGrouped<FMT> ? part[y] : acc[y], r0, r1, r2, r3, b0, b1);
          }
        }
      }
      if (kGrouped<FMT>) {
        float2 xv = make_float2(0.f, 0.f);
        if (kCorrect) xv = *reinterpret_cast<const float2*>(xsum + group * 8 + 2 * t4);
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int q = 2 * y + (j >> 1);
            if (kCorrect) part[y][j] = fmaf(-off[q].plus, j & 1 ? xv.y : xv.x, part[y][j]);
            acc[y][j] = fmaf(part[y][j], sc[q], acc[y][j]);
          }
      }
      src += kStage;
      if (src >= iend) src -= static_cast<uint32_t>(depth * kStage);
    }
    // Join the warps' sums: thread (row, token, gate or up) of the first eight
    // warps.  With two buffers the other warps go on to the next unit.
    float* rd = red + buf * (kRedBytes / 4);
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int j = 0; j < 4; j += 2)
        *reinterpret_cast<float2*>(rd + warp * kRedWarp + y * kRedHalf + (g + 4 * j) * 8 + 2 * t4) =
            make_float2(acc[y][j], acc[y][j + 1]);
    __syncthreads();
    if (tid < 256) {
      const int half = tid & 1, t = (tid >> 1) & 7, i = tid >> 4;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += rd[w * kRedWarp + half * kRedHalf + i * 8 + t];
      float up = __shfl_xor_sync(0xffffffffu, v, 1);
      if (!half && t < a.T && (r.tokens[x] >> t & 1)) {
        if (FMT == kW_FP8) {
          const float s = a1 * static_cast<const float*>(a.w13_scale)[r.expert[x]];
          v *= s;
          up *= s;
        }
        // (to about 16 bits, as it is kept: the fast exponential is off by |v| * 2^-23)
        const float act = __fdividef(v, 1.0f + __expf(-v)) * up;
        uint16_t* dst = a.act + static_cast<size_t>(r.slot[x][t]) * 2 * a.I + frag_pos<FMT>(i0 + i, !a.paired);
        if (FMT == kW_FP8 && a.a2 != nullptr) {
          dst[0] = static_cast<uint16_t>(quantised_f16x2(__fdiv_rn(act, a.a2[0]), 0.f));
        } else if (FMT == kW_FP8) {  // the float's halves: quantised once the largest is known
          dst[0] = static_cast<uint16_t>(__float_as_uint(act) >> 16);
          dst[a.I] = static_cast<uint16_t>(__float_as_uint(act));
          amax = fmaxf(amax, fabsf(act));
        } else {
          const __nv_bfloat16 hi = __float2bfloat16_rn(act);
          dst[0] = __bfloat16_as_ushort(hi);
          dst[a.I] = __bfloat16_as_ushort(__float2bfloat16_rn(act - __bfloat162float(hi)));
        }
      }
    }
    if (reds == 2) buf ^= 1;
    else __syncthreads();
    tile += gridDim.x;
    while (tile >= tiles) {
      tile -= tiles;
      ++x;
    }
  }
  if (FMT == kW_FP8 && a.a2 == nullptr) {
    amax = block_max(amax, red);
    if (tid == 0) a.amax[blockIdx.x] = amax;
  }
}

// ----------------------------------------------------------------- down

// bytes of a stage: weights, scales and zero points, and the activations of up
// to `tokens` tokens (two 16-bit halves)
template <int FMT>
__host__ __device__ constexpr int down_stage(int tokens) {
  return Fmt<FMT>::DOWN * 1024 + (kGrouped<FMT> ? 128 : 0) + tokens * Fmt<FMT>::DOWN * Fmt<FMT>::KC * 4;
}

template <int FMT, int EPL>
__global__ void __launch_bounds__(kThreads, 1) few_down_kernel(GateArgs gate, FewArgs a, int up_ctas, int ring_bytes) {
  extern __shared__ __align__(128) uint8_t few_smem[];
  using F = Fmt<FMT>;
  Routing& r = *reinterpret_cast<Routing*>(few_smem);
  float* red = reinterpret_cast<float*>(few_smem + kRoutingBytes);  // [2][warp][16 rows][token]
  Weights weight = reinterpret_cast<Weights>(few_smem + kRoutingBytes + kDownRedBytes);
  uint8_t* rings = few_smem + kRoutingBytes + kDownRedBytes + kWeightBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;

  // Before the first kernel is waited for: the gate once more and the first
  // weights.  (It lets this one start when its own CTAs have passed their wait,
  // so the scores and weights, which precede it, are there.)
  route<EPL>(gate, a, r, weight, reinterpret_cast<float*>(rings), [] {});

  constexpr int STEP = F::KC * F::DOWN;
  constexpr int kActs = F::DOWN * 1024 + (kGrouped<FMT> ? 128 : 0);
  constexpr int kTok = F::DOWN * F::KC * 4;  // a token's activations in a stage
  const int stage = down_stage<FMT>(r.most);
  const int depth = min(kMaxDepth, ring_bytes / (kWarps * stage));
  const int per = a.I / STEP;  // steps of an expert
  const int nsteps = r.count * per;
  const int part_no = part_of(warp);
  const int s0 = static_cast<int>(static_cast<int64_t>(nsteps) * part_no / kWarps);
  const int s1 = static_cast<int>(static_cast<int64_t>(nsteps) * (part_no + 1) / kWarps);
  const uint32_t ring = smem_u32(rings) + static_cast<uint32_t>(warp * depth * stage);
  const uint32_t iend = ring + static_cast<uint32_t>(depth * stage);
  const int64_t rb = row_bytes<FMT>(a.I), to8 = 8 * rb;
  const int G = a.I / 128;
  const bool zero = a.w2_zero != nullptr;
  const bool dynamic = FMT == kW_FP8 && a.a2 == nullptr;
  const bool both = FMT != kW_FP8 || dynamic;  // two halves of an activation
  const int units = a.H / 16;
  const int x0 = s0 / per, c0 = s0 - x0 * per;  // where this warp's part begins

  // Where a stage holds the activations of this lane's token: one place for each
  // token that chose the expert (a lane whose token did not reads the last one,
  // and its sums are left out).
  auto place_of = [&](uint32_t mask) {
    const int at = min(__popc(mask & ((1u << g) - 1u)), __popc(mask) - 1);
    return kActs + static_cast<uint32_t>(at * kTok + t4 * 16);
  };
  struct Cursor {  // of the issue side
    int unit, left, x, c;       // unit, steps left of the part, expert, its step
    uint32_t dst;
    const uint8_t* w;           // weights of the step, row g
    const uint16_t* act;        // this lane's token, or null
    uint32_t place;             // where its activations go in a stage
    uint64_t sc, zp;            // row `lane`'s scale and zero point
  };
  auto start_expert = [&](Cursor& c) {
    const int64_t row = static_cast<int64_t>(r.expert[c.x]) * a.H + c.unit * 16;
    c.w = static_cast<const uint8_t*>(a.w2) + (row + g) * rb + row_bytes<FMT>(c.c * STEP) + t4 * 16;
    if (kGrouped<FMT>) {
      const int64_t at = (row + (lane & 15)) * G + c.c;
      c.sc = reinterpret_cast<uint64_t>(a.w2_scale) + 2 * at;
      c.zp = reinterpret_cast<uint64_t>(a.w2_zero) + at;
    }
    const uint32_t mask = r.tokens[c.x];
    c.act = (mask >> g & 1) ? a.act + static_cast<size_t>(r.slot[c.x][g]) * 2 * a.I + c.c * STEP + t4 * 8 : nullptr;
    c.place = place_of(mask);
  };
  auto start_unit = [&](Cursor& c) {
    c.left = s1 - s0;
    c.x = x0;
    c.c = c0;
    if (c.left > 0 && c.unit < units) start_expert(c);
    else c.unit = units;
  };
  auto issue = [&](Cursor& c, bool weights, bool acts) {
    if (c.unit < units) {
      if (weights) {
#pragma unroll
        for (int u = 0; u < F::DOWN; ++u) {
          cp_async16(c.dst + u * 1024 + lane * 16, c.w + u * 64);
          cp_async16(c.dst + u * 1024 + 512 + lane * 16, c.w + u * 64 + to8);
        }
        if (kGrouped<FMT> && lane < 16) {
          const uint32_t d = c.dst + F::DOWN * 1024 + (lane & 7) * 8 + (lane >> 3) * 4;
          cp_async4(d, reinterpret_cast<const void*>(c.sc & ~3ull));
          if (zero) cp_async4(d + 64, reinterpret_cast<const void*>(c.zp & ~3ull));
        }
      }
      if (acts && c.act != nullptr) {
        // this lane's token: its slices of both halves
        const uint32_t d = c.dst + c.place;
#pragma unroll
        for (int n = 0; n < F::DOWN * F::NS; ++n) {
          cp_async16(d + n * 64, c.act + n * 32);
          if (both) cp_async16(d + kTok / 2 + n * 64, c.act + a.I + n * 32);
        }
      }
      c.w += F::DOWN * 64;
      if (kGrouped<FMT>) {
        c.sc += 2;
        c.zp += 1;
      }
      if (c.act != nullptr) c.act += STEP;
      ++c.c;
      if (--c.left == 0) {
        c.unit += gridDim.x;
        start_unit(c);
      } else if (c.c == per) {
        c.c = 0;
        ++c.x;
        start_expert(c);
      }
    }
    c.dst += stage;
    if (c.dst >= iend) c.dst -= static_cast<uint32_t>(depth * stage);
  };
  static_assert(!kGrouped<FMT> || STEP == 128, "a step is a group");
  Cursor cur;
  cur.unit = blockIdx.x;
  cur.dst = ring;
  start_unit(cur);
  {
    Cursor early = cur;
    for (int i = 0; i < depth - 1; ++i) issue(early, true, false);
  }
  pdl_wait();
  pdl_trigger();
  for (int i = 0; i < depth - 1; ++i) {
    issue(cur, false, true);
    cp_async_commit();
  }
  float a2 = 1.f;
  if (FMT == kW_FP8) {
    if (dynamic) {
      float m = 0.f;
      for (int i = tid; i < up_ctas; i += kThreads) m = fmaxf(m, a.amax[i]);
      a2 = act_scale_of(block_max(m, red));
    } else {
      a2 = a.a2[0];
    }
    // the experts' scales go with the weights of the sum; a2 follows it, because its
    // product with a scale may be too small for a float where the sum's is not
    for (int i = tid; i < r.count * kFewMaxTokens; i += kThreads)
      (&weight[0][0])[i] *= static_cast<const float*>(a.w2_scale)[r.expert[i / kFewMaxTokens]];
    __syncthreads();
  }
  // act / a2 by the reciprocal, which is within the quotient's last bits (an IEEE
  // division per value: Qwen2 fp8, one token 69 us, eight 326; the reciprocal 51 and
  // 227); of a scale so small that it would overflow, with both sides times 2^64 (in a
  // step of its own below: as part of every value's product 52 and 234)
  const bool tiny = a2 < 0x1p-64f;
  const float rs = __fdiv_rn(1.0f, tiny ? a2 * 0x1p64f : a2);

  uint32_t src = ring;
  int buf = 0;
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    float acc[4] = {};
    float part[2][4] = {};  // of the activations' two halves
    int x = x0, c = c0;
    for (int s = s0; s < s1; c = 0, ++x) {
      const int from = s, end = min(s1, s + per - c);  // of this expert's part
      const uint32_t mask = r.tokens[x];
      const uint32_t place = place_of(mask);
      const bool use0 = mask >> (2 * t4) & 1, use1 = mask >> (2 * t4 + 1) & 1;
      const float2 wt = *reinterpret_cast<const float2*>(&weight[x][2 * t4]);
      auto join = [&](const float (&sc)[2]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j & 1 ? use1 : use0) acc[j] = fmaf(part[0][j] + part[1][j], sc[j >> 1] * (j & 1 ? wt.y : wt.x), acc[j]);
          if (!kGrouped<FMT>) part[0][j] = part[1][j] = 0.f;
        }
      };
      for (; s < end; ++s) {
        __syncwarp();
        issue(cur, true, true);
        cp_async_commit();
        cp_async_wait(depth - 1);
        __syncwarp();
        float sc[2] = {1.f, 1.f};
        Offset off[2] = {};
        if (kGrouped<FMT>) {
          const uint2 sw = lds64(src + F::DOWN * 1024 + g * 8);  // rows g, g + 8
          uint2 zw = make_uint2(0, 0);
          if (zero) zw = lds64(src + F::DOWN * 1024 + 64 + g * 8);
          const Place at(static_cast<uint32_t>(g * G + c + s - from));
#pragma unroll
          for (int q = 0; q < 2; ++q) group_of<FMT>(q ? sw.y : sw.x, q ? zw.y : zw.x, at, zero, sc[q], off[q]);
        }
#pragma unroll
        for (int u = 0; u < F::DOWN; ++u) {
          uint4 w[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) w[q] = lds128(src + static_cast<uint32_t>((2 * u + q) * 512 + lane * 16));
#pragma unroll
          for (int n = 0; n < F::NS; ++n) {
            uint4 hi = lds128(src + place + (u * F::NS + n) * 64), lo = make_uint4(0, 0, 0, 0);
            if (both) lo = lds128(src + place + kTok / 2 + (u * F::NS + n) * 64);
            if (dynamic) {
              auto q2 = [&](uint32_t h, uint32_t l) {
                float v0 = __uint_as_float(__byte_perm(l, h, 0x5410)), v1 = __uint_as_float(__byte_perm(l, h, 0x7632));
                return quantised_f16x2(v0 * rs, v1 * rs);
              };
              if (tiny) {
                auto up = [](uint32_t& h, uint32_t& l) {
                  const uint32_t v0 = __float_as_uint(__uint_as_float(__byte_perm(l, h, 0x5410)) * 0x1p64f);
                  const uint32_t v1 = __float_as_uint(__uint_as_float(__byte_perm(l, h, 0x7632)) * 0x1p64f);
                  l = __byte_perm(v0, v1, 0x5410);
                  h = __byte_perm(v0, v1, 0x7632);
                };
                up(hi.x, lo.x);
                up(hi.y, lo.y);
                up(hi.z, lo.z);
                up(hi.w, lo.w);
              }
              hi = make_uint4(q2(hi.x, lo.x), q2(hi.y, lo.y), q2(hi.z, lo.z), q2(hi.w, lo.w));
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t r0, r1, r2, r3;
              convert<FMT, true>(w[0], 2 * n + h, off[0], r0, r2);
              convert<FMT, true>(w[1], 2 * n + h, off[1], r1, r3);
              const uint32_t b0 = h ? hi.z : hi.x, b1 = h ? hi.w : hi.y, l0 = h ? lo.z : lo.x, l1 = h ? lo.w : lo.y;
              if (FMT == kW_FP8) {
                mma16816<true>(part[h], r0, r1, r2, r3, b0, b1);
              } else if (kGrouped<FMT> && u == 0 && n == 0 && h == 0) {
                mma16816_first<false>(part[0], r0, r1, r2, r3, b0, b1);
                mma16816_first<false>(part[1], r0, r1, r2, r3, l0, l1);
              } else {
                mma16816<false>(part[0], r0, r1, r2, r3, b0, b1);
                mma16816<false>(part[1], r0, r1, r2, r3, l0, l1);
              }
            }
          }
        }
        if (kGrouped<FMT>) join(sc);  // the group's scales
        src += stage;
        if (src >= iend) src -= static_cast<uint32_t>(depth * stage);
      }
      if (!kGrouped<FMT>) {
        const float one[2] = {1.f, 1.f};
        join(one);
      }
    }
    float* rd = red + buf * (kWarps * 128);
    buf ^= 1;
#pragma unroll
    for (int j = 0; j < 4; j += 2)
      *reinterpret_cast<float2*>(rd + (warp * 16 + g + 4 * j) * 8 + 2 * t4) = make_float2(acc[j], acc[j + 1]);
    __syncthreads();
    if (tid < 128) {
      const int row = tid & 15, t = tid >> 4;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += rd[(w * 16 + row) * 8 + t];
      if (t < a.T) a.out[static_cast<size_t>(t) * a.H + unit * 16 + row] = __float2bfloat16_rn(FMT == kW_FP8 ? v * a2 : v);
    }
  }
}

constexpr size_t kMaxSmem = 232448;

template <typename K>
cudaError_t allow_smem(K kernel, int* configured) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64 || configured[dev] == 0) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxSmem));
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  return cudaSuccess;
}

template <int FMT, int EPL>
cudaError_t launch_both(const GateArgs& g, const FewArgs& a, int sms, cudaStream_t s) {
  static int configured_up[64] = {}, configured_down[64] = {};
  cudaError_t err = allow_smem(few_up_kernel<FMT, EPL>, configured_up);
  if (err == cudaSuccess) err = allow_smem(few_down_kernel<FMT, EPL>, configured_down);
  if (err != cudaSuccess) return err;
  const size_t gate = static_cast<size_t>(a.T) * 32 * EPL * 4;
  const size_t tokens = (static_cast<size_t>(a.T) * token_stride(a.H) + 127) / 128 * 128;
  const size_t sums = FMT == kW_INT4 ? static_cast<size_t>(a.H) / 128 * 32 : 0;
  const size_t stage = static_cast<size_t>(kWarps) * up_stage<FMT>();
  // a second reduction buffer where it leaves four stages
  const int reds = kRoutingBytes + 2 * kRedBytes + sums + tokens + 4 * stage <= kMaxSmem ? 2 : 1;
  const size_t fixed = kRoutingBytes + reds * kRedBytes + sums + tokens;
  if (fixed + 2 * stage > kMaxSmem) return cudaErrorInvalidValue;  // (refused before, by the limits asserted below)
  const int depth = static_cast<int>(std::min<size_t>(kMaxDepth, (kMaxSmem - fixed) / stage));
  const int up_grid = std::min(sms, std::min(a.E, a.T * a.k) * (a.I / 16));
  err = launch_pdl(few_up_kernel<FMT, EPL>, dim3(up_grid), dim3(kThreads), fixed + std::max(depth * stage, gate), s, g,
                   a, depth, reds);
  if (err != cudaSuccess) return err;
  constexpr size_t down_fixed = kRoutingBytes + kDownRedBytes + kWeightBytes;
  static_assert(kWarps * 2 * down_stage<FMT>(kFewMaxTokens) + down_fixed <= kMaxSmem,
                "two stages a warp for every routing");
  return launch_pdl(few_down_kernel<FMT, EPL>, dim3(std::min(sms, a.H / 16)), dim3(kThreads), kMaxSmem, s, g, a,
                    up_grid, static_cast<int>(kMaxSmem - down_fixed));
}

template <int FMT>
cudaError_t launch_gate_width(const GateArgs& g, const FewArgs& a, int sms, cudaStream_t s) {
  if (a.E <= 64) return launch_both<FMT, 2>(g, a, sms, s);
  if (a.E <= 256) return launch_both<FMT, 8>(g, a, sms, s);
  return launch_both<FMT, 32>(g, a, sms, s);
}

}  // namespace

// (a token's row takes 2 * (H + 32) bytes, all of them rounded up to 128; int4's sums H / 4)
static_assert(kRoutingBytes + kRedBytes + 2 * static_cast<size_t>(kFewMaxTokenValues) + 127 +
                      2 * kWarps * std::max(up_stage<kW_INT8>(), std::max(up_stage<kW_BF16>(), up_stage<kW_FP8>())) <=
                  kMaxSmem,
              "two stages a warp beside the most tokens");
static_assert(kRoutingBytes + kRedBytes + 2 * static_cast<size_t>(kFewMaxInt4Values) + 64 +
                      2 * kWarps * up_stage<kW_INT4>() <=
                  kMaxSmem,
              "two stages a warp beside the most tokens and their sums (rows of a multiple of 64 bytes)");

cudaError_t launch_few(const GateArgs& g, const FewArgs& a, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  switch (a.wkind) {
    case kW_BF16: return launch_gate_width<kW_BF16>(g, a, di.sms, s);
    case kW_FP8: return launch_gate_width<kW_FP8>(g, a, di.sms, s);
    case kW_INT8: return launch_gate_width<kW_INT8>(g, a, di.sms, s);
    default: return launch_gate_width<kW_INT4>(g, a, di.sms, s);
  }
}

}  // namespace moe
