// The MoE layer for a few tokens (moe_forward_few), in two launches.
//   up:   act[t, j, i] = silu(w13[e, i] . x[t]) (w13[e, I + i] . x[t]), e = ids[t, j]
//   down: out[t, h]    = sum_j w[t, j] (w2[e, h] . act[t, j])
// With at most 8 tokens the chosen experts' weights are read once and nothing
// else is large, so the layer is bound by the rate at which the weights stream
// in (int4: nearly by the integer work that unpacks them, see convert()).
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
// bits: as a bf16 and the bf16 of what that left over (two MMAs), or for fp8
// as the format's codes.
#include "gate_token.cuh"

namespace moe {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxSlots = kFewMaxTokens * gate_detail::kMaxTopK;
constexpr int kMaxDepth = 8;

// K per lane load of 16 bytes by four lanes, 16-byte slices of a token's
// fragment per load, and loads per step of the two kernels.  A step lies within
// one scale group of 128 (int4, int8).
template <int FMT>
struct Fmt;
template <>
struct Fmt<kW_BF16> {
  static constexpr int KC = 32, NS = 1, UP = 1, DOWN = 2;
};
template <>
struct Fmt<kW_FP8> {
  static constexpr int KC = 64, NS = 2, UP = 1, DOWN = 2;
};
template <>
struct Fmt<kW_INT8> {
  static constexpr int KC = 64, NS = 2, UP = 1, DOWN = 2;
};
template <>
struct Fmt<kW_INT4> {
  static constexpr int KC = 128, NS = 4, UP = 1, DOWN = 1;
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest n groups have landed
__device__ __forceinline__ void cp_async_wait(int n) {
  switch (n) {
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    case 7: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
  }
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
  return r;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// What a lane needs to turn codes into integers: flip is xored into the codes
// (signed ones become offset ones), then the offset is subtracted (one per row:
// the zero point, or the sign's offset).
struct Offset {
  uint32_t flip;
  uint32_t pair;   // int4: bf16x2 of 128 + offset
  float magic;     // int8: 2^23 + offset
};

// The A registers (one row) of MMA m of a 16-byte load.
//   int4: a nibble in the low bits of the bf16 128.0 is 128 + code; a pair of
//     them is one shift, one masked xor and one exact subtraction (1.4
//     operations a code)
//   int8: a byte in the low bits of the float 2^23 is 2^23 + code
//   fp8: the converter's f16 pairs
template <int FMT>
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
    uint32_t a = (v & 0x000F000Fu) ^ o.flip, b = ((v >> 4) & 0x000F000Fu) ^ o.flip;
    const __nv_bfloat162 off = *reinterpret_cast<const __nv_bfloat162*>(&o.pair);
    __nv_bfloat162 pa = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), off);
    __nv_bfloat162 pb = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&b), off);
    lo = *reinterpret_cast<uint32_t*>(&pa);
    hi = *reinterpret_cast<uint32_t*>(&pb);
  }
}

// Scale and offset of one row's group, from the copied words that hold them.
template <int FMT>
__device__ __forceinline__ void group_of(uint32_t saddr, uint32_t zaddr, int64_t index, bool zero, float& scale,
                                         Offset& o) {
  uint16_t h;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(saddr + 2u * static_cast<uint32_t>(index & 1)) : "memory");
  scale = __half2float(__ushort_as_half(h));
  uint32_t z = FMT == kW_INT4 ? 8u : 128u;
  if (zero)
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(z) : "r"(zaddr + static_cast<uint32_t>(index & 3)) : "memory");
  if (FMT == kW_INT4) {
    o.flip = zero ? 0x43004300u : 0x43084308u;
    o.pair = 0x43004300u | z | (z << 16);
  } else {
    o.flip = zero ? 0u : 0x80808080u;
    o.magic = 8388608.0f + static_cast<float>(z);
  }
}

// What the chosen experts are, in shared memory: the distinct ones in ascending
// order, and for each which of the tokens' slots chose it.
struct Routing {
  int count;
  int32_t ids[kMaxSlots];              // per slot
  float w[kMaxSlots];                  // per slot
  uint32_t seen[32];                   // bit per expert
  int16_t expert[kMaxSlots];
  uint8_t tokens[kMaxSlots];           // bit per token
  int16_t slot[kMaxSlots][kFewMaxTokens];
  int most;                            // tokens of the expert with the most
};
// per chosen expert and token: the weight of the sum, 0 where the token did not choose it
typedef float (*Weights)[kFewMaxTokens];

// From r.ids and r.w; every thread of the CTA.  weight: null where it is not needed.
__device__ __forceinline__ void build_routing(Routing& r, const FewArgs& a, Weights weight) {
  const int S = a.T * a.k;
  if (threadIdx.x == 0) r.most = 1;
  for (int i = threadIdx.x; i < 32; i += kThreads) r.seen[i] = 0;
  if (weight != nullptr)
    for (int i = threadIdx.x; i < S * kFewMaxTokens; i += kThreads) (&weight[0][0])[i] = 0.f;
  for (int i = threadIdx.x; i < (S + 3) / 4; i += kThreads) reinterpret_cast<uint32_t*>(r.tokens)[i] = 0;
  __syncthreads();
  for (int s = threadIdx.x; s < S; s += kThreads) atomicOr(&r.seen[r.ids[s] >> 5], 1u << (r.ids[s] & 31));
  __syncthreads();
  for (int s = threadIdx.x; s < S; s += kThreads) {
    const int e = r.ids[s], t = s / a.k;
    int at = __popc(r.seen[e >> 5] & ((1u << (e & 31)) - 1u));
    for (int i = 0; i < (e >> 5); ++i) at += __popc(r.seen[i]);
    r.expert[at] = static_cast<int16_t>(e);
    r.slot[at][t] = static_cast<int16_t>(s);
    if (weight != nullptr) weight[at][t] = r.w[s];
    atomicOr(reinterpret_cast<uint32_t*>(r.tokens) + (at >> 2), 1u << (8 * (at & 3) + t));
  }
  if (threadIdx.x == 0) {
    int n = 0;
    for (int i = 0; i < 32; ++i) n += __popc(r.seen[i]);
    r.count = n;
  }
  __syncthreads();
  if (threadIdx.x < r.count) atomicMax(&r.most, __popc(r.tokens[threadIdx.x]));
  __syncthreads();
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

__device__ __forceinline__ float act_scale_of(float amax) { return amax > 0.f ? __fdiv_rn(amax, 448.0f) : 1.0f; }

// e4m3 of two values as the f16 pair that they stand for
__device__ __forceinline__ uint32_t quantised_f16x2(float a, float b) { return e4m3x2_f16x2(f32x2_to_e4m3x2(a, b)); }

constexpr size_t kRoutingBytes = (sizeof(Routing) + 127) / 128 * 128;
constexpr size_t kWeightBytes = sizeof(float) * kMaxSlots * kFewMaxTokens;
constexpr size_t kRedBytes = static_cast<size_t>(kWarps) * 32 * 8 * 4;
// row stride of a token in shared memory: 64 bytes over a multiple of 128, so
// that the lanes of two tokens read different banks
__host__ __device__ constexpr int token_stride(int H) { return 2 * H + 64; }

template <int FMT>
constexpr int up_stage() {
  return Fmt<FMT>::UP * 4 * 512 + (kGrouped<FMT> ? 256 : 0);
}

// ------------------------------------------------------------------- up

template <int FMT, int EPL>
__global__ void __launch_bounds__(kThreads, 1) few_up_kernel(GateArgs gate, FewArgs a, int depth) {
  extern __shared__ __align__(128) uint8_t few_smem[];
  using F = Fmt<FMT>;
  Routing& r = *reinterpret_cast<Routing*>(few_smem);
  float* red = reinterpret_cast<float*>(few_smem + kRoutingBytes);  // [warp][row 0-15 gate, 16-31 up][token]
  uint8_t* xs = few_smem + kRoutingBytes + kRedBytes;
  const int xstride = token_stride(a.H);
  uint8_t* rings = xs + (static_cast<size_t>(a.T) * xstride + 127) / 128 * 128;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  pdl_wait();
  pdl_trigger();

  // the gate, one warp per token, with the reduction buffer (up to 4 KB a token
  // would not fit there for E > 512) and rings as its scratch
  {
    GateArgs gl = gate;
    gl.ids = r.ids;
    gl.w = r.w;
    if (warp < a.T) gate_detail::gate_token<EPL>(gl, warp, lane, reinterpret_cast<float*>(rings) + warp * (32 * EPL));
  }
  __syncthreads();
  for (int s = tid; s < a.T * a.k; s += kThreads) {
    // (a NaN bias can leave the gate without a choice)
    if (static_cast<unsigned>(r.ids[s]) >= static_cast<unsigned>(a.E)) {
      if (blockIdx.x == 0) record_error(a.err, kErrBadIndex, static_cast<uint32_t>(s));
      r.ids[s] = 0;
    }
    if (blockIdx.x == 0) {
      a.ids[s] = r.ids[s];
      a.topk_w[s] = r.w[s];
    }
  }
  build_routing(r, a, nullptr);

  // tokens into shared memory in fragment order; fp8: as codes of x / a1
  float a1 = 1.f;
  const uint4* xg = reinterpret_cast<const uint4*>(a.x);
  if (FMT == kW_FP8) {
    if (a.a1 != nullptr) {
      a1 = a.a1[0];
    } else {
      float m = 0.f;
      for (int i = tid; i < a.T * a.H / 8; i += kThreads) {
        const uint4 v = xg[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(fabsf(bf16_lo(word(v, j))), fabsf(bf16_hi(word(v, j)))));
      }
      a1 = act_scale_of(block_max(m, red));
    }
  }
  for (int i = tid; i < a.T * a.H / 8; i += kThreads) {
    const int t = i / (a.H / 8), k = (i - t * (a.H / 8)) * 8;
    uint4 v = xg[i];
    if (FMT == kW_FP8) {
      uint32_t q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        q[j] = quantised_f16x2(__fdiv_rn(bf16_lo(word(v, j)), a1), __fdiv_rn(bf16_hi(word(v, j)), a1));
      v = make_uint4(q[0], q[1], q[2], q[3]);
    } else if (FMT == kW_INT4 && !a.paired) {
      v = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                     __byte_perm(v.y, v.w, 0x7632));
    }
    *reinterpret_cast<uint4*>(xs + static_cast<size_t>(t) * xstride + 2 * frag_pos<FMT>(k, 0)) = v;
  }
  __syncthreads();

  constexpr int STEP = F::KC * F::UP;  // K of a step
  constexpr int kStage = up_stage<FMT>();
  const int tiles = a.I / 16;
  const int units = r.count * tiles;
  const int nsteps = a.H / STEP;
  const int s0 = nsteps * warp / kWarps, s1 = nsteps * (warp + 1) / kWarps;
  const uint32_t ring = smem_u32(rings) + static_cast<uint32_t>(warp * depth * kStage);
  const int64_t rb = row_bytes<FMT>(a.H);
  const int G = a.H / 128;
  const bool zero = a.w13_zero != nullptr;

  // issue side: unit iu, step is
  int iu = blockIdx.x, is = s0, islot = 0;
  auto issue = [&] {
    if (iu < units && s0 < s1) {
      const int x = iu / tiles;
      const int64_t row = static_cast<int64_t>(r.expert[x]) * 2 * a.I + (iu - x * tiles) * 16;
      const uint8_t* src = static_cast<const uint8_t*>(a.w13) + (row + g) * rb + row_bytes<FMT>(static_cast<int64_t>(is) * STEP) + t4 * 16;
      const uint32_t dst = ring + static_cast<uint32_t>(islot * kStage + lane * 16);
#pragma unroll
      for (int u = 0; u < F::UP; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q)  // gate rows g and g + 8, up rows g and g + 8
          cp_async16(dst + static_cast<uint32_t>((4 * u + q) * 512),
                     src + u * 64 + ((q & 1) * 8 + static_cast<int64_t>(q >> 1) * a.I) * rb);
      if (kGrouped<FMT>) {
        // the 4-byte words that hold row `lane`'s scale and zero point
        const int64_t at = (row + (lane & 15) + static_cast<int64_t>(lane >> 4) * a.I) * G + is * STEP / 128;
        const uint32_t d = ring + static_cast<uint32_t>(islot * kStage + F::UP * 2048 + lane * 4);
        cp_async4(d, static_cast<const uint16_t*>(a.w13_scale) + (at & ~1ll));
        if (zero) cp_async4(d + 128, a.w13_zero + (at & ~3ll));
      }
      if (++is == s1) {
        is = s0;
        iu += gridDim.x;
      }
    }
    cp_async_commit();
    if (++islot == depth) islot = 0;
  };
  for (int i = 0; i < depth - 1; ++i) issue();

  int slot = 0;
  float amax = 0.f;
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int x = unit / tiles, i0 = (unit - x * tiles) * 16;
    const int64_t row0 = static_cast<int64_t>(r.expert[x]) * 2 * a.I + i0;
    float acc[2][4] = {};
    for (int s = s0; s < s1; ++s) {
      __syncwarp();
      issue();
      cp_async_wait(depth - 1);
      __syncwarp();
      const uint32_t src = ring + static_cast<uint32_t>(slot * kStage);
      if (++slot == depth) slot = 0;
      float sc[4] = {1.f, 1.f, 1.f, 1.f};
      Offset off[4] = {};
      float part[2][4] = {};
      if (kGrouped<FMT>) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int rr = g + 8 * q;  // gate g, gate g + 8, up g, up g + 8
          const int64_t at = (row0 + (rr & 15) + static_cast<int64_t>(rr >> 4) * a.I) * G + s * STEP / 128;
          group_of<FMT>(src + F::UP * 2048 + rr * 4, src + F::UP * 2048 + 128 + rr * 4, at, zero, sc[q], off[q]);
        }
      }
#pragma unroll
      for (int u = 0; u < F::UP; ++u) {
        uint4 w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = lds128(src + static_cast<uint32_t>((4 * u + q) * 512 + lane * 16));
#pragma unroll
        for (int n = 0; n < F::NS; ++n) {
          uint4 b = make_uint4(0, 0, 0, 0);
          if (g < a.T)
            b = *reinterpret_cast<const uint4*>(xs + static_cast<size_t>(g) * xstride +
                                                2 * ((s * F::UP + u) * F::KC) + n * 64 + t4 * 16);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int m = 2 * n + h;
            const uint32_t b0 = h ? b.z : b.x, b1 = h ? b.w : b.y;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint32_t a0, a1r, a2, a3;
              convert<FMT>(w[2 * y], m, off[2 * y], a0, a2);
              convert<FMT>(w[2 * y + 1], m, off[2 * y + 1], a1r, a3);
              mma16816<FMT == kW_FP8>(kGrouped<FMT> ? part[y] : acc[y], a0, a1r, a2, a3, b0, b1);
            }
          }
        }
      }
      if (kGrouped<FMT>) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[y][j] = fmaf(part[y][j], sc[2 * y + (j >> 1)], acc[y][j]);
      }
    }
    // join the warps' sums: thread (i, token, gate or up)
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int j = 0; j < 4; j += 2)
        *reinterpret_cast<float2*>(red + (warp * 32 + y * 16 + g + 4 * j) * 8 + 2 * t4) =
            make_float2(acc[y][j], acc[y][j + 1]);
    __syncthreads();
    if (tid < 256) {
      const int half = tid >> 7 & 1, i = tid >> 3 & 15, t = tid & 7;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += red[(w * 32 + half * 16 + i) * 8 + t];
      if (half) red[(16 + i) * 8 + t] = v;  // (row of warp 0, read by this thread alone)
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (!half && t < a.T && (r.tokens[x] >> t & 1)) {
        float up = red[(16 + i) * 8 + t];
        if (FMT == kW_FP8) {
          const float s = a1 * static_cast<const float*>(a.w13_scale)[r.expert[x]];
          v *= s;
          up *= s;
        }
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
    __syncthreads();
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

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1) few_down_kernel(FewArgs a, int up_ctas, int ring_bytes) {
  extern __shared__ __align__(128) uint8_t few_smem[];
  using F = Fmt<FMT>;
  Routing& r = *reinterpret_cast<Routing*>(few_smem);
  float* red = reinterpret_cast<float*>(few_smem + kRoutingBytes);  // [warp][16 rows][token]
  Weights weight = reinterpret_cast<Weights>(few_smem + kRoutingBytes + kRedBytes / 2);
  uint8_t* rings = few_smem + kRoutingBytes + kRedBytes / 2 + kWeightBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  pdl_wait();
  pdl_trigger();
  for (int s = tid; s < a.T * a.k; s += kThreads) {
    r.ids[s] = a.ids[s];
    r.w[s] = a.topk_w[s];
  }
  float a2 = 1.f;
  const bool dynamic = FMT == kW_FP8 && a.a2 == nullptr;
  if (FMT == kW_FP8) {
    if (dynamic) {
      float m = 0.f;
      for (int i = tid; i < up_ctas; i += kThreads) m = fmaxf(m, a.amax[i]);
      a2 = act_scale_of(block_max(m, red));
    } else {
      a2 = a.a2[0];
    }
  }
  __syncthreads();
  build_routing(r, a, weight);
  if (FMT == kW_FP8) {  // the experts' scales go with the weights of the sum
    for (int i = tid; i < r.count * kFewMaxTokens; i += kThreads)
      (&weight[0][0])[i] *= a2 * static_cast<const float*>(a.w2_scale)[r.expert[i / kFewMaxTokens]];
    __syncthreads();
  }

  constexpr int STEP = F::KC * F::DOWN;
  const int stage = down_stage<FMT>(r.most);
  const int depth = min(kMaxDepth, ring_bytes / (kWarps * stage));
  const int per = a.I / STEP;  // steps of an expert
  const int nsteps = r.count * per;
  const int s0 = static_cast<int>(static_cast<int64_t>(nsteps) * warp / kWarps);
  const int s1 = static_cast<int>(static_cast<int64_t>(nsteps) * (warp + 1) / kWarps);
  const uint32_t ring = smem_u32(rings) + static_cast<uint32_t>(warp * depth * stage);
  const int64_t rb = row_bytes<FMT>(a.I);
  const int G = a.I / 128;
  const bool zero = a.w2_zero != nullptr;
  constexpr int kActs = F::DOWN * 1024 + (kGrouped<FMT> ? 128 : 0);
  constexpr int kTok = F::DOWN * F::KC * 4;  // a token's activations in a stage
  const float rs = 1.0f / a2;
  const int units = a.H / 16;

  int iu = blockIdx.x, is = s0, islot = 0;
  auto issue = [&] {
    if (iu < units && s0 < s1) {
      const int x = is / per, k0 = (is - x * per) * STEP;
      const int64_t row = static_cast<int64_t>(r.expert[x]) * a.H + iu * 16;
      const uint8_t* src = static_cast<const uint8_t*>(a.w2) + (row + g) * rb + row_bytes<FMT>(k0) + t4 * 16;
      const uint32_t dst = ring + static_cast<uint32_t>(islot * stage);
#pragma unroll
      for (int u = 0; u < F::DOWN; ++u)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          cp_async16(dst + static_cast<uint32_t>((2 * u + q) * 512 + lane * 16), src + u * 64 + q * 8 * rb);
      if (kGrouped<FMT> && lane < 16) {
        const int64_t at = (row + lane) * G + k0 / 128;
        cp_async4(dst + F::DOWN * 1024 + lane * 4, static_cast<const uint16_t*>(a.w2_scale) + (at & ~1ll));
        if (zero) cp_async4(dst + F::DOWN * 1024 + 64 + lane * 4, a.w2_zero + (at & ~3ll));
      }
      const uint32_t mask = r.tokens[x];
      if (mask >> g & 1) {
        // this lane's token: its slices of both halves
        const uint32_t d = dst + kActs + static_cast<uint32_t>(__popc(mask & ((1u << g) - 1u)) * kTok + t4 * 16);
        const uint16_t* act = a.act + static_cast<size_t>(r.slot[x][g]) * 2 * a.I + k0 + t4 * 8;
#pragma unroll
        for (int n = 0; n < F::DOWN * F::NS; ++n) {
          cp_async16(d + n * 64, act + n * 32);
          if (FMT != kW_FP8 || dynamic) cp_async16(d + kTok / 2 + n * 64, act + a.I + n * 32);
        }
      }
      if (++is == s1) {
        is = s0;
        iu += gridDim.x;
      }
    }
    cp_async_commit();
    if (++islot == depth) islot = 0;
  };
  for (int i = 0; i < depth - 1; ++i) issue();

  int slot = 0;
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    float acc[4] = {};
    float part[4] = {};
    for (int s = s0; s < s1; ++s) {
      const int x = s / per, k0 = (s - x * per) * STEP;
      __syncwarp();
      issue();
      cp_async_wait(depth - 1);
      __syncwarp();
      const uint32_t src = ring + static_cast<uint32_t>(slot * stage);
      if (++slot == depth) slot = 0;
      float sc[2] = {1.f, 1.f};
      Offset off[2] = {};
      if (kGrouped<FMT>) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int rr = g + 8 * q;
          const int64_t at = (static_cast<int64_t>(r.expert[x]) * a.H + unit * 16 + rr) * G + k0 / 128;
          group_of<FMT>(src + F::DOWN * 1024 + rr * 4, src + F::DOWN * 1024 + 64 + rr * 4, at, zero, sc[q], off[q]);
        }
      }
      const uint32_t mask = r.tokens[x];
      const bool mine = mask >> g & 1;
      const uint32_t acts = src + kActs + static_cast<uint32_t>(__popc(mask & ((1u << g) - 1u)) * kTok + t4 * 16);
#pragma unroll
      for (int u = 0; u < F::DOWN; ++u) {
        uint4 w[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) w[q] = lds128(src + static_cast<uint32_t>((2 * u + q) * 512 + lane * 16));
#pragma unroll
        for (int n = 0; n < F::NS; ++n) {
          uint4 hi = make_uint4(0, 0, 0, 0), lo = make_uint4(0, 0, 0, 0);
          if (mine) {
            hi = lds128(acts + (u * F::NS + n) * 64);
            if (FMT != kW_FP8 || dynamic) lo = lds128(acts + kTok / 2 + (u * F::NS + n) * 64);
            if (FMT == kW_FP8 && dynamic) {
              auto q2 = [&](uint32_t h, uint32_t l) {
                return quantised_f16x2(__uint_as_float(__byte_perm(l, h, 0x5410)) * rs,
                                       __uint_as_float(__byte_perm(l, h, 0x7632)) * rs);
              };
              hi = make_uint4(q2(hi.x, lo.x), q2(hi.y, lo.y), q2(hi.z, lo.z), q2(hi.w, lo.w));
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t a0, a1, a2r, a3;
            convert<FMT>(w[0], 2 * n + h, off[0], a0, a2r);
            convert<FMT>(w[1], 2 * n + h, off[1], a1, a3);
            mma16816<FMT == kW_FP8>(part, a0, a1, a2r, a3, h ? hi.z : hi.x, h ? hi.w : hi.y);
            if (FMT != kW_FP8) mma16816<false>(part, a0, a1, a2r, a3, h ? lo.z : lo.x, h ? lo.w : lo.y);
          }
        }
      }
      // the group's or expert's end: times the row's scale and the tokens' weights
      if (kGrouped<FMT> || s + 1 == s1 || (s + 1) / per != x) {
        const float w0 = weight[x][2 * t4], w1 = weight[x][2 * t4 + 1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[j] = fmaf(part[j], sc[j >> 1] * (j & 1 ? w1 : w0), acc[j]);
          part[j] = 0.f;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; j += 2)
      *reinterpret_cast<float2*>(red + (warp * 16 + g + 4 * j) * 8 + 2 * t4) = make_float2(acc[j], acc[j + 1]);
    __syncthreads();
    if (tid < 128) {
      const int row = tid & 15, t = tid >> 4;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += red[(w * 16 + row) * 8 + t];
      if (t < a.T) a.out[static_cast<size_t>(t) * a.H + unit * 16 + row] = __float2bfloat16_rn(v);
    }
    __syncthreads();
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
cudaError_t launch_up(const GateArgs& g, const FewArgs& a, int grid, cudaStream_t s) {
  static int configured[64] = {};
  cudaError_t err = allow_smem(few_up_kernel<FMT, EPL>, configured);
  if (err != cudaSuccess) return err;
  const size_t fixed = kRoutingBytes + kRedBytes + (static_cast<size_t>(a.T) * token_stride(a.H) + 127) / 128 * 128;
  const size_t gate = static_cast<size_t>(a.T) * 32 * EPL * 4;
  int depth = static_cast<int>((kMaxSmem - std::min(fixed, kMaxSmem)) / (kWarps * up_stage<FMT>()));
  if (depth > kMaxDepth) depth = kMaxDepth;
  if (depth < 2) return cudaErrorInvalidValue;  // (refused before: kFewMaxTokenValues)
  size_t smem = static_cast<size_t>(depth) * kWarps * up_stage<FMT>();
  smem = fixed + (smem > gate ? smem : gate);
  return launch_pdl(few_up_kernel<FMT, EPL>, dim3(grid), dim3(kThreads), smem, s, g, a, depth);
}

template <int FMT>
cudaError_t launch_both(const GateArgs& g, const FewArgs& a, int sms, cudaStream_t s) {
  const int up_units = std::min(a.E, a.T * a.k) * (a.I / 16);
  const int up_grid = std::min(sms, up_units);
  cudaError_t err = a.E <= 64    ? launch_up<FMT, 2>(g, a, up_grid, s)
                    : a.E <= 256 ? launch_up<FMT, 8>(g, a, up_grid, s)
                                 : launch_up<FMT, 32>(g, a, up_grid, s);
  if (err != cudaSuccess) return err;
  static int configured[64] = {};
  err = allow_smem(few_down_kernel<FMT>, configured);
  if (err != cudaSuccess) return err;
  const size_t fixed = kRoutingBytes + kRedBytes / 2 + kWeightBytes;
  const int ring = static_cast<int>(kMaxSmem - fixed);
  static_assert(kWarps * 2 * down_stage<FMT>(kFewMaxTokens) + kRoutingBytes + kRedBytes / 2 + kWeightBytes <= kMaxSmem,
                "two stages a warp for every routing");
  return launch_pdl(few_down_kernel<FMT>, dim3(std::min(sms, a.H / 16)), dim3(kThreads), kMaxSmem, s, a, up_grid, ring);
}

}  // namespace

static_assert(kRoutingBytes + kRedBytes + 2 * static_cast<size_t>(kFewMaxTokenValues) + 128 +
                      2 * kWarps * up_stage<kW_INT4>() <=
                  kMaxSmem,
              "two stages a warp beside the most tokens");

cudaError_t launch_few(const GateArgs& g, const FewArgs& a, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  switch (a.wkind) {
    case kW_BF16: return launch_both<kW_BF16>(g, a, di.sms, s);
    case kW_FP8: return launch_both<kW_FP8>(g, a, di.sms, s);
    case kW_INT8: return launch_both<kW_INT8>(g, a, di.sms, s);
    default: return launch_both<kW_INT4>(g, a, di.sms, s);
  }
}

}  // namespace moe
