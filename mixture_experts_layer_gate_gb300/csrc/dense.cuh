// Dense matrix product out[m, n] = sum_k a[m, k] w[n, k] on the tensor cores,
// shared by the block-scaled 8-bit product and the router scores: tcgen05 MMAs
// fed by TMA, accumulators in tensor memory, sums in registers.
//
// Tiles of 128 rows (token rows on the M side) by BN columns, K in k-blocks of
// 128 bytes (128 e4m3 or 64 bf16 / f16 values).  Every `group` k-blocks the MMA
// thread turns to the other of two accumulators, and the eight joining warps
// (two per tensor-memory lane quarter: warp w holds rows 32 (w % 4) .. + 31,
// one per lane, and one half of the columns) add the finished one, times the
// scales of its block, to the tile's sums, which stay in registers.  The 8-bit
// product joins every k-block, which is its scale block; the 16-bit one every
// 16 (1024 values), which only bounds the length of the tensor core's own sums.
//
// PAIR: two CTAs share MMAs of M = 256 (cta_group::2): each loads its own 128
// rows and half of the columns' weights, which halves the weight traffic from
// L2 per product.  Else P CTAs of a cluster take P ranges of K of one tile and
// join their sums through distributed shared memory in rank order (no atomics:
// the order is fixed).
#pragma once

#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace dense {

constexpr int kJoinWarps = 8;
constexpr int kFirstJoin = 4;  // warp 0 issues TMA, warp 1 MMAs, 2 and 3 fetch scales
constexpr int kThreads = 32 * (kFirstJoin + kJoinWarps);
// Registers a thread: the launch gives 168 x 384 (three warps per sub-partition);
// 256-column tiles hold 128 sums per joining thread, so the first warpgroup
// hands most of its share over (128 x (56 + 2 x 224) = 168 x 384).
constexpr int kLeanRegs = 56, kJoinRegs = 224, kLaunchRegs = 168;
// two accumulators
__host__ __device__ constexpr uint32_t tmem_cols(int bn) { return 2u * static_cast<uint32_t>(bn); }
constexpr int kMaxStages = 12;
constexpr int kMiscBytes = 4096;        // barriers, flags and the row maxima
// Products of scales, 8-bit operands: groups of four k-blocks x 128 rows x two
// weight-scale rows.
constexpr uint32_t kScaleSlots = 4, kScaleSlotBytes = 2 * 4 * 128 * 4;
// Transposition of the stored sums: per joining warp 32 rows of 16 floats, rows
// 80 bytes apart (eight lanes' 16-byte stores fall into different banks); of
// 256-column tiles that TMA stores, two boxes of 32 rows by 64 bytes, or four
// where it also fetches what the sums are added to and the ring keeps its stages
// (CTA pairs).
constexpr int kStageRow = 80, kBoxBytes = 32 * 64, kMaxBoxes = 4;
__host__ __device__ constexpr int out_stage_bytes(int bn, int boxes) {
  return bn == 256 ? boxes * kBoxBytes : 32 * kStageRow;
}
__host__ __device__ constexpr int fixed_bytes(int kind, bool swiglu, int bn, int boxes) {
  return kMiscBytes + (kind == 0 ? static_cast<int>(kScaleSlots * kScaleSlotBytes) : 0) +
         (swiglu ? 0 : kJoinWarps * out_stage_bytes(bn, boxes));
}
constexpr int kTileABytes = 128 * 128;  // what an MMA reads of A: 128 rows of a k-block

enum Kind : int { kE4M3 = 0, kHalf = 1 };

struct Params {
  const float* a_scale;  // [M, KB] (8-bit)
  const float* w_scale;  // [ceil(N / 128) or 2N / 128, KB] (8-bit)
  void* out;
  uint8_t* codes;        // SwiGLU
  float* scales;         // SwiGLU
  uint32_t* err;
  int64_t a_scale_stride, out_stride;
  int M, N, KB;
  int group;             // k-blocks per accumulator
  int P;                 // CTAs of a cluster that split K (not PAIR)
  int mt, nt;            // tiles
  int arows;             // rows of an A load: a multiple of 8, at most 128
  int stages;
  int fmt;               // 16-bit operands: 1 bf16, 0 f16
  int out_dtype;         // moe_dtype_t
  int accumulate;
  int vec;               // out rows take 16-byte stores
  int tma_out;           // 256-column tiles are stored by TMA
  int boxes;             // of each joining warp, for that: 2 or 4
  int vec_scale;         // rows of a_scale take 16-byte loads at multiples of four blocks
};

struct Maps {
  CUtensorMap a, w, out;
};

__host__ __device__ constexpr int wrows(int bn, bool pair) { return pair ? 128 : (bn < 128 ? bn : 128); }
__host__ __device__ constexpr int stage_bytes(int arows, int bn, bool pair) {
  return arows * 128 + (pair ? 128 : bn) * 128;
}
// shared row of a split-K partial, padded so that 8 lanes' 16-byte stores of 8
// rows fall into different banks
__host__ __device__ constexpr int part_ld(int bn) { return bn + 4; }

// 32 columns of this lane; r is there after tmem_ld32_wait(r)
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// waits for this thread's loads; r passes through, so that nothing reads it earlier
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// 16 columns of this lane, complete on return
__device__ __forceinline__ void tmem_ld16_wait(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds_u4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ void sts_u4(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ void sts_f4(uint32_t a, float4 v) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// A box of shared memory to `map` at (x, y); rows and columns past the tensor's
// are left out.
__device__ __forceinline__ void tma_store_box(const void* map, uint32_t src, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y), "r"(src)
      : "memory");
}

// acc += d * s, two floats at a time
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t d0, uint32_t d1, uint64_t s) {
  asm("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\tfma.rn.f32x2 %0, d, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(d0), "r"(d1), "l"(s));
}
// The same as two scalar multiply-adds where PACKED is false: the packed form
// needs its operands in register pairs and is the slower one in the storing
// kernels, with 124 bytes of spills a thread or (16 columns a load) without (down
// projection, M = 4096: 70 and 60 us packed, 51 us scalar), the faster one with
// SwiGLU (103 us packed, 107 us scalar).
template <bool PACKED>
__device__ __forceinline__ void add2(uint64_t& acc, uint32_t d0, uint32_t d1, uint64_t s) {
  if (PACKED) {
    fma2(acc, d0, d1, s);
  } else {
    const float f = __uint_as_float(static_cast<uint32_t>(s));
    const float x = fmaf(__uint_as_float(d0), f, __uint_as_float(static_cast<uint32_t>(acc)));
    const float y = fmaf(__uint_as_float(d1), f, __uint_as_float(static_cast<uint32_t>(acc >> 32)));
    acc = (static_cast<uint64_t>(__float_as_uint(y)) << 32) | __float_as_uint(x);
  }
}
__device__ __forceinline__ uint64_t pair2(float v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "r"(__float_as_uint(v)));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  return make_float2(__uint_as_float(static_cast<uint32_t>(v)), __uint_as_float(static_cast<uint32_t>(v >> 32)));
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// one arrival whose earlier shared-memory writes the waiters see
__device__ __forceinline__ void mbar_arrive_cta(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// mbar_wait without a call (a function call leaves no room for a warp to change
// its register count).
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* err,
                                     uint32_t info) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 0u) {
      if (abort_flag != nullptr && *abort_flag != 0) return false;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        if (abort_flag != nullptr) *abort_flag = 1;
        record_error(err, kErrTimeout, info);
        return false;
      }
    }
  }
}

__device__ __forceinline__ float max_nan(float a, float b) { return (a > b || a != a) ? a : b; }
__device__ __forceinline__ float quant_scale(float amax) {
  const float s = __fdiv_rn(amax, 448.0f);
  return s == 0.f ? 1.0f : s;
}
// By the fast exponential and division: within (8 + |g|) * 2^-23 of the value (zero
// below g = -87.3, where it is under 1e-36 u).  With expf M = 4096, K = 7168, N = 2048
// takes 104.7 us instead of 101.9, with an IEEE division too 113.7.
__device__ __forceinline__ float swiglu(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float scale) {
  return f32x2_to_e4m3x2(__fdiv_rn(a, scale), __fdiv_rn(b, scale)) |
         (static_cast<uint32_t>(f32x2_to_e4m3x2(__fdiv_rn(c, scale), __fdiv_rn(d, scale))) << 16);
}

// out[row, col .. col + 3] of four sums
__device__ __forceinline__ void store4(const Params& p, int64_t row, int col, float4 v) {
  const int64_t at = row * p.out_stride + col;
  float f[4] = {v.x, v.y, v.z, v.w};
  if (p.vec && col + 4 <= p.N) {
    if (p.out_dtype == 2) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
      if (p.accumulate) {
        const float4 u = *o;
        v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
      }
      *o = v;
    } else {
      uint2* o = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at);
      uint2 u = make_uint2(0, 0);
      if (p.accumulate) u = *o;
      if (p.out_dtype == 0) {
        if (p.accumulate) {
          f[0] += bf16_lo(u.x);
          f[1] += bf16_hi(u.x);
          f[2] += bf16_lo(u.y);
          f[3] += bf16_hi(u.y);
        }
        u = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
      } else {
        if (p.accumulate) {
          const float2 a = __half22float2(*reinterpret_cast<__half2*>(&u.x));
          const float2 b = __half22float2(*reinterpret_cast<__half2*>(&u.y));
          f[0] += a.x;
          f[1] += a.y;
          f[2] += b.x;
          f[3] += b.y;
        }
        __half2 a = __floats2half2_rn(f[0], f[1]), b = __floats2half2_rn(f[2], f[3]);
        u = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
      }
      *o = u;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (col + j >= p.N) return;
    if (p.out_dtype == 0) {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at + j;
      *o = __float2bfloat16_rn(p.accumulate ? f[j] + __bfloat162float(*o) : f[j]);
    } else if (p.out_dtype == 1) {
      __half* o = static_cast<__half*>(p.out) + at + j;
      *o = __float2half_rn(p.accumulate ? f[j] + __half2float(*o) : f[j]);
    } else {
      float* o = static_cast<float*>(p.out) + at + j;
      *o = p.accumulate ? f[j] + *o : f[j];
    }
  }
}

// ---- Single-thread instructions of a whole warp.  The TMA and MMA roles run
// their loops with all 32 lanes and predicate the instructions themselves on one
// lane: in code that only one lane enters, every descriptor has to be moved from
// a vector register to a uniform one, and a k-block's four MMAs and two commits
// took 450 cycles to issue, with their waits twice as long as the tensor pipe.

__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
  return p;
}

// The four MMAs of a k-block (32 bytes of K each); descriptors as (low, high)
// words, the low one advancing by 32 bytes >> 4.
template <int KIND, bool PAIR>
__device__ __forceinline__ void mma_kblock(uint32_t leader, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                           uint32_t idesc, uint32_t accumulate_first) {
#define MOE_DENSE_MMA4(GROUP, TYPE)                                                                                  \
  asm volatile(                                                                                                      \
      "{\n\t.reg .pred l, p, q;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\t"                                           \
      "setp.ne.b32 l, %0, 0;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 q, %4, %4;\n\t"                                 \
      "mov.b64 a, {%2, %4};\n\tmov.b64 b, {%3, %4};\n\t"                                                             \
      "@l tcgen05.mma.cta_group::" GROUP ".kind::" TYPE " [%1], a, b, %5, p;\n\t"                                    \
      "add.u32 x, %2, 2;\n\tadd.u32 y, %3, 2;\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t"                     \
      "@l tcgen05.mma.cta_group::" GROUP ".kind::" TYPE " [%1], a, b, %5, q;\n\t"                                    \
      "add.u32 x, %2, 4;\n\tadd.u32 y, %3, 4;\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t"                     \
      "@l tcgen05.mma.cta_group::" GROUP ".kind::" TYPE " [%1], a, b, %5, q;\n\t"                                    \
      "add.u32 x, %2, 6;\n\tadd.u32 y, %3, 6;\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t"                     \
      "@l tcgen05.mma.cta_group::" GROUP ".kind::" TYPE " [%1], a, b, %5, q;\n\t}" ::"r"(leader),                    \
      "r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate_first)                                       \
      : "memory")
  if (KIND == 0) {
    if (PAIR) MOE_DENSE_MMA4("2", "f8f6f4");
    else MOE_DENSE_MMA4("1", "f8f6f4");
  } else {
    if (PAIR) MOE_DENSE_MMA4("2", "f16");
    else MOE_DENSE_MMA4("1", "f16");
  }
#undef MOE_DENSE_MMA4
}

// Arrives on the barrier (PAIR: of both CTAs) when the MMAs issued so far complete.
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t leader, uint32_t bar) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred l;\n\t.reg .b16 m;\n\tsetp.ne.b32 l, %0, 0;\n\tmov.b16 m, 3;\n\t"
        "@l tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%1], m;\n\t}" ::"r"(
            leader),
        "r"(bar)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %0, 0;\n\t"
        "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(leader),
        "r"(bar)
        : "memory");
}

__device__ __forceinline__ void expect_tx(uint32_t leader, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %0, 0;\n\t"
      "@l mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%1], %2;\n\t}" ::"r"(leader),
      "r"(bar), "r"(bytes)
      : "memory");
}

// One box into this CTA's shared memory, counted on `bar` (PAIR: a barrier of the pair's leader).
template <bool PAIR>
__device__ __forceinline__ void load_box(uint32_t leader, uint32_t dst, const void* map, uint32_t bar, int c0, int c1) {
#define MOE_DENSE_LOAD(GROUP)                                                                                   \
  asm volatile(                                                                                                 \
      "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %0, 0;\n\t"                                                         \
      "@l cp.async.bulk.tensor.2d" GROUP ".shared::cluster.global.tile.mbarrier::complete_tx::bytes"            \
      " [%1], [%2, {%4, %5}], [%3];\n\t}" ::"r"(leader),                                                        \
      "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)                                \
      : "memory")
  if (PAIR) MOE_DENSE_LOAD(".cta_group::2");
  else MOE_DENSE_LOAD("");
#undef MOE_DENSE_LOAD
}

// ADD: 256-column tiles that are added to what out holds (a kernel of its own: what
// fetches the old values costs the storing one 51 -> 57 us at M = 4096, N = 7168,
// K = 2048); of narrower tiles p.accumulate tells.
template <int KIND, bool SWIGLU, bool PAIR, int BN, bool ADD>
__global__ void __launch_bounds__(kThreads, 1) dense_kernel(const __grid_constant__ Maps maps, const Params p) {
  static_assert(!SWIGLU || BN == 256, "gate and up halves of 128 columns");
  static_assert(!PAIR || BN == 256, "a pair's halves are 128 weight rows");
  static_assert(!ADD || (BN == 256 && !SWIGLU), "narrower tiles add at run time");
  constexpr int W = BN / 2;              // columns per joining warp
  constexpr int CH = W < 32 ? W : 32;    // columns per tensor-memory load
  constexpr int NCH = W / CH;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - raw_u32);
  const int ns = p.stages;
  const uint32_t abytes = static_cast<uint32_t>(p.arows) * 128u;
  const uint32_t sbytes = static_cast<uint32_t>(stage_bytes(p.arows, BN, PAIR));
  // barriers first, then the ring
  const uint32_t bars = base_u32;
  const uint32_t ring0 = base_u32 + kMiscBytes;  // scale products
  const uint32_t ring = base_u32 + fixed_bytes(KIND, SWIGLU, BN, p.boxes);
  const uint32_t stage0 = ring - kJoinWarps * out_stage_bytes(BN, p.boxes);
#define FULL(s) (bars + 8u * static_cast<uint32_t>(s))
#define EMPTY(s) (bars + 8u * static_cast<uint32_t>(kMaxStages + (s)))
#define SFULL(s) (bars + 16u * kMaxStages + 80u + 8u * (s))
#define BOX(s) (bars + 512u + 8u * (static_cast<uint32_t>(warp - kFirstJoin) * kMaxBoxes + (s)))
#define SEMPTY(s) (bars + 16u * kMaxStages + 80u + 8u * (kScaleSlots + (s)))
  const uint32_t dfull = bars + 16u * kMaxStages, dempty = dfull + 16u, drain = dfull + 32u;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(base + 16 * kMaxStages + 40);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + 16 * kMaxStages + 44);
  const uint32_t pairs = bars + 16u * kMaxStages + 48u;    // one per lane quarter
  float* row_max = reinterpret_cast<float*>(base + 1024);  // [2][2][128]: tile parity, column half, row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = (PAIR || p.P > 1) ? cluster_ctarank() : 0u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ns; ++s) {
      mbar_init(FULL(s), 1u);
      mbar_init(EMPTY(s), 1u);
    }
    for (uint32_t b = 0; b < 2; ++b) {
      mbar_init(dfull + 8u * b, 1u);
      mbar_init(dempty + 8u * b, kJoinWarps * (PAIR ? 2u : 1u));
    }
    mbar_init(drain, 1u);
    for (uint32_t q = 0; q < 4; ++q) mbar_init(pairs + 8u * q, 2u);
    for (uint32_t q = 0; q < kScaleSlots; ++q) {
      mbar_init(SFULL(q), 1u);
      mbar_init(SEMPTY(q), kJoinWarps);
    }
    if (ADD)
      for (uint32_t q = 0; q < kJoinWarps * kMaxBoxes; ++q) mbar_init(bars + 512u + 8u * q, 1u);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.w);
    if (p.tma_out) tma_prefetch_desc(&maps.out);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(smem_u32(const_cast<uint32_t*>(tmem_slot)), tmem_cols(BN));
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), tmem_cols(BN));
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();  // the peer's barriers are initialised before anyone signals them
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;

  // tiles of this cluster (PAIR) or CTA; a K-splitting cluster has one
  const int tiles = p.mt * p.nt;
  const int width = PAIR ? 2 : p.P;
  const int first = static_cast<int>(blockIdx.x) / width;
  const int step = static_cast<int>(gridDim.x) / width;
  const int kb0 = PAIR ? 0 : static_cast<int>(static_cast<int64_t>(p.KB) * rank / p.P);
  const int kb1 = PAIR ? p.KB : static_cast<int>(static_cast<int64_t>(p.KB) * (rank + 1) / p.P);
  constexpr int kTileM = PAIR ? 256 : 128;
  constexpr int kElems = KIND == kE4M3 ? 128 : 64;

  if (warp < kFirstJoin) {
    if (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLeanRegs));
    if (warp == 0) {
      // ------------------------------------------------------ TMA producer
      const uint32_t leader = elect_one();
      int st = 0, issued = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        const int m0 = (t % p.mt) * kTileM + (PAIR ? 128 * static_cast<int>(rank) : 0);
        const int n0 = (t / p.mt) * (SWIGLU ? 128 : BN);
        // the weight rows: PAIR loads one half here, the peer the other
        const int second = SWIGLU ? n0 + p.N : n0 + 128;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait(EMPTY(st), ph ^ 1u, abort_flag, p.err, 0x600u)) {
            ok = false;
            break;
          }
          const uint32_t dst = ring + static_cast<uint32_t>(st) * sbytes;
          if (PAIR) {
            const uint32_t bar = map_to_rank(FULL(st), 0);
            if (rank == 0) expect_tx(leader, FULL(st), 2u * sbytes);
            load_box<true>(leader, dst, &maps.a, bar, kb * kElems, m0);
            load_box<true>(leader, dst + abytes, &maps.w, bar, kb * kElems, rank == 0 ? n0 : second);
          } else {
            expect_tx(leader, FULL(st), sbytes);
            load_box<false>(leader, dst, &maps.a, FULL(st), kb * kElems, m0);
            load_box<false>(leader, dst + abytes, &maps.w, FULL(st), kb * kElems, n0);
            if (BN == 256) load_box<false>(leader, dst + abytes + 128u * 128u, &maps.w, FULL(st), kb * kElems, second);
          }
          ++issued;
          if (++st == ns) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok && (!PAIR || rank == 0)) {
        // after an abort the loads in flight land before the CTA (or its pair,
        // whose leader counts both CTAs' bytes) may leave
        for (int i = min(issued, ns); i > 0; --i) {
          st = st == 0 ? ns - 1 : st - 1;
          if (st == ns - 1) ph ^= 1u;
          wait(FULL(st), ph, nullptr, p.err, 0x601u);
        }
      }
    } else if (warp == 1 && (!PAIR || rank == 0)) {
      // --------------------------------------------- MMA issuer (leader CTA)
      const uint32_t leader = elect_one();
      const uint32_t idesc = make_idesc(kTileM, BN, KIND == kE4M3 ? 0u : static_cast<uint32_t>(p.fmt));
      const uint64_t desc0 = sw128_kmajor_desc(ring);
      const uint32_t desc_lo = static_cast<uint32_t>(desc0), desc_hi = static_cast<uint32_t>(desc0 >> 32);
      int st = 0;
      uint32_t ph = 0, buf = 0, dph = 0;
      bool ok = true, any = false;
      for (int t = first; t < tiles && ok; t += step) {
        for (int kb = kb0; kb < kb1 && ok;) {
          const uint32_t d = tmem + buf * static_cast<uint32_t>(BN);
          const int end = min(kb + p.group, kb1);
          for (uint32_t accum = 0; kb < end; ++kb, accum = 1) {
            // the operands first: they are there by the time the accumulator is
            if (!wait(FULL(st), ph, abort_flag, p.err, 0x620u) ||
                (accum == 0 && !wait(dempty + 8u * buf, dph ^ 1u, abort_flag, p.err, 0x610u))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a_lo = desc_lo + ((static_cast<uint32_t>(st) * sbytes) >> 4);
            mma_kblock<KIND, PAIR>(leader, d, a_lo, a_lo + (abytes >> 4), desc_hi, idesc, accum);
            commit<PAIR>(leader, EMPTY(st));
            any = true;
            if (++st == ns) {
              st = 0;
              ph ^= 1u;
            }
          }
          if (!ok) break;
          commit<PAIR>(leader, dfull + 8u * buf);
          buf ^= 1u;
          if (buf == 0u) dph ^= 1u;
        }
      }
      if (!ok && any) {  // MMAs in flight end before tensor memory is freed
        if (leader != 0u) {
          if (PAIR) mma_commit_pair(drain, 0x1);
          else mma_commit(drain);
        }
        wait(drain, 0u, nullptr, p.err, 0x630u);
      }
    }
    if (KIND == kE4M3 && warp >= 2) {
      // ------------------------------------------------------- scale warps
      // A row's scale times its weight block's, for four k-blocks at a time and
      // up to kScaleSlots such groups ahead of the joining warps (a load from L2
      // takes longer than a block's product).  The two warps take turns.
      uint32_t n = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        const int m0 = (t % p.mt) * kTileM + (PAIR ? 128 * static_cast<int>(rank) : 0);
        const int n0 = (t / p.mt) * (SWIGLU ? 128 : BN);
        // the tile's two weight-scale rows: gate and up, or the column halves
        const int last = (p.N - 1) / 128;
        const float* ws0 = p.w_scale + static_cast<int64_t>(n0 / 128) * p.KB;
        const float* ws1 = p.w_scale + static_cast<int64_t>(SWIGLU ? (n0 + p.N) / 128 : min(n0 / 128 + 1, last)) * p.KB;
        for (int kq = kb0; kq < kb1; kq += 4, ++n) {
          if ((n & 1u) != static_cast<uint32_t>(warp & 1)) continue;
          const uint32_t slot = n & (kScaleSlots - 1);
          if (!wait(SEMPTY(slot), (n / kScaleSlots & 1u) ^ 1u, abort_flag, p.err, 0x670u)) {
            ok = false;
            break;
          }
          float4 sa[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float* as = p.a_scale + static_cast<int64_t>(min(m0 + 32 * q + lane, p.M - 1)) * p.a_scale_stride;
            if (p.vec_scale && kq + 4 <= kb1) {
              sa[q] = *reinterpret_cast<const float4*>(as + kq);
            } else {
              sa[q].x = as[kq];
              sa[q].y = as[min(kq + 1, kb1 - 1)];
              sa[q].z = as[min(kq + 2, kb1 - 1)];
              sa[q].w = as[min(kq + 3, kb1 - 1)];
            }
          }
          float* dst = reinterpret_cast<float*>(base + kMiscBytes) + slot * (kScaleSlotBytes / 4) + lane;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int kb = min(kq + j, kb1 - 1);
            const float w0 = ws0[kb], w1 = ws1[kb];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float v = j == 0 ? sa[q].x : j == 1 ? sa[q].y : j == 2 ? sa[q].z : sa[q].w;
              dst[j * 128 + 32 * q] = v * w0;
              dst[512 + j * 128 + 32 * q] = v * w1;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(SFULL(slot));
        }
      }
    }
    // Every warp leaves its role with the registers of the launch.  The joining
    // warps give theirs back before this warpgroup takes its own again: a warp
    // without a role that took them at once could leave a joining warp waiting
    // for registers that nobody returns.
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLaunchRegs));
  } else {
    if (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kJoinRegs));
    // ------------------------------------------------------- joining warps
    const int quarter = warp & 3, half = (warp - kFirstJoin) >> 2;
    const uint32_t lane_base = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t dempty_to = PAIR ? map_to_rank(dempty, 0) : dempty;
    uint32_t buf = 0, dph = 0, tile = 0, quad = 0;
    // boxes that TMA fetches: the parity of each one's next arrival, and those on their way
    uint32_t box_phase = 0, box_loads = 0;
    const bool fetch = ADD && p.tma_out;
    const uint32_t boxes0 = stage0 + static_cast<uint32_t>(warp - kFirstJoin) * out_stage_bytes(BN, p.boxes);
    const int box_cols = p.out_dtype == 2 ? 16 : 32;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      const int m0 = (t % p.mt) * kTileM + (PAIR ? 128 * static_cast<int>(rank) : 0);
      const int n0 = (t / p.mt) * (SWIGLU ? 128 : BN);
      // what chunk i of the warp's columns is added to, into its box; the box's
      // last store has read it
      auto fetch_box = [&](int i) {
        const uint32_t slot = static_cast<uint32_t>(i & (p.boxes - 1));
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        expect_tx(lane == 0, BOX(slot), kBoxBytes);
        load_box<false>(lane == 0, boxes0 + slot * kBoxBytes, &maps.out, BOX(slot), n0 + W * half + i * box_cols,
                        m0 + 32 * quarter);
        box_loads |= 1u << slot;
      };
      const int row = m0 + 32 * quarter + lane;
      const bool live = m0 + 32 * quarter < p.M;  // some row of this warp exists
      // columns of load c: SwiGLU takes 64 gate columns, then the 64 up columns
      // that go with them
      auto column_of = [&](int c) {
        return static_cast<uint32_t>(SWIGLU ? 64 * half + (c & 1) * 32 + (c >> 1) * 128 : W * half + CH * c);
      };
      if (fetch && live)
        for (int i = 0; i < p.boxes; ++i) fetch_box(i);
      uint64_t acc[W / 2];
#pragma unroll
      for (int i = 0; i < W / 2; ++i) acc[i] = 0;
      for (int kq = kb0; kq < kb1 && ok; kq += 4 * p.group) {
        const uint32_t slot = quad & (kScaleSlots - 1);
        const uint32_t factors = ring0 + slot * kScaleSlotBytes + static_cast<uint32_t>(32 * quarter + lane) * 4u;
        if (KIND == kE4M3 && !wait(SFULL(slot), quad / kScaleSlots & 1u, abort_flag, p.err, 0x660u)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int j4 = 0; j4 < 4; ++j4) {
          if (kq + j4 * p.group >= kb1) break;
          if (!wait(dfull + 8u * buf, dph, abort_flag, p.err, 0x640u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint64_t g0, g1;
          if (KIND == kE4M3) {
            g0 = pair2(lds_f32(factors + static_cast<uint32_t>(SWIGLU || BN < 256 ? 0 : half) * 2048u + j4 * 512u));
            g1 = SWIGLU ? pair2(lds_f32(factors + 2048u + j4 * 512u)) : g0;
          } else {
            g0 = g1 = pair2(1.f);
          }
          const uint32_t src = tmem + lane_base + buf * static_cast<uint32_t>(BN);
          if constexpr (CH == 32) {
            // a load of 32 columns runs while the 32 before are added
            if (live) {
              uint32_t r[2][32];
              tmem_ld32(src + column_of(0), r[0]);
#pragma unroll
              for (int c = 0; c < NCH; ++c) {
                tmem_ld32_wait(r[c & 1]);
                if (c + 1 < NCH) tmem_ld32(src + column_of(c + 1), r[(c + 1) & 1]);
                if (c + 1 == NCH) {
                  tc_fence_before();
                  if (lane == 0) mbar_arrive_cluster(dempty_to + 8u * buf);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  add2<SWIGLU>(acc[16 * c + j], r[c & 1][2 * j], r[c & 1][2 * j + 1], (SWIGLU && c >= 2) ? g1 : g0);
              }
            } else {
              tc_fence_before();
              if (lane == 0) mbar_arrive_cluster(dempty_to + 8u * buf);
            }
          } else {
            if (live) {
              uint32_t r[16];
              tmem_ld16_wait(src + column_of(0), r);
#pragma unroll
              for (int j = 0; j < 8; ++j) add2<SWIGLU>(acc[j], r[2 * j], r[2 * j + 1], g0);
            }
            tc_fence_before();
            if (lane == 0) mbar_arrive_cluster(dempty_to + 8u * buf);
          }
          buf ^= 1u;
          if (buf == 0u) dph ^= 1u;
        }
        if (KIND == kE4M3) {
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(SEMPTY(slot));
          ++quad;
        }
      }
      if (!ok) break;

      if (!PAIR && p.P > 1) {
        // partial sums into this CTA's shared memory (the ring is drained: the
        // last accumulator was finished by the last MMA that read it)
        if (row < p.M) {
          float* dst = reinterpret_cast<float*>(base + fixed_bytes(KIND, SWIGLU, BN, p.boxes)) + (32 * quarter + lane) * part_ld(BN);
#pragma unroll
          for (int c = 0; c < NCH; ++c) {
            const int col = SWIGLU ? 64 * half + (c & 1) * 32 + (c >> 1) * 128 : W * half + CH * c;
#pragma unroll
            for (int j = 0; j < CH / 4; ++j) {
              const float2 u = unpair(acc[CH / 2 * c + 2 * j]), v = unpair(acc[CH / 2 * c + 2 * j + 1]);
              *reinterpret_cast<float4*>(dst + col + 4 * j) = make_float4(u.x, u.y, v.x, v.y);
            }
          }
        }
      } else if (SWIGLU) {
        float v[W / 2];
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < W / 4; ++j) {
          const float2 g = unpair(acc[j]), u = unpair(acc[W / 4 + j]);
          v[2 * j] = swiglu(g.x, u.x);
          v[2 * j + 1] = swiglu(g.y, u.y);
          amax = max_nan(amax, max_nan(fabsf(v[2 * j]), fabsf(v[2 * j + 1])));
        }
        // the other half of the row's block is held by the warp four further on
        // (or back); a warp writes a buffer again two tiles later, when the
        // other has read it before arriving for the tile between
        float* mine = row_max + (tile & 1u) * 256 + 32 * quarter + lane;
        mine[half * 128] = amax;
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(pairs + 8u * quarter);
        if (!wait(pairs + 8u * quarter, tile & 1u, abort_flag, p.err, 0x650u)) {
          ok = false;
          break;
        }
        amax = max_nan(amax, mine[(half ^ 1) * 128]);
        ++tile;
        if (row < p.M) {
          const float scale = quant_scale(amax);
          if (half == 0) p.scales[static_cast<int64_t>(row) * (p.N / 128) + n0 / 128] = scale;
          uint4* dst = reinterpret_cast<uint4*>(p.codes + static_cast<int64_t>(row) * p.N + n0 + 64 * half);
#pragma unroll
          for (int j = 0; j < W / 32; ++j)
            dst[j] = make_uint4(codes4(v[16 * j], v[16 * j + 1], v[16 * j + 2], v[16 * j + 3], scale),
                                codes4(v[16 * j + 4], v[16 * j + 5], v[16 * j + 6], v[16 * j + 7], scale),
                                codes4(v[16 * j + 8], v[16 * j + 9], v[16 * j + 10], v[16 * j + 11], scale),
                                codes4(v[16 * j + 12], v[16 * j + 13], v[16 * j + 14], v[16 * j + 15], scale));
        }
      } else if (BN == 256 && p.tma_out) {
        // 64 bytes of a row at a time: boxes in shared memory (16-byte pieces swizzled
        // so that eight lanes' stores fall into different banks), which TMA
        // writes while the next box is filled and the next tile's blocks are joined.
        // What the sums are added to is there by then (fetch_box).  M = 4096, N =
        // 7168, K = 2048, bf16: 51 us, added 62; plain stores of the tile 62 and 130.
        if (live) {
          auto box = [&](int i, auto&& piece) {  // piece(j, old): 16 bytes
            const uint32_t slot = static_cast<uint32_t>(i & (p.boxes - 1));
            const uint32_t dst = boxes0 + slot * kBoxBytes, mine = dst + static_cast<uint32_t>(lane * 64);
            if (fetch) {
              ok = ok && wait(BOX(slot), box_phase >> slot & 1u, abort_flag, p.err, 0x680u);
              if (!ok) return;
              box_phase ^= 1u << slot;
              box_loads &= ~(1u << slot);
            } else {
              if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");  // the last one but one is read
              __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t at = mine + static_cast<uint32_t>(16 * (j ^ (lane >> 1 & 3)));
              sts_u4(at, piece(j, fetch ? lds_u4(at) : make_uint4(0u, 0u, 0u, 0u)));
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            const int x = n0 + W * half + i * box_cols;
            if (lane == 0) {
              if (x < p.N) tma_store_box(&maps.out, dst, x, m0 + 32 * quarter);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");  // (a group for every box)
            }
            if (fetch && (i + p.boxes) * box_cols < W) fetch_box(i + p.boxes);
          };
          if (p.out_dtype == 2) {
#pragma unroll
            for (int i = 0; i < W / 16; ++i)
              box(i, [&](int j, uint4 old) {
                const float2 u = unpair(acc[8 * i + 2 * j]), v = unpair(acc[8 * i + 2 * j + 1]);
                if (!ADD) return make_uint4(__float_as_uint(u.x), __float_as_uint(u.y), __float_as_uint(v.x), __float_as_uint(v.y));
                return make_uint4(__float_as_uint(u.x + __uint_as_float(old.x)), __float_as_uint(u.y + __uint_as_float(old.y)),
                                  __float_as_uint(v.x + __uint_as_float(old.z)), __float_as_uint(v.y + __uint_as_float(old.w)));
              });
          } else {
            const bool f16 = p.out_dtype == 1;
            auto two = [&](uint64_t a, uint32_t old) {
              float2 v = unpair(a);
              if (ADD) {
                const float2 o = f16 ? __half22float2(*reinterpret_cast<const __half2*>(&old))
                                     : make_float2(bf16_lo(old), bf16_hi(old));
                v = make_float2(v.x + o.x, v.y + o.y);
              }
              const __half2 h = __floats2half2_rn(v.x, v.y);
              return f16 ? *reinterpret_cast<const uint32_t*>(&h) : pack_bf16x2(v.x, v.y);
            };
#pragma unroll
            for (int i = 0; i < W / 32; ++i)
              box(i, [&](int j, uint4 old) {
                const uint64_t* q = acc + 16 * i + 4 * j;
                return make_uint4(two(q[0], old.x), two(q[1], old.y), two(q[2], old.z), two(q[3], old.w));
              });
          }
        }
        if (!ok) break;
      } else {
        // 16 columns at a time through shared memory, so that four lanes write 16
        // adjacent columns of a row: whole 32-byte sectors (one row per lane
        // wrote 8 bytes of 32 rows at a time and took twice the product's time
        // at M = 4096, N = 7168, K = 2048)
        const uint32_t mine = stage0 + static_cast<uint32_t>(4 * half + quarter) * out_stage_bytes(BN, p.boxes);
        const int to0 = m0 + 32 * quarter + (lane >> 2), col0 = n0 + W * half + 4 * (lane & 3);
        // a whole tile's columns, aligned stores (of 256-column tiles those are TMA's)
        const bool fast = BN < 256 && p.vec && !p.accumulate && n0 + BN <= p.N;
        const int64_t at = static_cast<int64_t>(to0) * p.out_stride + col0, eight = 8 * p.out_stride;
#pragma unroll
        for (int c = 0; c < W / 16; ++c) {
          const int col = 16 * c;
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 u = unpair(acc[8 * c + 2 * j]), v = unpair(acc[8 * c + 2 * j + 1]);
            sts_f4(mine + static_cast<uint32_t>(lane * kStageRow + 16 * j), make_float4(u.x, u.y, v.x, v.y));
          }
          __syncwarp();
          const uint32_t from = mine + static_cast<uint32_t>((lane >> 2) * kStageRow + 16 * (lane & 3));
          if (!fast) {
#pragma unroll 1
            for (int i = 0; i < 4; ++i)
              if (to0 + 8 * i < p.M) store4(p, to0 + 8 * i, col0 + col, lds_f4(from + static_cast<uint32_t>(8 * i * kStageRow)));
          } else if (p.out_dtype == 2) {
            float* o = static_cast<float*>(p.out) + at + col;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (to0 + 8 * i < p.M)
                *reinterpret_cast<float4*>(o + i * eight) = lds_f4(from + static_cast<uint32_t>(8 * i * kStageRow));
          } else {
            uint16_t* o = static_cast<uint16_t*>(p.out) + at + col;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 v = lds_f4(from + static_cast<uint32_t>(8 * i * kStageRow));
              uint2 q = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
              if (p.out_dtype == 1) {
                __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
                q = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
              }
              if (to0 + 8 * i < p.M) *reinterpret_cast<uint2*>(o + i * eight) = q;
            }
          }
        }
      }
    }
    if (BN == 256 && !SWIGLU) {
      for (uint32_t i = 0; ADD && i < kMaxBoxes; ++i)  // (after an abort only)
        if (box_loads >> i & 1u) wait(BOX(i), box_phase >> i & 1u, nullptr, p.err, 0x681u);
      if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // stored
    }
    __syncwarp();
    if (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLaunchRegs));
    tc_fence_before();
    __syncthreads();
  }
#undef FULL
#undef EMPTY
#undef SFULL
#undef SEMPTY
#undef BOX

  if (PAIR || p.P > 1) cluster_sync_all();  // signals and partial sums have arrived
  if (!PAIR && p.P > 1) {
    // a warp per row of this rank's share, a lane per four columns
    const int m0 = (first % p.mt) * 128, n0 = (first / p.mt) * (SWIGLU ? 128 : BN);
    const int rows = min(128, p.M - m0);
    for (int r = static_cast<int>(rank) + p.P * warp; r < rows; r += p.P * (kThreads / 32)) {
      const uint32_t src = ring + static_cast<uint32_t>(r * part_ld(BN)) * 4u;
      auto joined = [&](int col) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q = 0; q < p.P; ++q) {
          const float4 v = ld_cluster_f4(map_to_rank(src + static_cast<uint32_t>(col) * 4u, static_cast<uint32_t>(q)));
          s.x += v.x;
          s.y += v.y;
          s.z += v.z;
          s.w += v.w;
        }
        return s;
      };
      if (SWIGLU) {
        const float4 g = joined(4 * lane), u = joined(128 + 4 * lane);
        const float a = swiglu(g.x, u.x), b = swiglu(g.y, u.y), c = swiglu(g.z, u.z), d = swiglu(g.w, u.w);
        float amax = max_nan(max_nan(fabsf(a), fabsf(b)), max_nan(fabsf(c), fabsf(d)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float scale = quant_scale(amax);
        if (lane == 0) p.scales[static_cast<int64_t>(m0 + r) * (p.N / 128) + n0 / 128] = scale;
        reinterpret_cast<uint32_t*>(p.codes + static_cast<int64_t>(m0 + r) * p.N + n0)[lane] = codes4(a, b, c, d, scale);
      } else {
        for (int col = 4 * lane; col < BN; col += 128) store4(p, m0 + r, n0 + col, joined(col));
      }
    }
    cluster_sync_all();  // no CTA leaves while a peer reads its sums
  }
  if (warp == 1) {
    tc_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem, tmem_cols(BN));
    else tmem_dealloc(tmem, tmem_cols(BN));
  }
}

// ------------------------------------------------------------------ launch

constexpr size_t kMaxSmem = 232448;

// Dynamic shared memory for `stages` ring stages: what an MMA of a short A tile
// reads past its rows, and a split-K partial, stay inside.
template <int KIND, bool SWIGLU>
size_t smem_bytes(const Params& p, int bn, bool pair) {
  size_t ring = static_cast<size_t>(p.stages) * stage_bytes(p.arows, bn, pair) + (kTileABytes - p.arows * 128);
  if (!pair && p.P > 1) {
    const int rows = p.M < 128 ? p.M : 128;
    const size_t part = static_cast<size_t>(rows) * part_ld(bn) * 4;
    if (part > ring) ring = part;
  }
  return std::max(kTensorMemorySmem, 1024 + fixed_bytes(KIND, SWIGLU, bn, p.boxes) + ring);
}

template <int KIND, bool SWIGLU, bool PAIR, int BN, bool ADD = false>
cudaError_t launch(const Maps& maps, const Params& p, int grid, cudaStream_t s) {
  static int configured[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  auto kernel = dense_kernel<KIND, SWIGLU, PAIR, BN, ADD>;
  if (dev < 0 || dev >= 64 || configured[dev] == 0) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxSmem));
    if (err != cudaSuccess) return err;
    cudaFuncAttributes attr;
    err = cudaFuncGetAttributes(&attr, kernel);
    if (err != cudaSuccess) return err;
    // the warps' register counts add up to the launch's only if it has these
    if (BN == 256 && attr.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  return launch_pdl_cluster(kernel, dim3(grid), dim3(kThreads), smem_bytes<KIND, SWIGLU>(p, BN, PAIR), s,
                            static_cast<unsigned>(PAIR ? 2 : p.P), maps, p);
}

// Tile width, CTA pairs and the split of K.
struct Choice {
  int bn;
  bool pair;
  int P;
};

// The candidate with the least estimated time in cycles: rounds of the SMs times
// (k-blocks of a CTA times a k-block's time, and the tile's end).  The k-block
// times are measured ones of the whole loop (16-bit: H = 7168, 256 experts, 1 to
// 4096 tokens; 8-bit: 1 to 4096 rows of the DeepSeek-V3 shared expert).  Eight
// CTAs a cluster only for eight tiles at most: more such clusters do not all fit
// on the SMs at once (one row, N = 2048, K = 7168 with SwiGLU: 24 us by eights,
// 18 us by fours).
inline Choice choose(int M, int N, int KB, bool swiglu, bool e4m3, int sms) {
  Choice best{256, false, 1};
  double best_time = 1e30;
  const double arows = std::min(128, (M + 7) / 8 * 8);
  for (int w = 0; w < 5; ++w) {
    constexpr int width[5] = {32, 64, 128, 256, 256};
    constexpr double half_block[5] = {250, 340, 560, 1150, 1150}, e4m3_block[5] = {600, 690, 800, 1250, 950};
    const int bn = width[w];
    const bool pair = w == 4;
    if ((swiglu && bn != 256) || (pair && (M <= 128 || !e4m3))) continue;
    const int tm = pair ? 256 : 128, tn = swiglu ? 128 : bn;
    const long long tiles = static_cast<long long>((M + tm - 1) / tm) * ((N + tn - 1) / tn);
    for (int P = 1; P <= 8 && P <= KB; P *= 2) {
      if (P > 1 && (pair || tiles * P > sms || (P == 8 && tiles > 8))) break;
      const long long slots = pair ? sms / 2 : sms / P;
      const double rounds = static_cast<double>((tiles + slots - 1) / slots);
      const double end = (P > 1 ? 2500.0 : 300.0) + arows * bn / 7.0;
      const double time = rounds * ((KB + P - 1) / P * (e4m3 ? e4m3_block[w] : half_block[w]) + end);
      if (time < best_time) {
        best_time = time;
        best = {bn, pair, P};
      }
    }
  }
  return best;
}

// Descriptors, tile counts and ring depth, then the launch.  p: everything but
// mt, nt, arows and stages.  a [M, K] and w [wrows_total, K] of 1-byte (kE4M3)
// or 2-byte elements, strides in elements.
template <int KIND>
cudaError_t plan_and_launch(Params p, int bn, bool pair, bool swiglu, const void* a, int64_t a_stride, const void* w,
                            int64_t w_stride, int64_t w_total, int64_t K, int sms, cudaStream_t s) {
  const uint64_t esz = KIND == kE4M3 ? 1 : 2;
  const CUtensorMapDataType dt = KIND == kE4M3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : p.fmt == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int tile_m = pair ? 256 : 128;
  p.mt = (p.M + tile_m - 1) / tile_m;
  p.nt = (p.N + (swiglu ? 128 : bn) - 1) / (swiglu ? 128 : bn);
  p.arows = pair || p.M >= 128 ? 128 : (p.M + 7) / 8 * 8;
  const int sb = stage_bytes(p.arows, bn, pair);
  p.tma_out = bn == 256 && !swiglu && p.P == 1 && p.vec;
  p.boxes = p.tma_out && p.accumulate && pair ? kMaxBoxes : 2;
  const int fixed = fixed_bytes(KIND, swiglu, bn, p.boxes);
  const size_t room = kMaxSmem - 1024 - fixed - (kTileABytes - p.arows * 128);
  const int per_cta = pair ? p.KB : (p.KB + p.P - 1) / p.P;
  const int most = static_cast<int>(room / sb);
  p.stages = most < kMaxStages ? most : kMaxStages;
  // a K-splitting CTA has one tile: no more stages than k-blocks
  if (p.P > 1 && p.stages > per_cta) p.stages = per_cta;
  Maps maps = {};
  if (p.tma_out) {
    const uint64_t osz = p.out_dtype == 2 ? 4 : 2;
    const uint64_t dims[2] = {static_cast<uint64_t>(p.N), static_cast<uint64_t>(p.M)};
    const uint64_t str[1] = {static_cast<uint64_t>(p.out_stride) * osz};
    const uint32_t box[2] = {static_cast<uint32_t>(64 / osz), 32};
    if (!encode_map(&maps.out, osz == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.out,
                    dims, str, box, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  }
  {
    const uint64_t dims[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(p.M)};
    const uint64_t str[1] = {static_cast<uint64_t>(a_stride) * esz};
    const uint32_t box[2] = {static_cast<uint32_t>(128 / esz), static_cast<uint32_t>(p.arows)};
    if (!encode_map(&maps.a, dt, 2, a, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
  }
  {
    const uint64_t dims[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(w_total)};
    const uint64_t str[1] = {static_cast<uint64_t>(w_stride) * esz};
    const uint32_t box[2] = {static_cast<uint32_t>(128 / esz), static_cast<uint32_t>(wrows(bn, pair))};
    if (!encode_map(&maps.w, dt, 2, w, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
  }
  const long long tiles = static_cast<long long>(p.mt) * p.nt;
  if (tiles * 16 > (1ll << 30)) return cudaErrorInvalidValue;
  int grid;
  if (pair) {
    grid = 2 * static_cast<int>(tiles < sms / 2 ? tiles : sms / 2);
    if constexpr (KIND == kE4M3) {
      if (swiglu) return launch<KIND, true, true, 256>(maps, p, grid, s);
      return p.accumulate ? launch<KIND, false, true, 256, true>(maps, p, grid, s)
                          : launch<KIND, false, true, 256>(maps, p, grid, s);
    } else {
      return cudaErrorInvalidValue;  // (choose() pairs CTAs for 8-bit operands only)
    }
  }
  if (p.P > 1) grid = static_cast<int>(tiles) * p.P;
  else grid = static_cast<int>(tiles < sms ? tiles : sms);
  if constexpr (KIND == kE4M3) {
    if (swiglu) return launch<KIND, true, false, 256>(maps, p, grid, s);
    if (bn == 256 && p.accumulate) return launch<KIND, false, false, 256, true>(maps, p, grid, s);
  }
  switch (bn) {
    case 32: return launch<KIND, false, false, 32>(maps, p, grid, s);
    case 64: return launch<KIND, false, false, 64>(maps, p, grid, s);
    case 128: return launch<KIND, false, false, 128>(maps, p, grid, s);
    default: return launch<KIND, false, false, 256>(maps, p, grid, s);
  }
}

}  // namespace dense
}  // namespace moe
