// Attention of many rows (chunks of prompts, whole prompts) on the tensor cores:
// tcgen05 MMAs with scores, weights and outputs in tensor memory.
//
// An item is 256 rows of a sequence and key head (row i G + g: query head g of the
// group, new token i), two halves of 128 that share every key and value tile: S =
// Q K^T (128 x 128 scores a half), the softmax's weights P over S in place as 16-bit
// values, O += P V with P as the tensor-memory operand.  While one half's warps turn
// its scores into weights, the other half's products run.
//
// Warps: 0-3 and 4-7 the halves' softmax (a thread a row: no exchange between
// threads), 8 loads (16-bit: TMA, a box a page and 64 values) or scales (8-bit), 9
// MMAs; 16-bit: 10 and 11 look at the values of tiles that some row does not wholly
// see; 8-bit: 10 to 15 turn codes into f16 tiles.
//
// The running maximum is only raised, and O rescaled, when it grew by more than 8
// (factors of 2^8 stay far inside the sums' and the weights' range), which is rare
// after the first tiles.  A row's result does not depend on it but for roundings.
//
// Masked scores become -inf whatever they were.  Values behind the sequence's end
// are zeroed in shared memory, and values that are not finite in a tile that some row
// does not wholly see are taken out there and added at the end to the rows that do
// see them: 0 * NaN would reach the others.
#include "attention.cuh"
#include "dense.cuh"

namespace moe {
namespace {

using namespace attn;
using dense::commit;
using dense::elect_one;
using dense::expect_tx;
using dense::mbar_arrive_cta;
using dense::wait;

constexpr int kHalf = 128, kRows = 2 * kHalf, kKeys = 128;
constexpr int kMaxSlots = 8, kScaleSlots = 2, kDirty = 16;
constexpr size_t kSmem = 232448;
// Registers a thread of the softmax's warpgroups and of the others; 3 x 168 and 4 x
// 128 at launch.
constexpr int kSoftRegs16 = 200, kLeanRegs16 = 104, kLaunchRegs16 = 168;
constexpr int kSoftRegs8 = 192, kLeanRegs8 = 64, kLaunchRegs8 = 128;
template <bool E4M3>
constexpr int kThreads = E4M3 ? 512 : 384;
constexpr int kGuards = 2, kConverters = 6;  // warps from 10 on
constexpr uint32_t kTmemCols = 512, kOut = 256;  // scores of half i at 128 i, outputs at 256 + 128 i

using BigWalk = Walk<kRows, kKeys>;

// Barriers and small arrays, then (1024-byte aligned) Q's halves and the ring of key
// and value tiles.
constexpr int kBarBytes = 1024;
constexpr int kScaleBytes = kScaleSlots * (2 * kKeys + 4) * 4;
template <bool E4M3>
constexpr int kMiscBytes = E4M3 ? 4096 : kBarBytes;
static_assert(kBarBytes + kScaleBytes <= kMiscBytes<true>, "scales lie between the barriers and Q");
__host__ __device__ constexpr int tile_bytes(int dp) { return kKeys * dp * 2; }

struct Maps {
  CUtensorMap k, v;
};

__device__ __forceinline__ void load_box4(uint32_t leader, uint32_t dst, const void* map, uint32_t bar, int c0, int c1,
                                          int c2, int c3) {
  asm volatile(
      "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %0, 0;\n\t"
      "@l cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%1], [%2, {%4, %5, %6, %7}], [%3];\n\t}" ::"r"(leader),
      "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// One MMA with A in shared memory, and one with A in tensor memory, by one lane.
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred l, p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 l, %0, 0;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%2, %4};\n\tmov.b64 b, {%3, %4};\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %5, p;\n\t}" ::"r"(leader),
      "r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred l, p;\n\t.reg .b64 b;\n\tsetp.ne.b32 l, %0, 0;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], b, %5, p;\n\t}" ::"r"(leader),
      "r"(d), "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  return (static_cast<uint64_t>(__float_as_uint(b)) << 32) | __float_as_uint(a);
}
__device__ __forceinline__ float lo2(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi2(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }

__device__ __forceinline__ float f32_of(uint32_t v, bool f16) {
  return f16 ? __half2float(__ushort_as_half(static_cast<uint16_t>(v))) : __uint_as_float(v << 16);
}
__device__ __forceinline__ uint32_t e4m3x2_half2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
  return r;
}

// Byte offset of 16-byte piece c of row r in an operand tile: 64 values (128 bytes) of
// a row are swizzled, the next 64 lie a whole tile of rows further.
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  return static_cast<uint32_t>((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// two 16-bit values with those that are not finite set to zero
__device__ __forceinline__ uint32_t tame(uint32_t w, bool f16, uint32_t& odd) {
  const uint32_t e = f16 ? 0x7C00u : 0x7F80u;
  if ((w & e) == e) {
    odd = 1;
    w &= 0xFFFF0000u;
  }
  if ((w >> 16 & e) == e) {
    odd = 1;
    w &= 0xFFFFu;
  }
  return w;
}

// Where key j of sequence b lies: page and place in it; false for a page outside.
__device__ __forceinline__ bool locate(const AttnArgs& a, const Seq& s, int b, int j, int64_t& page, int64_t& place) {
  if (a.page_table == nullptr) {
    page = 0;
    place = static_cast<int64_t>(s.row0) + j;
    return true;
  }
  const int p = a.page_table[b * a.table_stride + (j >> a.page_shift)];
  page = p;
  place = j & ((1 << a.page_shift) - 1);
  return p >= 0 && p < a.num_pages;
}

// DP: D rounded up to 64 or 128; the products are of that depth and width.
template <bool E4M3, int DP>
__global__ void __launch_bounds__(kThreads<E4M3>, 1)
attention_kernel(const __grid_constant__ Maps maps, const __grid_constant__ AttnArgs a, const int slots, const int box_rows) {
  extern __shared__ __align__(1024) uint8_t attn_smem[];
  constexpr int kChunks = DP / 64;
  constexpr uint32_t kTile = tile_bytes(DP);
  const uint32_t base = smem_u32(attn_smem);
  const uint32_t qbase = base + kMiscBytes<E4M3>, ring = qbase + 2u * kTile;
#define FULL(s) (base + 8u * static_cast<uint32_t>(s))
#define EMPTY(s) (base + 64u + 8u * static_cast<uint32_t>(s))
#define QFULL(i) (base + 128u + 8u * static_cast<uint32_t>(i))
#define SFULL(i) (base + 144u + 8u * static_cast<uint32_t>(i))
#define PFULL(i) (base + 160u + 8u * static_cast<uint32_t>(i))
#define OFULL(i) (base + 176u + 8u * static_cast<uint32_t>(i))
#define SCFULL(s) (base + 192u + 8u * static_cast<uint32_t>(s))
#define SCEMPTY(s) (base + 208u + 8u * static_cast<uint32_t>(s))
#define READY(s) (base + 320u + 8u * static_cast<uint32_t>(s))
  const uint32_t drain = base + 232u, join0 = base + 384u, join1 = base + 392u;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(attn_smem + 240);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(attn_smem + 244);
  volatile int* last_flag = reinterpret_cast<volatile int*>(attn_smem + 248);
  volatile int* dirty = reinterpret_cast<volatile int*>(attn_smem + 256);  // [kDirty]: the item that has such values
  int64_t* scratch = reinterpret_cast<int64_t*>(attn_smem + 512);
  float* scales = reinterpret_cast<float*>(attn_smem + kBarBytes);  // [slot]: of 128 keys, of their values, unit, shrink
  constexpr int kScaleSlot = 2 * kKeys + 4;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool f16 = E4M3 || a.f16;  // of the products

  if (tid == 0) {
    for (int s = 0; s < kMaxSlots; ++s) {
      mbar_init(FULL(s), E4M3 ? kConverters : 1u);
      mbar_init(EMPTY(s), 1u);
      mbar_init(READY(s), kGuards);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(QFULL(i), 4u);
      mbar_init(SFULL(i), 1u);
      mbar_init(PFULL(i), 4u);
      mbar_init(OFULL(i), 1u);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(SCFULL(s), 1u);
      mbar_init(SCEMPTY(s), 8u);
    }
    mbar_init(join0, 8u);
    mbar_init(join1, 1u);
    mbar_init(drain, 1u);
    for (int i = 0; i < kDirty; ++i) dirty[i] = -1;
    *abort_flag = 0;
    fence_mbar_init();
    if (!E4M3) {
      tma_prefetch_desc(&maps.k);
      tma_prefetch_desc(&maps.v);
    }
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  clear_empty_rows(a);
  BigWalk w;
  Shares shares;
  const bool some = start<kRows, kKeys, kThreads<E4M3>>(a, scratch, w, shares);

  // rows of half i in an item, and the end of its key tiles in this run
  auto rows_of = [&](const BigWalk& x) { return x.s.n * a.G - x.r * kRows; };
  auto end_of = [&](const BigWalk& x, int i) {
    if (rows_of(x) <= i * kHalf) return x.t;
    return max(x.t, min(x.end, key_tiles<kHalf, kKeys>(x.s, a.G, 2 * x.r + i)));
  };
  // the last key that every row of the item sees
  auto least_of = [&](const BigWalk& x) { return x.s.past + divided(x.r * kRows, a.G); };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(E4M3 ? kLeanRegs8 : kLeanRegs16));
    bool ok = true;
    if (some && warp == 8 && !E4M3) {
      // ------------------------------------------------------ TMA producer
      const uint32_t leader = elect_one();
      const bool paged = a.page_table != nullptr;
      const int boxes = kKeys / box_rows, box_shift = 31 - __clz(box_rows);
      int st = 0, issued = 0;
      uint32_t ph = 0;
      // lane i: the page of the tile's i-th box
      auto page_of = [&](const BigWalk& x, int t) {
        const int key = t * kKeys + (lane << box_shift);
        int p = 0;
        if (paged && lane < boxes && key < x.s.L) {
          p = a.page_table[x.b * a.table_stride + (key >> a.page_shift)];
          if (p < 0 || p >= a.num_pages) {
            record_error(a.err, kErrBadIndex, static_cast<uint32_t>(x.b));
            p = a.num_pages;  // (outside the map: read as zeros)
          }
        }
        return p;
      };
      int page = page_of(w, w.t);
      for (bool more = true; more && ok;) {
        int t = w.t;
        const int end = w.end, b_h = w.h;
        const Seq s = w.s;
        BigWalk next = w;
        more = next.next(a);
        for (; t < end && ok; ++t) {
          const int mine = page;
          if (t + 1 < end) page = page_of(w, t + 1);
          else if (more) page = page_of(next, next.t);
          const int key0 = t * kKeys, there = min(boxes, (s.L - key0 + box_rows - 1) >> box_shift);
#pragma unroll 1
          for (int kv = 0; kv < 2 && ok; ++kv) {
            ok = wait(EMPTY(st), ph ^ 1u, abort_flag, a.err, 0x700u);
            if (!ok) break;
            const uint32_t dst = ring + static_cast<uint32_t>(st) * kTile;
            expect_tx(leader, FULL(st), static_cast<uint32_t>(there * box_rows * 128 * kChunks));
            for (int i = 0; i < there; ++i) {
              const int p = __shfl_sync(0xffffffffu, mine, i);
              const int row = paged ? (key0 + (i << box_shift)) & ((1 << a.page_shift) - 1) : s.row0 + key0;
#pragma unroll
              for (int c = 0; c < kChunks; ++c)
                load_box4(leader, dst + static_cast<uint32_t>(c * 128 * 128 + ((i << box_shift) * 128)),
                          kv == 0 ? &maps.k : &maps.v, FULL(st), 64 * c, row, b_h, p);
            }
            ++issued;
            if (++st == slots) {
              st = 0;
              ph ^= 1u;
            }
          }
        }
        w = next;
      }
      if (!ok) {  // after an abort the loads in flight land before the CTA leaves
        for (int i = min(issued, slots); i > 0; --i) {
          st = st == 0 ? slots - 1 : st - 1;
          if (st == slots - 1) ph ^= 1u;
          wait(FULL(st), ph, nullptr, a.err, 0x701u);
        }
      }
    } else if (some && warp == 8) {
      // ------------------------------------ 8-bit: scales of a tile's keys and values
      // four keys a lane; the values' relative to the largest so far, rounded up to
      // a power of two
      uint32_t n = 0;
      for (bool more = true; more && ok;) {
        float unit = 0.f;
        for (int t = w.t; t < w.end; ++t, ++n) {
          const uint32_t slot = n % kScaleSlots;
          const int key = t * kKeys + 4 * lane;
          float4 ks = make_float4(0.f, 0.f, 0.f, 0.f), vs = ks;
          if (key < w.s.L) {
            int64_t page, place;
            if (locate(a, w.s, w.b, key, page, place)) {
              const int64_t at = ((page * a.Hkv + w.h) << a.page_shift) + place;
              ks = *reinterpret_cast<const float4*>(a.kv.k_scale + at);
              vs = *reinterpret_cast<const float4*>(a.kv.v_scale + at);
            }
          }
          float most = 0.f;
          const float each[4] = {vs.x, vs.y, vs.z, vs.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key + e < w.s.L && fabsf(each[e]) < INFINITY) most = fmaxf(most, fabsf(each[e]));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
          float shrink = 1.f;
          if (most >= unit) {
            const float grown = __uint_as_float(min((__float_as_uint(most) & 0x7F800000u) + 0x00800000u, 0x7F000000u));
            if (grown > unit) {
              shrink = unit / grown;
              unit = grown;
            }
          }
          const float per = 1.f / unit;
          ok = wait(SCEMPTY(slot), (n / kScaleSlots & 1u) ^ 1u, abort_flag, a.err, 0x710u);
          if (!ok) break;
          float* to = scales + slot * kScaleSlot;
          *reinterpret_cast<float4*>(to + 4 * lane) = ks;
          *reinterpret_cast<float4*>(to + kKeys + 4 * lane) = make_float4(vs.x * per, vs.y * per, vs.z * per, vs.w * per);
          if (lane == 0) {
            to[2 * kKeys] = unit;
            to[2 * kKeys + 1] = shrink;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(SCFULL(slot));
        }
        more = ok && w.next(a);
      }
    } else if (some && warp == 9) {
      // -------------------------------------------------------- MMA issuer
      const uint32_t leader = elect_one();
      const uint32_t fmt = f16 ? 0u : 1u;
      const uint32_t idesc_s = make_idesc(128u, kKeys, fmt), idesc_o = make_idesc(128u, DP, fmt) | (1u << 16);
      const uint64_t kd = sw128_kmajor_desc(qbase);
      const uint32_t hi = static_cast<uint32_t>(kd >> 32);
      const uint32_t low = static_cast<uint32_t>(kd) & ~0x3FFFu;  // (its address is added below)
      // values, read along the head: 64 of them a swizzled row, the next 64 a tile of
      // rows further (leading offset), 8 keys 1024 bytes apart (stride offset)
      const uint32_t v_low = ((128u * 128u) >> 4) << 16;
      auto addr = [&](uint32_t p) { return (p & 0x3FFFFu) >> 4; };
      auto scores = [&](int i, uint32_t tile) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(leader, tmem + 128u * i, low | (addr(qbase + i * kTile + c * 16384u) + 2u * k),
                   low | (addr(tile + c * 16384u) + 2u * k), hi, idesc_s, (c | k) != 0);
        commit<false>(leader, SFULL(i));
      };
      auto outputs = [&](int i, uint32_t tile, bool first) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ts(leader, tmem + kOut + 128u * i, tmem + 128u * i + 8u * k, v_low | (addr(tile) + 128u * k), hi, idesc_o,
                 !(first && k == 0));
      };
      int st = 0;
      uint32_t ph = 0, pph[2] = {0, 0}, qph[2] = {0, 0};
      bool any = false;
      auto step = [&] {
        if (++st == slots) {
          st = 0;
          ph ^= 1u;
        }
      };
      // a tile is there (16-bit: and looked at, in which the others' wait lies already)
      auto there = [&](uint32_t info) {
        return (E4M3 || wait(READY(st), ph, abort_flag, a.err, info)) && wait(FULL(st), ph, abort_flag, a.err, info);
      };
      auto tile_at = [&](int s) { return ring + static_cast<uint32_t>(s) * kTile; };
      for (bool more = true; more && ok;) {
        const int e[2] = {end_of(w, 0), end_of(w, 1)};
        for (int i = 0; i < 2 && ok; ++i)
          if (w.t < e[i]) {
            ok = wait(QFULL(i), qph[i], abort_flag, a.err, 0x720u);
            qph[i] ^= 1u;
          }
        ok = ok && there(0x721u);
        if (!ok) break;
        tc_fence_after();
        any = true;
        for (int i = 0; i < 2; ++i)
          if (w.t < e[i]) scores(i, tile_at(st));
        commit<false>(leader, EMPTY(st));
        step();
        for (int t = w.t; t < w.end && ok; ++t) {
          const int vs = st;
          ok = there(0x722u);
          step();
          const int ks = st;
          const bool again = t + 1 < w.end;
          if (again) {
            ok = ok && there(0x724u);
            step();
          }
          for (int i = 0; i < 2 && ok; ++i) {
            if (t < e[i]) {
              ok = wait(PFULL(i), pph[i], abort_flag, a.err, 0x725u);
              if (!ok) break;
              pph[i] ^= 1u;
              tc_fence_after();
              outputs(i, tile_at(vs), t == w.t);
              if (t + 1 >= e[i]) commit<false>(leader, OFULL(i));
            }
            if (i == 1) commit<false>(leader, EMPTY(vs));
            if (t + 1 < e[i]) scores(i, tile_at(ks));
          }
          if (again && ok) commit<false>(leader, EMPTY(ks));
        }
        more = ok && w.next(a);
      }
      if (!ok && any) {  // MMAs in flight end before tensor memory is freed
        if (leader != 0u) mma_commit(drain);
        wait(drain, 0u, nullptr, a.err, 0x730u);
      }
    } else if (some && !E4M3) {
      // ------------------- 16-bit: values of tiles that some row does not wholly see
      const int me = (warp - 10) * 32 + lane;
      int st = 0, item = 0;
      uint32_t ph = 0;
      for (bool more = true; more && ok; ++item) {
        const int least = least_of(w);
        for (int u = 2 * w.t; u < 2 * w.end; ++u) {  // keys, values
          const int t = u >> 1;
          ok = wait(FULL(st), ph, abort_flag, a.err, 0x740u);
          if (!ok) break;
          if ((u & 1) != 0 && t * kKeys + kKeys - 1 > least) {
            const uint32_t tile = ring + static_cast<uint32_t>(st) * kTile;
            const int there = min(kKeys, w.s.L - t * kKeys);
            uint32_t odd = 0;
#pragma unroll 4
            for (int i = me; i < kKeys * DP / 8; i += 32 * kGuards) {
              const int r = i / (DP / 8), c = i % (DP / 8);
              const uint32_t at = tile + piece_at(r, c);
              if (r >= there) {
                dense::sts_u4(at, make_uint4(0, 0, 0, 0));
              } else {
                const uint4 v = dense::lds_u4(at);
                uint32_t bad = 0;
                const uint4 x = make_uint4(tame(v.x, f16, bad), tame(v.y, f16, bad), tame(v.z, f16, bad), tame(v.w, f16, bad));
                if (bad) dense::sts_u4(at, x);
                odd |= bad;
              }
            }
            if (odd) dirty[item % kDirty] = item;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(READY(st));
          if (++st == slots) {
            st = 0;
            ph ^= 1u;
          }
        }
        more = ok && w.next(a);
      }
    } else if (some) {
      // ------------------------------------------- 8-bit: codes into f16 tiles
      // Thread j takes 16-byte pieces j, j + 192, ... of a tile (lanes go along a
      // row); a tile's codes are fetched before the wait for the place they go to.
      constexpr int kPer = kKeys * DP / 16, kT = 32 * kConverters, kMine = (kPer + kT - 1) / kT, kRowPieces = DP / 16;
      const int me = (warp - 10) * 32 + lane;
      int st = 0, item = 0;
      uint32_t ph = 0;
      uint4 next[kMine];
      auto fetch = [&](const BigWalk& x, int t, int kv) {
        // lane i < 8: the page of keys 16 i .. of the tile
        const int key0 = t * kKeys;
        int p = 0;
        if (lane < 8 && key0 + 16 * lane < x.s.L) {
          p = a.page_table[x.b * a.table_stride + ((key0 + 16 * lane) >> a.page_shift)];
          if (p < 0 || p >= a.num_pages) {
            record_error(a.err, kErrBadIndex, static_cast<uint32_t>(x.b));
            p = -1;
          }
        }
        const uint8_t* from = kv == 0 ? a.kv.k : a.kv.v;
        const int64_t ps = kv == 0 ? a.kv.k_page : a.kv.v_page, ts = kv == 0 ? a.kv.k_token : a.kv.v_token;
        from += x.h * (kv == 0 ? a.kv.k_head : a.kv.v_head);
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          const int i = me + j * kT, r = i / kRowPieces, c = i % kRowPieces;
          const int page = __shfl_sync(0xffffffffu, p, (r >> 4) & 7);
          const bool there = i < kPer && key0 + r < x.s.L && page >= 0 && 16 * c < a.D;
          next[j] = there ? *reinterpret_cast<const uint4*>(from + page * ps +
                                                            ((key0 + r) & ((1 << a.page_shift) - 1)) * ts + 16 * c)
                          : make_uint4(0, 0, 0, 0);
        }
      };
      fetch(w, w.t, 0);
      for (bool more = true; more && ok; ++item) {
        const int least = least_of(w);
        BigWalk after = w;
        more = after.next(a);
#pragma unroll 1
        for (int u = 2 * w.t; u < 2 * w.end; ++u) {
          const int t = u >> 1, kv = u & 1;
          ok = wait(EMPTY(st), ph ^ 1u, abort_flag, a.err, 0x750u);
          if (!ok) break;
          const uint32_t tile = ring + static_cast<uint32_t>(st) * kTile;
          const bool partly = kv == 1 && t * kKeys + kKeys - 1 > least;
          uint32_t odd = 0;
#pragma unroll
          for (int j = 0; j < kMine; ++j) {
            const int i = me + j * kT, r = i / kRowPieces, c = i % kRowPieces;
            if (i >= kPer) break;
            const uint32_t q[4] = {next[j].x, next[j].y, next[j].z, next[j].w};
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              h[2 * e] = e4m3x2_half2(q[e] & 0xFFFFu);
              h[2 * e + 1] = e4m3x2_half2(q[e] >> 16);
            }
            if (partly) {
#pragma unroll
              for (int e = 0; e < 8; ++e) h[e] = tame(h[e], true, odd);
            }
            // (lanes 4 to 7 of a row's eight begin with their second piece: other banks)
            const uint4 u0 = make_uint4(h[0], h[1], h[2], h[3]), u1 = make_uint4(h[4], h[5], h[6], h[7]);
            const int swap = c >> 2 & 1;
            dense::sts_u4(tile + piece_at(r, 2 * c + swap), swap ? u1 : u0);
            dense::sts_u4(tile + piece_at(r, 2 * c + 1 - swap), swap ? u0 : u1);
          }
          if (odd) dirty[item % kDirty] = item;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(FULL(st));
          if (++st == slots) {
            st = 0;
            ph ^= 1u;
          }
          if (u + 1 < 2 * w.end) fetch(w, (u + 1) >> 1, kv ^ 1);
          else if (more) fetch(after, after.t, 0);
        }
        w = after;
      }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(E4M3 ? kLaunchRegs8 : kLaunchRegs16));
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(E4M3 ? kSoftRegs8 : kSoftRegs16));
    // ------------------------------------------------------------- softmax
    const int half = warp >> 2, row = tid & (kHalf - 1);
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t S = tmem + 128u * half + lanes, O = tmem + kOut + 128u * half + lanes;
    const uint32_t q_at = qbase + static_cast<uint32_t>(half) * kTile;
    uint32_t sph = 0, oph = 0, scn = 0, jph = 0;
    bool ok = true;
    int item = 0;
    // this thread's row of an item
    struct Row {
      bool live;
      int limit;  // the last key that it sees
      int64_t token;
      int head;
    };
    auto row_of = [&](const BigWalk& x) {
      Row y;
      y.live = half * kHalf + row < rows_of(x);
      const int R = x.r * kRows + (y.live ? half * kHalf + row : 0);
      const int tok = divided(R, a.G);
      y.limit = x.s.past + tok;
      y.token = x.s.row0 + tok;
      y.head = x.h * a.G + R - tok * a.G;
      return y;
    };
    // Its queries into shared memory; what their scores are multiplied with.  8-bit:
    // as f16, the largest brought to 2^14.
    auto put_queries = [&](const Row& y) {
      const uint16_t* q = a.q + y.token * a.q_stride + static_cast<int64_t>(y.head) * a.D;
      uint4 v[DP / 8];
#pragma unroll
      for (int c = 0; c < DP / 8; ++c)
        v[c] = y.live && 8 * c < a.D ? *reinterpret_cast<const uint4*>(q + 8 * c) : make_uint4(0, 0, 0, 0);
      float factor = a.scale_log2;
      if (E4M3) {
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < DP / 8; ++c) {
          const uint32_t u[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(f32_of(u[e] & 0xFFFFu, a.f16)), fabsf(f32_of(u[e] >> 16, a.f16))));
        }
        const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100), 126);
        const bool scaled = amax > 0.f && amax < INFINITY;
        const float up = scaled ? __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23) : 1.f;
        if (scaled) factor *= __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
#pragma unroll
        for (int c = 0; c < DP / 8; ++c) {
          uint32_t* u = &v[c].x;
#pragma unroll
          for (int k = 0; k < 4; ++k) u[k] = pack_half(f32_of(u[k] & 0xFFFFu, a.f16) * up, f32_of(u[k] >> 16, a.f16) * up);
        }
      }
#pragma unroll
      for (int c = 0; c < DP / 8; ++c) dense::sts_u4(q_at + piece_at(row, c), v[c]);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(QFULL(half));
      return factor;
    };
    Row y{};
    float factor = a.scale_log2;
    if (some) {
      y = row_of(w);
      if (w.t < end_of(w, half)) factor = put_queries(y);
    }
    for (bool more = some; more && ok; ++item) {
      const int end = end_of(w, half), t0 = w.t;
      // the first key that some row of this half does not see
      const int least = w.s.past + divided(w.r * kRows + half * kHalf, a.G);
      float top = -INFINITY;  // of the row's scores, what its weights are relative to
      float unit = 1.f;
      uint64_t sum = 0;
      BigWalk next = w;
      more = next.next(a);
      Row y_next = y;
      float factor_next = factor;
      for (int t = t0; t < (E4M3 ? w.end : end) && ok; ++t) {
        const float* sc = nullptr;
        uint32_t slot = 0;
        if (E4M3) {
          slot = scn % kScaleSlots;
          ok = wait(SCFULL(slot), scn / kScaleSlots & 1u, abort_flag, a.err, 0x760u);
          ++scn;
          if (!ok) break;
          sc = scales + slot * kScaleSlot;
          if (t >= end) {  // (the other half's tile)
            __syncwarp();
            if (lane == 0) mbar_arrive_cta(SCEMPTY(slot));
            continue;
          }
          unit = sc[2 * kKeys];
        }
        ok = wait(SFULL(half), sph, abort_flag, a.err, 0x761u);
        if (!ok) break;
        sph ^= 1u;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) dense::tmem_ld32(S + 32u * c, s[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) dense::tmem_ld32_wait(s[c]);
        if (E4M3) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 k = *reinterpret_cast<const float4*>(sc + 32 * c + 4 * j);
              const float kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) s[c][4 * j + e] = __float_as_uint(__uint_as_float(s[c][4 * j + e]) * kk[e]);
            }
        }
        if (t * kKeys + kKeys - 1 > least) {
          const int seen = y.limit - t * kKeys;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * c + j > seen) s[c][j] = __float_as_uint(-INFINITY);
        }
        float m4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          m4[c] = __uint_as_float(s[c][0]);
#pragma unroll
          for (int j = 1; j < 32; ++j) m4[c] = fmaxf(m4[c], __uint_as_float(s[c][j]));
        }
        const float now = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * factor;
        const float shrink = E4M3 ? sc[2 * kKeys + 1] : 1.f;
        if (t == t0) {
          top = fmaxf(top, now);  // (NaN leaves it)
        } else if (__any_sync(0xffffffffu, now > top + 8.f) || shrink != 1.f) {
          // O of the tiles before is complete: their products precede these scores
          const float up = fmaxf(top, now), keep = exp2_fast(top - reference(up));
          top = up;
          sum = mul2(sum, pack2(keep, keep));
          const float f = keep * shrink;
#pragma unroll
          for (int c = 0; c < DP / 32; ++c) {
            uint32_t o[32];
            dense::tmem_ld32(O + 32u * c, o);
            dense::tmem_ld32_wait(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st32(O + 32u * c, o);
          }
        }
        const float r = reference(top);
        const uint64_t f2 = pack2(factor, factor), r2 = pack2(-r, -r);
        uint64_t sums[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t p[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const uint32_t* x = &s[2 * c + (j >> 4)][2 * (j & 15)];
            const uint64_t z = fma2((static_cast<uint64_t>(x[1]) << 32) | x[0], f2, r2);
            uint64_t e = pack2(exp2_fast(lo2(z)), exp2_fast(hi2(z)));
            sums[j & 1] = add2(sums[j & 1], e);
            if (E4M3) {
              const float2 v = *reinterpret_cast<const float2*>(sc + kKeys + 64 * c + 2 * j);
              // (a weight of zero stays zero whatever its value's scale is)
              e = pack2(lo2(e) == 0.f ? 0.f : lo2(e) * v.x, hi2(e) == 0.f ? 0.f : hi2(e) * v.y);
            }
            p[j] = f16 ? pack_half(lo2(e), hi2(e)) : pack_bf16x2(lo2(e), hi2(e));
          }
          tmem_st32(S + 32u * c, p);
        }
        sum = add2(sum, add2(sums[0], sums[1]));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_cta(PFULL(half));
          if (E4M3) mbar_arrive_cta(SCEMPTY(slot));
        }
        // the item's last scores are read: the next item's queries may come
        if (t + 1 == end && more) {
          y_next = row_of(next);
          if (next.t < end_of(next, half)) factor_next = put_queries(y_next);
        }
      }
      if (!ok) break;
      const bool has = t0 < end;
      if (!has && more) {
        y_next = row_of(next);
        if (next.t < end_of(next, half)) factor_next = put_queries(y_next);
      }
      // ---- the item's end
      float total = lo2(sum) + hi2(sum);
      if (has) {
        ok = wait(OFULL(half), oph, abort_flag, a.err, 0x762u);
        if (!ok) break;
        oph ^= 1u;
        tc_fence_after();
      }
      const bool spoiled = dirty[item % kDirty] == item;
      const bool whole = w.end - w.t == w.len;
      const int first = t0 > 0 ? shares.first : static_cast<int>(blockIdx.x);
      constexpr size_t kPiece = attn_piece_bytes(kRows, DP) / 4;
      auto piece = [&](int i) { return a.partial + (2 * (first + i) + (i == 0 ? 1 : 0)) * kPiece + half * kHalf + row; };
      uint16_t* to = a.out + y.token * a.out_stride + static_cast<int64_t>(y.head) * a.D;
      auto write = [&](int c, const float (&v)[32], float inv) {  // 32 columns of the row
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (32 * c + 8 * j < a.D) {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              u[e] = a.f16 ? pack_half(v[8 * j + 2 * e] * inv, v[8 * j + 2 * e + 1] * inv)
                           : pack_bf16x2(v[8 * j + 2 * e] * inv, v[8 * j + 2 * e + 1] * inv);
            *reinterpret_cast<uint4*>(to + 32 * c + 8 * j) = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
      };
      float* mine = piece(static_cast<int>(blockIdx.x) - first);
      const float inv = 1.f / total;
#pragma unroll 1
      for (int c = 0; c < DP / 32; ++c) {
        float v[32];
        if (has) {
          uint32_t o[32];
          dense::tmem_ld32(O + 32u * c, o);
          dense::tmem_ld32_wait(o);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(o[j]) * (E4M3 ? unit : 1.f);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.f;
        }
        if (spoiled && y.live && has) {
          // values that are not finite, of the keys that this row sees among those looked at
          const int from = max(t0, (least_of(w) + 1) / kKeys) * kKeys;
          for (int key = from; key <= min(y.limit, end * kKeys - 1); ++key) {
            int64_t page, place;
            if (!locate(a, w.s, w.b, key, page, place)) continue;
            const int64_t in = page * a.kv.v_page + place * a.kv.v_token + w.h * a.kv.v_head + 32 * c;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (32 * c + j >= a.D) break;
              const float x = E4M3 ? ((a.kv.v[in + j] & 0x7F) == 0x7F ? NAN : 0.f)
                                   : f32_of(reinterpret_cast<const uint16_t*>(a.kv.v)[in + j], a.f16);
              if (!(fabsf(x) < INFINITY)) v[j] += x;
            }
          }
        }
        if (whole) {
          if (y.live) write(c, v, inv);
        } else if (y.live) {
#pragma unroll
          for (int j = 0; j < 32; ++j) __stcg(mine + (32 * c + j) * kRows, v[j]);
        }
      }
      tc_fence_before();  // (the next item's products write O after this half's weights)
      if (whole) {
        if (y.live && a.lse != nullptr) a.lse[y.token * a.Hq + y.head] = (top + log2_fast(total)) * 0.69314718055994531f;
      } else {
        // the item lies in several runs: the last one to finish joins them
        if (y.live) {
          __stcg(mine + DP * kRows, top);
          __stcg(mine + (DP + 1) * kRows, total);
        }
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(join0);
        ok = wait(join0, jph, abort_flag, a.err, 0x770u);
        if (!ok) break;
        const int pieces = shares.pieces(first, w.len - w.end);
        if (tid == 0) {
          const bool last = atomicAdd(a.tickets + first, 1u) == static_cast<uint32_t>(pieces - 1);
          if (last) a.tickets[first] = 0;
          __threadfence();
          *last_flag = last;
          mbar_arrive_cta(join1);
        }
        ok = wait(join1, jph, abort_flag, a.err, 0x771u);
        if (!ok) break;
        jph ^= 1u;
        if (*last_flag != 0 && y.live) {
          __threadfence();
          float m = -INFINITY;
          for (int i = 0; i < pieces; ++i) m = fmaxf(m, __ldcg(piece(i) + DP * kRows));
          const float r = reference(m);
          float l = 0.f;
          for (int i = 0; i < pieces; ++i) l = fmaf(__ldcg(piece(i) + (DP + 1) * kRows), exp2_fast(__ldcg(piece(i) + DP * kRows) - r), l);
#pragma unroll 1
          for (int c = 0; c < DP / 32; ++c) {
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.f;
#pragma unroll 1
            for (int i = 0; i < pieces; ++i) {
              const float f = exp2_fast(__ldcg(piece(i) + DP * kRows) - r);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = fmaf(__ldcg(piece(i) + (32 * c + j) * kRows), f, v[j]);
            }
            write(c, v, 1.f / l);
          }
          if (a.lse != nullptr) a.lse[y.token * a.Hq + y.head] = (m + log2_fast(l)) * 0.69314718055994531f;
        }
      }
      w = next;
      y = y_next;
      factor = factor_next;
    }
    __syncwarp();
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(E4M3 ? kLaunchRegs8 : kLaunchRegs16));
    tc_fence_before();
    __syncthreads();
  }
#undef FULL
#undef EMPTY
#undef QFULL
#undef SFULL
#undef PFULL
#undef OFULL
#undef SCFULL
#undef SCEMPTY
#undef READY
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <bool E4M3, int DP>
cudaError_t launch(const AttnArgs& a, int sms, cudaStream_t s) {
  auto kernel = attention_kernel<E4M3, DP>;
  static int configured[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64 || configured[dev] == 0) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (err != cudaSuccess) return err;
    cudaFuncAttributes attr;
    err = cudaFuncGetAttributes(&attr, kernel);
    if (err != cudaSuccess) return err;
    // the warps' register counts add up to the launch's only if it has these, and
    // the tiles are aligned only if nothing lies before them
    if (attr.numRegs != (E4M3 ? kLaunchRegs8 : kLaunchRegs16) || attr.sharedSizeBytes != 0)
      return cudaErrorInvalidConfiguration;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  const int room = static_cast<int>((kSmem - kMiscBytes<E4M3>) / tile_bytes(DP)) - 2;
  const int slots = room < kMaxSlots ? room : kMaxSlots;
  const size_t smem = std::max(kTensorMemorySmem, static_cast<size_t>(kMiscBytes<E4M3> + (2 + slots) * tile_bytes(DP)));
  Maps maps = {};
  int box_rows = kKeys;
  if (!E4M3) {
    const bool paged = a.page_table != nullptr;
    const uint64_t page = paged ? 1ull << a.page_shift : static_cast<uint64_t>(a.T);
    box_rows = paged && page < kKeys ? static_cast<int>(page) : kKeys;
    const CUtensorMapDataType dt = a.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t dims[4] = {static_cast<uint64_t>(a.D), page, static_cast<uint64_t>(a.Hkv), static_cast<uint64_t>(a.num_pages)};
    const uint32_t box[4] = {64, static_cast<uint32_t>(box_rows), 1, 1};
    const int64_t far = 16;  // (of one page: no stride)
    const uint64_t ks[3] = {static_cast<uint64_t>(2 * a.kv.k_token), static_cast<uint64_t>(2 * a.kv.k_head),
                            static_cast<uint64_t>(paged ? 2 * a.kv.k_page : far)};
    const uint64_t vs[3] = {static_cast<uint64_t>(2 * a.kv.v_token), static_cast<uint64_t>(2 * a.kv.v_head),
                            static_cast<uint64_t>(paged ? 2 * a.kv.v_page : far)};
    if (!encode_map(&maps.k, dt, 4, a.kv.k, dims, ks, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_map(&maps.v, dt, 4, a.kv.v, dims, vs, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  return launch_pdl(kernel, dim3(sms < kAttnMaxCtas ? sms : kAttnMaxCtas), dim3(kThreads<E4M3>), smem, s, maps, a, slots,
                    box_rows);
}

}  // namespace

cudaError_t launch_attention(const AttnArgs& a, int sms, cudaStream_t s) {
  if (a.e4m3) return a.D <= 64 ? launch<true, 64>(a, sms, s) : launch<true, 128>(a, sms, s);
  return a.D <= 64 ? launch<false, 64>(a, sms, s) : launch<false, 128>(a, sms, s);
}

}  // namespace moe
