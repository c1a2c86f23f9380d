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
// threads), 8 loads (TMA, a box a page and 128 bytes of its rows), 9 MMAs; 16-bit: 10
// and 11 look at the values of tiles that some row does not wholly see; 8-bit: 10
// the tiles' scales (a value's counts in its row's maximum: scale_log2), 12 to 15 turn
// codes, which TMA left in a ring of their own, into f16 tiles.
//
// The running maximum is only raised, and O rescaled, when it grew by more than 8
// (factors of 2^8 stay far inside the sums' and the weights' range), which is rare
// after the first tiles.  A row's result does not depend on it but for roundings.  f16
// weights are 2^7 times those relative to it, so that they reach 2^15: those under f16's
// normal range then weigh 2^-21 of the largest and less (8-bit 2^-17, kClose), where 2^-14
// showed beside a key that takes nearly all of the weight and adds nothing.
//
// Masked scores become -inf whatever they were.  Values behind the sequence's end
// are zeroed in shared memory, and values that are not finite in a tile that some row
// does not wholly see are taken out there and added at the end to the rows that do
// see them: 0 * NaN would reach the others.
//
// Bound by the softmax's chain (scores from tensor memory, maximum, exponentials,
// weights back), which the other half's products overlap: tensor pipe 65%, issue slots
// 42% busy.  In a graph, 32 query and 8 key heads of 128, bf16: one prompt of 8192
// tokens 365 us = 1.5 PFLOP/s, a chunk of 2048 after 6000 tokens 170; over an e4m3
// cache 249, where the converters' shared-memory traffic and the scales are added (28 + 4
// heads, 2048 after 30000: 830 us = 1.10 PFLOP/s; heads of 64, 8 key heads, 2048 after
// 6000 219).  Tiles of 128 keys and two halves
// fill tensor memory's 512 columns.  All code of an instance stays under 128 KB, what
// the instruction cache holds: at 149 KB the e4m3 one took twice its time.
#include "attention.cuh"
#include "dense.cuh"
#include "stream.cuh"

namespace moe {
namespace {

using namespace attn;
using dense::commit;
using dense::elect_one;
using dense::expect_tx;
using dense::mbar_arrive_cta;

constexpr int kHalf = 128, kRows = 2 * kHalf, kKeys = 128;
constexpr int kMaxSlots = 8, kScaleSlots = 2, kDirty = 16;
constexpr size_t kSmem = 232448;
// Registers a thread of the softmax's warpgroups and of the others; 3 x 168 and 4 x
// 128 at launch.
constexpr int kSoftRegs16 = 200, kLeanRegs16 = 104, kLaunchRegs16 = 168;
constexpr int kSoftRegs8 = 192, kLeanRegs8 = 64, kLaunchRegs8 = 128;
template <bool E4M3>
constexpr int kThreads = E4M3 ? 512 : 384;
constexpr int kGuards = 2, kConverters = 4;  // warps from 10, from 12 on
constexpr uint32_t kTmemCols = 512, kOut = 256;  // scores of half i at 128 i, outputs at 256 + 128 i

using BigWalk = Walk<Shape<kRows, kKeys, 3, 3, 4>>;

// Barriers and small arrays, then (1024-byte aligned) Q's halves, the ring of key and
// value tiles and the ring of their codes.
constexpr int kBarBytes = 640;
constexpr int kScaleSlot = 3 * kKeys + 4;  // of 128 keys, of their values, the latter's logarithms (scale_log2), the tile's
constexpr int kItems = 4;
// An item as its warps see it: end is of its key tiles in this run, end0 that of the
// first half's; least the last key that all rows see.
struct Item {
  int b, h, r, t, end, len, row0, L, past, rows, least, end0, first, pieces;
};
template <bool E4M3>
constexpr int kMiscBytes = E4M3 ? 4 * 1024 : 1024;
template <bool E4M3>
constexpr int kItemsAt = kBarBytes + (E4M3 ? kScaleSlots * kScaleSlot * 4 : 0);
static_assert(kItemsAt<true> + kItems * sizeof(Item) <= kMiscBytes<true> &&
                  kItemsAt<false> + kItems * sizeof(Item) <= kMiscBytes<false>,
              "all before Q");
__host__ __device__ constexpr int tile_bytes(int dp) { return kKeys * dp * 2; }
__host__ __device__ constexpr int code_bytes(int dp) { return kKeys * dp; }
// the codes' ring: what three f16 tiles leave
constexpr int kMaxCodeSlots = 4;
__host__ __device__ constexpr int code_slots(int dp) { return dp == 64 ? 4 : 3; }

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

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// dense::wait in fewer instructions (there are many waits, and the code is long for
// the instruction caches): a wait that runs out leaves `info` in the flag that ends
// all waits, and it is recorded when the roles have ended.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int info) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    if ((i & 63u) != 0u) continue;
    if (abort_flag != nullptr && *abort_flag != 0) return false;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitLimitNs) {
      if (abort_flag != nullptr) *abort_flag = info;
      return false;
    }
  }
  return true;
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
__device__ __forceinline__ bool locate(const AttnArgs& a, int row0, int b, int j, int64_t& page, int64_t& place) {
  if (a.page_table == nullptr) {
    page = 0;
    place = static_cast<int64_t>(row0) + j;
    return true;
  }
  const int p = a.page_table[b * a.table_stride + (j >> a.page_shift)];
  page = p;
  place = j & ((1 << a.page_shift) - 1);
  return p >= 0 && p < a.num_pages;
}

// How far a row's maximum grows before it is raised, and how far under it f16 weights'
// reference lies: they reach 2^15.  8-bit: where a half's rows all see a tile and its values'
// scales' logarithms differ by at most kClose, the largest of these is added to the largest
// score, at most kClose too much; else each to its key's score in another turn over the
// scores (2048 tokens after 30000, 28 + 4 heads: 830 us, scales over a range of 2^12 1074).
constexpr int kClose = 3;
constexpr float kLag = 8.f;
template <bool F16>
constexpr float kLift = F16 ? 7.f : 0.f;
static_assert(kLag + kLift<true> <= 15.f, "f16 ends below 2^16");

// DP: D rounded up to 64 or 128; the products are of that depth and width.
// F16: the products' type (8-bit: always), else bf16.
template <bool E4M3, bool F16, int DP>
__global__ void __launch_bounds__(kThreads<E4M3>, 1)
attention_kernel(const __grid_constant__ Maps maps, const __grid_constant__ AttnArgs a, const int slots, const int box_rows) {
  extern __shared__ __align__(1024) uint8_t attn_smem[];
  constexpr int kChunks = DP / 64, kCodeSlots = code_slots(DP);
  constexpr uint32_t kTile = tile_bytes(DP);
  const uint32_t base = smem_u32(attn_smem);
  const uint32_t qbase = base + kMiscBytes<E4M3>, ring = qbase + 2u * kTile;
  const uint32_t codes = ring + static_cast<uint32_t>(slots) * kTile;  // 8-bit
#define FULL(s) (base + 8u * static_cast<uint32_t>(s))
#define EMPTY(s) (base + 64u + 8u * static_cast<uint32_t>(s))
#define QFULL(i) (base + 128u + 8u * static_cast<uint32_t>(i))
#define SFULL(i) (base + 144u + 8u * static_cast<uint32_t>(i))
#define PFULL(i, part) (base + 464u + 16u * static_cast<uint32_t>(i) + 8u * static_cast<uint32_t>(part))
#define OFULL(i) (base + 176u + 8u * static_cast<uint32_t>(i))
#define SCFULL(s) (base + 192u + 8u * static_cast<uint32_t>(s))
#define SCEMPTY(s) (base + 208u + 8u * static_cast<uint32_t>(s))
#define READY(s) (base + 320u + 8u * static_cast<uint32_t>(s))
#define CFULL(s) (base + 400u + 8u * static_cast<uint32_t>(s))
#define CEMPTY(s) (base + 432u + 8u * static_cast<uint32_t>(s))
#define IFULL(s) (base + 512u + 8u * static_cast<uint32_t>(s))
#define IEMPTY(s) (base + 544u + 8u * static_cast<uint32_t>(s))
  const uint32_t drain = base + 232u, join0 = base + 384u, join1 = base + 392u;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(attn_smem + 240);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(attn_smem + 244);
  volatile int* last_flag = reinterpret_cast<volatile int*>(attn_smem + 248);
  volatile int* dirty = reinterpret_cast<volatile int*>(attn_smem + 256);  // [kDirty]: the item that has such values
  int64_t* scratch = reinterpret_cast<int64_t*>(attn_smem + kMiscBytes<E4M3>);  // (Q's place, until the roles begin)
  Item* items = reinterpret_cast<Item*>(attn_smem + kItemsAt<E4M3>);
  float* scales = reinterpret_cast<float*>(attn_smem + kBarBytes);         // [slot]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  static_assert(F16 || !E4M3, "codes become f16");

  if (tid == 0) {
    for (int s = 0; s < kMaxSlots; ++s) {
      mbar_init(FULL(s), E4M3 ? kConverters : 1u);
      mbar_init(EMPTY(s), 1u);
      mbar_init(READY(s), kGuards);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(QFULL(i), 4u);
      mbar_init(SFULL(i), 1u);
      mbar_init(PFULL(i, 0), 4u);
      mbar_init(PFULL(i, 1), 4u);
      mbar_init(OFULL(i), 1u);
    }
    for (int s = 0; s < kItems; ++s) {
      mbar_init(IFULL(s), 1u);
      mbar_init(IEMPTY(s), 9u + (E4M3 ? 1u + kConverters : kGuards));
    }
    for (int s = 0; s < kMaxCodeSlots; ++s) {
      mbar_init(CFULL(s), 1u);
      mbar_init(CEMPTY(s), kConverters);
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
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
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
  BigWalk w;
  const bool some = start<kThreads<E4M3>>(a, scratch, w);
  __syncthreads();

  // the n-th item (null after an abort; t < 0: there is none), and its release
  auto take = [&](int n) -> const Item* {
    return wait(IFULL(n % kItems), n / kItems & 1, abort_flag, 0x780) ? items + n % kItems : nullptr;
  };
  auto leave = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive_cta(IEMPTY(n % kItems));
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(E4M3 ? kLeanRegs8 : kLeanRegs16));
    bool ok = true;
    if (some && warp == 8) {
      // ------------------------------------------------------ TMA producer
      // (8-bit: of codes, into their own ring)
      const int my_slots = E4M3 ? kCodeSlots : slots;
      constexpr uint32_t kMine = E4M3 ? code_bytes(DP) : kTile, kRowBytes = E4M3 ? DP : 128u;
      constexpr int kBoxes = E4M3 ? 1 : kChunks;  // side by side
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
      int page = page_of(w, w.t), n = 0;
      for (bool more = true; more && ok; ++n) {
        ok = wait(IEMPTY(n % kItems), (n / kItems & 1) ^ 1, abort_flag, 0x702);
        if (!ok) break;
        int t = w.t;
        const int end = w.end, b_h = w.h;
        const Seq s = w.s;
        if (lane == 0) {
          const int rows = min(s.n * a.G - w.r * kRows, kRows);
          items[n % kItems] = {w.b,    w.h, w.r,  t, end, w.len, s.row0, s.L, s.past, rows, s.past + divided(w.r * kRows, a.G),
                               max(t, min(end, key_tiles<kHalf, kKeys>(s, a.G, 2 * w.r))), w.first_cta(), w.cta_count()};
          mbar_arrive_cta(IFULL(n % kItems));
        }
        BigWalk next = w;
        more = next.next(a);
        for (; t < end && ok; ++t) {
          const int mine = page;
          if (t + 1 < end) page = page_of(w, t + 1);
          else if (more) page = page_of(next, next.t);
          const int key0 = t * kKeys, there = min(boxes, (s.L - key0 + box_rows - 1) >> box_shift);
#pragma unroll 1
          for (int kv = 0; kv < 2 && ok; ++kv) {
            const uint32_t full = E4M3 ? CFULL(st) : FULL(st);
            ok = wait(E4M3 ? CEMPTY(st) : EMPTY(st), ph ^ 1u, abort_flag, 0x700);
            if (!ok) break;
            const uint32_t dst = (E4M3 ? codes : ring) + static_cast<uint32_t>(st) * kMine;
            expect_tx(leader, full, static_cast<uint32_t>(there * box_rows) * kRowBytes * kBoxes);
            for (int i = 0; i < there; ++i) {
              const int p = __shfl_sync(0xffffffffu, mine, i);
              const int row = paged ? (key0 + (i << box_shift)) & ((1 << a.page_shift) - 1) : s.row0 + key0;
#pragma unroll
              for (int c = 0; c < kBoxes; ++c)
                load_box4(leader, dst + static_cast<uint32_t>(c * 128 * 128) + static_cast<uint32_t>(i << box_shift) * kRowBytes,
                          kv == 0 ? &maps.k : &maps.v, full, 64 * c, row, b_h, p);
            }
            ++issued;
            if (++st == my_slots) {
              st = 0;
              ph ^= 1u;
            }
          }
        }
        w = next;
      }
      ok = ok && wait(IEMPTY(n % kItems), (n / kItems & 1) ^ 1, abort_flag, 0x703);
      if (ok && lane == 0) {
        items[n % kItems].t = -1;
        mbar_arrive_cta(IFULL(n % kItems));
      }
      if (!ok) {  // after an abort the loads in flight land before the CTA leaves
        for (int i = min(issued, my_slots); i > 0; --i) {
          st = st == 0 ? my_slots - 1 : st - 1;
          if (st == my_slots - 1) ph ^= 1u;
          wait(E4M3 ? CFULL(st) : FULL(st), ph, nullptr, 0x701);
        }
      }
    } else if (E4M3 && some && warp == 10) {
      // ------------------------------------ 8-bit: scales of a tile's keys and values
      // four keys a lane
      uint32_t n = 0;
      for (int item = 0; ok; ++item) {
        const Item* it = take(item);
        if (it == nullptr || it->t < 0) break;
        const int end = it->end, L = it->L, least = it->least;
        for (int t = it->t; t < end; ++t, ++n) {
          const uint32_t slot = n % kScaleSlots;
          const int key = t * kKeys + 4 * lane;
          float4 ks = make_float4(0.f, 0.f, 0.f, 0.f), vs = ks;
          if (key < L) {
            int64_t page, place;
            if (locate(a, it->row0, it->b, key, page, place)) {
              const int64_t at = ((page * a.Hkv + it->h) << a.page_shift) + place;
              ks = *reinterpret_cast<const float4*>(a.kv.k_scale + at);
              vs = *reinterpret_cast<const float4*>(a.kv.v_scale + at);
            }
          }
          float* each = &vs.x;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (key + e >= L) {
              each[e] = 0.f;
            } else if (!(fabsf(each[e]) < INFINITY) && t * kKeys + kKeys - 1 > least) {  // (as values that are not finite)
              each[e] = 0.f;
              dirty[item % kDirty] = item;
            }
          }
          const float4 by = make_float4(scale_log2(vs.x), scale_log2(vs.y), scale_log2(vs.z), scale_log2(vs.w));
          // (whole numbers)
          const int most = __reduce_max_sync(0xffffffffu, static_cast<int>(fmaxf(fmaxf(by.x, by.y), fmaxf(by.z, by.w))));
          const int fewest = __reduce_min_sync(0xffffffffu, static_cast<int>(fminf(fminf(by.x, by.y), fminf(by.z, by.w))));
          ok = wait(SCEMPTY(slot), (n / kScaleSlots & 1u) ^ 1u, abort_flag, 0x710);
          if (!ok) break;
          float* to = scales + slot * kScaleSlot;
          *reinterpret_cast<float4*>(to + 4 * lane) = ks;
          *reinterpret_cast<float4*>(to + kKeys + 4 * lane) = vs;
          *reinterpret_cast<float4*>(to + 2 * kKeys + 4 * lane) = by;
          if (lane == 0) to[3 * kKeys] = most - fewest <= kClose ? static_cast<float>(most) : INFINITY;
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(SCFULL(slot));
        }
        leave(item);
      }
    } else if (some && warp == 9) {
      // -------------------------------------------------------- MMA issuer
      const uint32_t leader = elect_one();
      const uint32_t fmt = F16 ? 0u : 1u;
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
      // (a tile's keys in two parts: the first's products run while the second's weights are made)
      auto outputs = [&](int i, int part, uint32_t tile, bool first) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ts(leader, tmem + kOut + 128u * i, tmem + 128u * i + 32u * part + 8u * k,
                 v_low | (addr(tile) + 512u * part + 128u * k), hi, idesc_o, !first || k > 0);
      };
      int st = 0;
      uint32_t ph = 0, pph = 0, qph = 0;  // (a bit a half)
      bool any = false;
      auto step = [&] {
        if (++st == slots) {
          st = 0;
          ph ^= 1u;
        }
      };
      // a tile is there (16-bit: and looked at, in which the others' wait lies already)
      auto there = [&](int info) {
        return (E4M3 || wait(READY(st), ph, abort_flag, info)) && wait(FULL(st), ph, abort_flag, info);
      };
      auto tile_at = [&](int s) { return ring + static_cast<uint32_t>(s) * kTile; };
      for (int item = 0; ok; ++item) {
        const Item* it = take(item);
        if (it == nullptr) ok = false;
        if (!ok || it->t < 0) break;
        const int t0 = it->t, end = it->end, e[2] = {it->end0, it->rows > kHalf ? end : t0};
#pragma unroll 1
        for (int i = 0; i < 2 && ok; ++i)
          if (t0 < (i == 0 ? e[0] : e[1])) {
            ok = wait(QFULL(i), qph >> i & 1u, abort_flag, 0x720);
            qph ^= 1u << i;
          }
        ok = ok && there(0x721);
        if (!ok) break;
        tc_fence_after();
        any = true;
#pragma unroll 1
        for (int i = 0; i < 2; ++i)
          if (t0 < (i == 0 ? e[0] : e[1])) scores(i, tile_at(st));
        commit<false>(leader, EMPTY(st));
        step();
        for (int t = t0; t < end && ok; ++t) {
          const int vs = st;
          ok = there(0x722);
          step();
          const int ks = st;
          const bool again = t + 1 < end;
          if (again) {
            ok = ok && there(0x724);
            step();
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int ends = e[i];
            if (ok && t < ends) {
#pragma unroll
              for (int part = 0; part < 2 && ok; ++part) {
                ok = wait(PFULL(i, part), pph >> i & 1u, abort_flag, 0x725);
                if (!ok) break;
                tc_fence_after();
                outputs(i, part, tile_at(vs), t == t0 && part == 0);
              }
              pph ^= 1u << i;
              if (ok && t + 1 >= ends) commit<false>(leader, OFULL(i));
            }
            if (ok && i == 1) commit<false>(leader, EMPTY(vs));
            if (ok && t + 1 < ends) scores(i, tile_at(ks));
          }
          if (again && ok) commit<false>(leader, EMPTY(ks));
        }
        leave(item);
      }
      if (!ok && any) {  // MMAs in flight end before tensor memory is freed
        if (leader != 0u) mma_commit(drain);
        wait(drain, 0u, nullptr, 0x730);
      }
    } else if (some && !E4M3) {
      // ------------------- 16-bit: values of tiles that some row does not wholly see
      const int me = (warp - 10) * 32 + lane;
      int st = 0;
      uint32_t ph = 0;
      for (int item = 0; ok; ++item) {
        const Item* it = take(item);
        if (it == nullptr || it->t < 0) break;
        const int least = it->least, L = it->L, end = it->end;
        for (int u = 2 * it->t; u < 2 * end; ++u) {  // keys, values
          const int t = u >> 1;
          ok = wait(FULL(st), ph, abort_flag, 0x740);
          if (!ok) break;
          if ((u & 1) != 0 && t * kKeys + kKeys - 1 > least) {
            const uint32_t tile = ring + static_cast<uint32_t>(st) * kTile;
            const int there = min(kKeys, L - t * kKeys);
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
                const uint4 x = make_uint4(tame(v.x, F16, bad), tame(v.y, F16, bad), tame(v.z, F16, bad), tame(v.w, F16, bad));
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
        leave(item);
      }
    } else if (E4M3 && some && warp >= 12) {
      // ------------------------------------------- 8-bit: codes into f16 tiles
      // Eight lanes take half a row each of two neighbouring rows, 64 codes, whose swizzled
      // f16 pieces lie in different banks; a thread's pieces are 32 rows and half a row
      // apart, so that all its addresses are two plus constants.
      static_assert(kConverters == 4, "32 rows at a time");
      const int me = (warp - 12) * 32 + lane, my_row = (me >> 3) * 2 + (me >> 2 & 1), my_piece = me & 3;
      const uint32_t my_codes = static_cast<uint32_t>(my_row * DP + 16 * my_piece);
      const uint32_t my_f16[2] = {piece_at(my_row, 2 * my_piece), piece_at(my_row, 2 * my_piece + 1)};
      int st = 0, cs = 0;
      uint32_t ph = 0, cph = 0;
      for (int item = 0; ok; ++item) {
        const Item* it = take(item);
        if (it == nullptr || it->t < 0) break;
        const int least = it->least, L = it->L, end = it->end;
#pragma unroll 1
        for (int u = 2 * it->t; u < 2 * end; ++u) {  // keys, values
          const int t = u >> 1;
          ok = wait(CFULL(cs), cph, abort_flag, 0x750) && wait(EMPTY(st), ph ^ 1u, abort_flag, 0x751);
          if (!ok) break;
          const uint32_t from = codes + static_cast<uint32_t>(cs * code_bytes(DP)), tile = ring + static_cast<uint32_t>(st) * kTile;
          const bool partly = (u & 1) != 0 && t * kKeys + kKeys - 1 > least;
          const int there = L - t * kKeys;
          uint32_t odd = 0;
          auto convert = [&](uint32_t src, uint32_t (&h)[8]) {
            const uint4 v = dense::lds_u4(from + src);
            const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = e4m3x2_f16x2(e & 1 ? q[e >> 1] >> 16 : q[e >> 1] & 0xFFFFu);
          };
          auto put = [&](uint32_t dst, const uint32_t (&h)[8]) {
            dense::sts_u4(tile + my_f16[0] + dst, make_uint4(h[0], h[1], h[2], h[3]));
            dense::sts_u4(tile + my_f16[1] + dst, make_uint4(h[4], h[5], h[6], h[7]));
          };
          if (!partly) {
#pragma unroll
            for (int j = 0; j < 4 * kChunks; ++j) {
              uint32_t h[8];
              convert(my_codes + static_cast<uint32_t>((j / kChunks) * 32 * DP + (j % kChunks) * 64), h);
              put(static_cast<uint32_t>((j / kChunks) * 32 * 128 + (j % kChunks) * 128 * 128), h);
            }
          } else {
#pragma unroll 1
            for (int j = 0; j < 4 * kChunks; ++j) {
              uint32_t h[8];
              convert(my_codes + static_cast<uint32_t>((j / kChunks) * 32 * DP + (j % kChunks) * 64), h);
              const bool in = my_row + j / kChunks * 32 < there;
#pragma unroll
              for (int e = 0; e < 8; ++e) h[e] = in ? tame(h[e], true, odd) : 0u;
              put(static_cast<uint32_t>((j / kChunks) * 32 * 128 + (j % kChunks) * 128 * 128), h);
            }
          }
          if (odd) dirty[item % kDirty] = item;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive_cta(FULL(st));
            mbar_arrive_cta(CEMPTY(cs));
          }
          if (++st == slots) {
            st = 0;
            ph ^= 1u;
          }
          if (++cs == kCodeSlots) {
            cs = 0;
            cph ^= 1u;
          }
        }
        leave(item);
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
    // this thread's row of an item
    auto live_of = [&](const Item* x) { return half * kHalf + row < x->rows; };
    auto row_of = [&](const Item* x) { return x->r * kRows + (live_of(x) ? half * kHalf + row : 0); };
    auto asks = [&](const Item* x) { return x->t < (half == 0 ? x->end0 : x->rows > kHalf ? x->end : x->t); };
    // The warp's queries into shared memory, a row over DP / 8 lanes.  16-bit: started
    // here, there after queries_done.  8-bit: as f16, each row's largest brought to
    // 2^14; returns what this thread's row's scores are multiplied with.
    constexpr int kAcross = DP / 8, kTogether = 32 / kAcross;
    auto queries = [&](const Item* x) {
      const int tok = divided(row_of(x), a.G), hd = x->h * a.G + row_of(x) - tok * a.G;
      const uint64_t mine = live_of(x) ? reinterpret_cast<uint64_t>(a.q + (x->row0 + tok) * a.q_stride + static_cast<int64_t>(hd) * a.D) : 0;
      const int c = lane % kAcross, base_row = 32 * (warp & 3);
#pragma unroll 4
      for (int i = 0; i < kAcross; ++i) {
        const int r = i * kTogether + lane / kAcross;
        const uint64_t from = __shfl_sync(0xffffffffu, mine, r);
        const bool there = from != 0 && 8 * c < a.D;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(q_at + piece_at(base_row + r, c)),
                     "l"(there ? from + 16 * c : reinterpret_cast<uint64_t>(a.q)), "r"(there ? 16u : 0u)
                     : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // They are there; returns what this thread's row's scores are multiplied with.
    auto queries_done = [&] {
      float factor = a.scale_log2;
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      if constexpr (E4M3) {
        __syncwarp();
        float amax = 0.f;
#pragma unroll 2
        for (int c = 0; c < DP / 8; ++c) {
          const uint4 v = dense::lds_u4(q_at + piece_at(row, c));
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(f32_of(u[e] & 0xFFFFu, a.f16)), fabsf(f32_of(u[e] >> 16, a.f16))));
        }
        const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100), 126);
        const bool scaled = amax > 0.f && amax < INFINITY;
        const float up = scaled ? __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23) : 1.f;
        // (not zero, with which a masked score would be NaN)
        if (scaled) factor = fmaxf(factor * __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23), 0x1p-126f);
#pragma unroll 2
        for (int c = 0; c < DP / 8; ++c) {
          uint4 v = dense::lds_u4(q_at + piece_at(row, c));
          uint32_t* u = &v.x;
#pragma unroll
          for (int k = 0; k < 4; ++k) u[k] = pack_half(f32_of(u[k] & 0xFFFFu, a.f16) * up, f32_of(u[k] >> 16, a.f16) * up);
          dense::sts_u4(q_at + piece_at(row, c), v);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(QFULL(half));
      return factor;
    };
    float factor = a.scale_log2;
    // (the first turn has no item yet: it only asks for the first one's queries)
    const Item* w = nullptr;
    for (int item = -1; some; ++item) {
      const bool begun = item >= 0;
      const int t0 = begun ? w->t : 0, w_end = begun ? w->end : 0;
      const int end = !begun ? 0 : half == 0 ? w->end0 : w->rows > kHalf ? w_end : t0;
      // the last key that every row of this half sees, and that this row sees
      const int least = begun ? w->past + divided(w->r * kRows + half * kHalf, a.G) : 0;
      const int limit = begun ? w->past + divided(row_of(w), a.G) : 0;
      float top = -INFINITY;  // of the row's scores, what its weights are relative to
      const uint64_t f2 = pack2(factor, factor);
      uint64_t sum = 0;
      for (int t = t0; t < (E4M3 ? w_end : end); ++t) {
        const float* sc = nullptr;
        uint32_t slot = 0;
        if (E4M3) {
          slot = scn % kScaleSlots;
          ok = wait(SCFULL(slot), scn / kScaleSlots & 1u, abort_flag, 0x760);
          ++scn;
          if (!ok) break;
          sc = scales + slot * kScaleSlot;
          if (t >= end) {  // (the other half's tile)
            __syncwarp();
            if (lane == 0) mbar_arrive_cta(SCEMPTY(slot));
            continue;
          }
        }
        ok = wait(SFULL(half), sph, abort_flag, 0x761);
        if (!ok) break;
        sph ^= 1u;
        tc_fence_after();
        // Twice over the scores, some at a time: their maximum, then the weights.  (Held
        // in registers in between, 128 of them unrolled, the code did not fit the
        // instruction caches.)  Scores that are scaled or masked go back to tensor memory.
        constexpr int kSome = 64;
        const bool masked = t * kKeys + kKeys - 1 > least;
        const float by_tile = E4M3 ? sc[3 * kKeys] : 0.f;
        const bool each = E4M3 && (masked || by_tile == INFINITY);
        float now = -INFINITY;
#pragma unroll 1
        for (int part = 0; part < kKeys / kSome; ++part) {
          uint32_t s[kSome / 32][32];
#pragma unroll
          for (int c = 0; c < kSome / 32; ++c) dense::tmem_ld32(S + static_cast<uint32_t>(kSome * part + 32 * c), s[c]);
#pragma unroll
          for (int c = 0; c < kSome / 32; ++c) dense::tmem_ld32_wait(s[c]);
          if (E4M3) {
#pragma unroll
            for (int j = 0; j < kSome / 4; ++j) {
              const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(sc + kSome * part + 4 * j);
              uint32_t* x = &s[j >> 3][4 * (j & 7)];
              const uint64_t y = mul2((static_cast<uint64_t>(x[1]) << 32) | x[0], k.x);
              const uint64_t z = mul2((static_cast<uint64_t>(x[3]) << 32) | x[2], k.y);
              x[0] = static_cast<uint32_t>(y);
              x[1] = static_cast<uint32_t>(y >> 32);
              x[2] = static_cast<uint32_t>(z);
              x[3] = static_cast<uint32_t>(z >> 32);
            }
          }
          if (masked) {
            const int seen = limit - t * kKeys - kSome * part;
#pragma unroll
            for (int j = 0; j < kSome; ++j)
              if (j > seen) s[j >> 5][j & 31] = __float_as_uint(-INFINITY);
          }
          if (E4M3 || masked) {
#pragma unroll
            for (int c = 0; c < kSome / 32; ++c) tmem_st32(S + static_cast<uint32_t>(kSome * part + 32 * c), s[c]);
          }
          float m4[4] = {now, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < kSome; j += 2)
            m4[j >> 1 & 3] = fmaxf(m4[j >> 1 & 3], fmaxf(__uint_as_float(s[j >> 5][j & 31]), __uint_as_float(s[j >> 5][(j & 31) + 1])));
          now = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        }
        if (E4M3 || masked) tmem_st_wait();
        now = E4M3 ? fmaf(now, factor, by_tile) : now * factor;
        if (E4M3 && each) {  // the maximum with what each value's scale adds
          now = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < kKeys / 32; ++c) {
            uint32_t s[32];
            dense::tmem_ld32(S + 32u * c, s);
            dense::tmem_ld32_wait(s);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const ulonglong2 by = *reinterpret_cast<const ulonglong2*>(sc + 2 * kKeys + 32 * c + 4 * j);
              const uint64_t y = fma2((static_cast<uint64_t>(s[4 * j + 1]) << 32) | s[4 * j], f2, by.x);
              const uint64_t z = fma2((static_cast<uint64_t>(s[4 * j + 3]) << 32) | s[4 * j + 2], f2, by.y);
              now = fmaxf(fmaxf(now, fmaxf(lo2(y), hi2(y))), fmaxf(lo2(z), hi2(z)));
            }
          }
        }
        if (t == t0) {
          top = fmaxf(top, now);  // (NaN leaves it)
        } else if (__any_sync(0xffffffffu, now > top + kLag)) {
          // O of the tiles before is complete: their products precede these scores
          // (a row that did not grow so far keeps its bits, whatever its warp's others do)
          const bool grown = now > top + kLag;
          const float d = top - reference(now), keep = grown ? exp2_fast(E4M3 ? 0.5f * d : d) : 1.f;
          top = grown ? now : top;
          sum = mul2(sum, pack2(keep, keep));
          if (E4M3) sum = mul2(sum, pack2(keep, keep));  // (moved)
          const float f = E4M3 ? keep * keep : keep;
#pragma unroll 1
          for (int c = 0; c < DP / 16; ++c) {
            uint32_t o[16];
            dense::tmem_ld16_wait(O + 16u * c, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st16(O + 16u * c, o);
          }
        }
        const float r = reference(top, kLift<F16>);
        const uint64_t r2 = pack2(-r, -r);
#pragma unroll 1
        for (int part = 0; part < kKeys / kSome; ++part) {
          uint32_t s[kSome / 32][32];
#pragma unroll
          for (int c = 0; c < kSome / 32; ++c) dense::tmem_ld32(S + static_cast<uint32_t>(kSome * part + 32 * c), s[c]);
#pragma unroll
          for (int c = 0; c < kSome / 32; ++c) dense::tmem_ld32_wait(s[c]);
          uint64_t sums[2] = {0, 0};
#pragma unroll
          for (int c = 0; c < kSome / 32; ++c) {
            uint32_t p[16];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              ulonglong2 v = make_ulonglong2(0, 0);
              if (E4M3) v = *reinterpret_cast<const ulonglong2*>(sc + kKeys + kSome * part + 32 * c + 2 * j);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint64_t z = fma2((static_cast<uint64_t>(s[c][2 * (j + k) + 1]) << 32) | s[c][2 * (j + k)], f2, r2);
                uint64_t e = pack2(exp2_fast(lo2(z)), exp2_fast(hi2(z)));
                sums[k] = add2(sums[k], e);
                if (E4M3) e = mul2(e, k == 0 ? v.x : v.y);
                p[j + k] = F16 ? pack_half(lo2(e), hi2(e)) : pack_bf16x2(lo2(e), hi2(e));
              }
            }
            tmem_st16(S + static_cast<uint32_t>(kSome / 2 * part + 16 * c), p);
          }
          sum = add2(sum, add2(sums[0], sums[1]));
          // (half of the keys' weights)
          static_assert(kSome == 64, "two parts");
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(PFULL(half, part));
        }
        if (E4M3 && lane == 0) mbar_arrive_cta(SCEMPTY(slot));
      }
      if (!ok) break;
      // ---- the item's end: its last scores are read, so the next one's queries come
      const bool has = t0 < end;
      const Item* next = take(item + 1);
      if (next == nullptr) {
        ok = false;
        break;
      }
      const bool more = next->t >= 0, ask = more && asks(next);
      if (ask) queries(next);
      if (has) {
        ok = wait(OFULL(half), oph, abort_flag, 0x762);
        oph ^= 1u;
        tc_fence_after();
      }
      float factor_next = factor;
      if (ask) factor_next = queries_done();
      if (!ok) break;
      if (begun) {
        const float total = lo2(sum) + hi2(sum);
        const bool spoiled = dirty[item % kDirty] == item, live = live_of(w);
        const bool whole = w_end - t0 == w->len;
        const int tok = limit - w->past, hd = w->h * a.G + row_of(w) - tok * a.G;
        const int64_t out_row = w->row0 + tok;
        const uint64_t to = live ? reinterpret_cast<uint64_t>(a.out + out_row * a.out_stride + static_cast<int64_t>(hd) * a.D) : 0;
        // An item that lies in several runs leaves its sums in the workspace, and the
        // last of its CTAs to finish joins them in the order of the runs.
        const int first = w->first, pieces = w->pieces, me = static_cast<int>(blockIdx.x) - first;
        constexpr size_t kPiece = attn_piece_bytes(kRows, DP) / 4;
        auto piece = [&](int i) { return a.partial + (2 * (first + i) + (i == 0 ? 1 : 0)) * kPiece; };
        float* mine = piece(me) + half * kHalf + row;
        const float inv = 1.f / total;
#pragma unroll 1
        for (int c = 0; c < DP / 32; ++c) {
          float v[32];
          if (has) {
            uint32_t o[32];
            dense::tmem_ld32(O + 32u * c, o);
            dense::tmem_ld32_wait(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(o[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.f;
          }
          if (!whole) {
            if (live)
#pragma unroll
              for (int j = 0; j < 32; ++j) __stcg(mine + (32 * c + j) * kRows, v[j]);
            continue;
          }
          // The rows of four lanes are turned so that the four store 64 adjacent bytes of
          // one row at a time (a row a lane: 32 lines a store, 2 us an item).
          uint4 u[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t* x = &u[j].x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = v[8 * j + 2 * e] * inv, z = v[8 * j + 2 * e + 1] * inv;
              x[e] = (E4M3 ? a.f16 != 0 : F16) ? pack_half(y, z) : pack_bf16x2(y, z);
            }
          }
          // lane l of four holds pieces 0 to 3 of row l; afterwards piece l of rows 0 to 3
          auto turn = [&](uint4& p, uint4& q, int bit) {  // p of the lanes without the bit for q of those with it
            const bool up = (lane & bit) != 0;
            uint32_t *x = &p.x, *z = &q.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? x[e] : z[e], bit);
              if (up) x[e] = got;
              else z[e] = got;
            }
          };
          turn(u[0], u[1], 1);
          turn(u[2], u[3], 1);
          turn(u[0], u[2], 2);
          turn(u[1], u[3], 2);
          const int column = 32 * c + 8 * (lane & 3);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t row_at = __shfl_sync(0xffffffffu, to, (lane & ~3) + j);
            if (row_at != 0 && column < a.D) *reinterpret_cast<uint4*>(row_at + 2 * column) = u[j];
          }
        }
        if (spoiled && has) {
          // values that are not finite, of the keys that this row sees among those looked
          // at, added to what was written
          __syncwarp();
          const int from = max(t0, divided(w->least + 1, kKeys)) * kKeys;
          const int upto = live ? min(limit, end * kKeys - 1) : -1;
#pragma unroll 1
          for (int key = from; key <= upto; ++key) {
            int64_t page, place;
            if (!locate(a, w->row0, w->b, key, page, place)) continue;
            const float vscale = E4M3 ? a.kv.v_scale[((page * a.Hkv + w->h) << a.page_shift) + place] : 1.f;
            const int64_t in = page * a.kv.v_page + place * a.kv.v_token + w->h * a.kv.v_head;
#pragma unroll 1
            for (int d = 0; d < a.D; ++d) {
              const float x = E4M3 ? __half2float(__ushort_as_half(static_cast<uint16_t>(e4m3x2_f16x2(a.kv.v[in + d])))) * vscale
                                   : f32_of(reinterpret_cast<const uint16_t*>(a.kv.v)[in + d], F16);
              if (fabsf(x) < INFINITY) continue;
              if (!whole) {
                __stcg(mine + d * kRows, __ldcg(mine + d * kRows) + x);
              } else {
                uint16_t* o = reinterpret_cast<uint16_t*>(to) + d;
                const float y = f32_of(*o, a.f16) + x;
                *o = static_cast<uint16_t>(a.f16 ? pack_half(y, 0.f) : pack_bf16x2(y, 0.f));
              }
            }
          }
        }
        if (whole) {
          if (live && a.lse != nullptr) a.lse[out_row * a.Hq + hd] = (top - kLift<F16> + log2_fast(total)) * 0.69314718055994531f;
        } else {
          if (live) {
            __stcg(mine + DP * kRows, top);
            __stcg(mine + (DP + 1) * kRows, total);
          }
          // The warps share the live rows, 32 a warp, and where those are few also the
          // columns (a row a thread with all its columns: 32 rows of 19 pieces took 40 us).
          const int row_warps = (w->rows + 31) / 32;
          const int groups = min(DP / 32, row_warps <= 2 ? 4 : row_warps <= 4 ? 2 : 1);
          const int group = divided(warp, row_warps), join_row = 32 * (warp - group * row_warps) + lane;
          const bool joins = group < groups && join_row < w->rows;
          bool done = false;
#pragma unroll 1
          for (int level = 0; !done; ++level) {
            const Join j = join_of(a, first, pieces, me, level);
            __threadfence();
            __syncwarp();
            if (lane == 0) mbar_arrive_cta(join0);
            ok = wait(join0, jph, abort_flag, 0x770);
            if (!ok) break;
            if (tid == 0) {
              *last_flag = count_in(j);
              mbar_arrive_cta(join1);
            }
            ok = wait(join1, jph, abort_flag, 0x771);
            jph ^= 1u;
            if (!ok || *last_flag == 0) break;
            done = j.last;
            if (!joins) continue;
            // (a group's maxima and totals have a place of their own: warps read its first piece's)
            auto stats = [&](int i) { return piece(j.base + i * j.stride) + (j.stride == 1 ? DP : DP + 2) * kRows + join_row; };
            float m = -INFINITY, l = 0.f;
#pragma unroll 4
            for (int i = 0; i < j.count; ++i) m = fmaxf(m, __ldcg(stats(i)));
            const float r = reference(m);
#pragma unroll 4
            for (int i = 0; i < j.count; ++i) {
              const float d = __ldcg(stats(i)) - r;
              l += moved<E4M3>(__ldcg(stats(i) + kRows), d, exp2_fast(d));
            }
            const int R = w->r * kRows + join_row, join_tok = divided(R, a.G), join_head = w->h * a.G + R - join_tok * a.G;
            const int64_t join_out = w->row0 + join_tok;
            uint16_t* out = a.out + join_out * a.out_stride + static_cast<int64_t>(join_head) * a.D;
            const float per = 1.f / l;
#pragma unroll 1
            for (int c = group * (DP / 32) / groups; c < (group + 1) * (DP / 32) / groups; ++c) {
              float v[32];
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] = 0.f;
#pragma unroll 2
              for (int i = 0; i < j.count; ++i) {
                const float* from = piece(j.base + i * j.stride) + 32 * c * kRows + join_row;
                const float f = exp2_fast(__ldcg(stats(i)) - r);
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = fmaf(__ldcg(from + k * kRows), f, v[k]);
              }
              if (!done) {  // a group's sum, into its first piece's place
#pragma unroll
                for (int k = 0; k < 32; ++k) __stcg(piece(j.base) + (32 * c + k) * kRows + join_row, v[k]);
                continue;
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  u[e] = a.f16 ? pack_half(v[8 * k + 2 * e] * per, v[8 * k + 2 * e + 1] * per)
                               : pack_bf16x2(v[8 * k + 2 * e] * per, v[8 * k + 2 * e + 1] * per);
                if (32 * c + 8 * k < a.D) *reinterpret_cast<uint4*>(out + 32 * c + 8 * k) = make_uint4(u[0], u[1], u[2], u[3]);
              }
            }
            if (done && group == 0 && a.lse != nullptr) a.lse[join_out * a.Hq + join_head] = (m - kLift<F16> + log2_fast(l)) * 0.69314718055994531f;
            if (!done && group == 0) {
              __stcg(piece(j.base) + (DP + 2) * kRows + join_row, m);
              __stcg(piece(j.base) + (DP + 3) * kRows + join_row, l);
            }
          }
        }
        if (!ok) break;
        tc_fence_before();  // (the next item's products write O after this half's weights)
        leave(item);
      }
      if (!more) break;
      w = next;
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
#undef CFULL
#undef CEMPTY
#undef IFULL
#undef IEMPTY
  clear_empty_rows(a);
  if (tid == 0 && *abort_flag != 0) record_error(a.err, kErrTimeout, static_cast<uint32_t>(*abort_flag));
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <bool E4M3, bool F16, int DP>
cudaError_t launch(const AttnArgs& a, int sms, cudaStream_t s) {
  auto kernel = attention_kernel<E4M3, F16, DP>;
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
  const size_t fixed = kMiscBytes<E4M3> + 2 * tile_bytes(DP) + (E4M3 ? code_slots(DP) * code_bytes(DP) : 0);
  const int room = static_cast<int>((kSmem - fixed) / tile_bytes(DP));
  const int slots = room < kMaxSlots ? room : kMaxSlots;
  const size_t smem = std::max(kTensorMemorySmem, fixed + static_cast<size_t>(slots) * tile_bytes(DP));
  Maps maps = {};
  int box_rows = kKeys;
  {
    const bool paged = a.page_table != nullptr;
    const uint64_t page = paged ? 1ull << a.page_shift : static_cast<uint64_t>(a.T);
    box_rows = paged && page < kKeys ? static_cast<int>(page) : kKeys;
    const CUtensorMapDataType dt = E4M3    ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : a.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                           : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle swizzle = E4M3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
    constexpr int64_t size = E4M3 ? 1 : 2;
    const uint64_t dims[4] = {static_cast<uint64_t>(a.D), page, static_cast<uint64_t>(a.Hkv), static_cast<uint64_t>(a.num_pages)};
    const uint32_t box[4] = {E4M3 ? DP : 64, static_cast<uint32_t>(box_rows), 1, 1};
    const int64_t far = 16;  // (of one page: no stride)
    const uint64_t ks[3] = {static_cast<uint64_t>(size * a.kv.k_token), static_cast<uint64_t>(size * a.kv.k_head),
                            static_cast<uint64_t>(paged ? size * a.kv.k_page : far)};
    const uint64_t vs[3] = {static_cast<uint64_t>(size * a.kv.v_token), static_cast<uint64_t>(size * a.kv.v_head),
                            static_cast<uint64_t>(paged ? size * a.kv.v_page : far)};
    if (!encode_map(&maps.k, dt, 4, a.kv.k, dims, ks, box, swizzle) ||
        !encode_map(&maps.v, dt, 4, a.kv.v, dims, vs, box, swizzle))
      return cudaErrorInvalidValue;
  }
  return launch_pdl(kernel, dim3(sms < kAttnMaxCtas ? sms : kAttnMaxCtas), dim3(kThreads<E4M3>), smem, s, maps, a, slots,
                    box_rows);
}

}  // namespace

cudaError_t launch_attention(const AttnArgs& a, int sms, cudaStream_t s) {
  if (a.e4m3) return a.D <= 64 ? launch<true, true, 64>(a, sms, s) : launch<true, true, 128>(a, sms, s);
  if (a.f16) return a.D <= 64 ? launch<false, true, 64>(a, sms, s) : launch<false, true, 128>(a, sms, s);
  return a.D <= 64 ? launch<false, false, 64>(a, sms, s) : launch<false, false, 128>(a, sms, s);
}

}  // namespace moe
