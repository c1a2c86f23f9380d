// How the attention kernels share out their work.  An item is a tile of rows (the
// queries of one sequence and key head: row i G + g is query head g of the group,
// new token i) and reads the keys up to its last row's, in tiles of KT keys.  All
// items' tiles, in the order of sequences, key heads and row tiles, are cut into as
// many runs of about equal cost as there are CTAs, whatever the sequences' lengths are:
// a long context is spread over many SMs and short ones share one.  Lengths are read
// on the device, so a captured call follows them.  An item that lies in several runs
// is joined by the CTA that finishes last, in the order of the runs (the result does
// not depend on which one that is).  Runs of equal numbers of tiles, without the items'
// own costs, took 549 us for packed prompts of 513 to 7001 tokens, runs of equal cost
// 349.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace attn {

// The live rows of a sequence: its last n new tokens see keys [0, past + i]; of a
// sequence with fewer keys than new tokens the first `none` see nothing.
struct Seq {
  int row0;  // of the first live token
  int n, L, past, none;
};

__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b, bool report) {
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1];
  Seq s;
  int n = q1 - q0;
  bool bad = false;
  if (q0 < 0 || q1 < q0 || q1 > a.T) {
    bad = true;
    n = 0;
  }
  int L = a.kv_len != nullptr ? a.kv_len[b] : n;
  if (a.kv_len != nullptr && (L < 0 || L > a.max_len)) {
    bad = true;
    L = L < 0 ? 0 : a.max_len;
  }
  if (bad && report) record_error(a.err, kErrBadIndex, static_cast<uint32_t>(b));
  s.L = L;
  s.n = min(n, L);
  s.none = n - s.n;
  s.row0 = q0 + s.none;
  s.past = L - s.n;
  return s;
}

// Row tiles of M rows, and the key tiles that row tile r reads.  (A call's rows are
// fewer than 2^30: 32-bit divisions, which are no function calls.)
template <int M>
__device__ __forceinline__ int row_tiles(const Seq& s, int G) {
  return (s.n * G + M - 1) / M;
}
__device__ __forceinline__ int divided(int a, int b) {  // of numbers that are not negative
  return static_cast<int>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}
template <int M, int KT>
__device__ __forceinline__ int key_tiles(const Seq& s, int G, int r) {
  return (s.past + min(divided(M * (r + 1) - 1, G), s.n - 1) + KT) / KT;
}
// Key tiles of the row tiles before r.  But for the last tile, whose rows may end
// early, and with past = KT a + b, tile i reads a + 1 + floor((M i + M - 1 + b G) / (KT
// G)) tiles, the last term being floor((u i + e) / v) in small whole numbers.
template <int M, int KT>
__device__ __forceinline__ int64_t tiles_before(const Seq& s, int G, int r) {
  constexpr int kUnit = M < KT ? M : KT;  // divides both
  int u = M / kUnit, v = KT / kUnit * G, e = (M - 1 + s.past % KT * G) / kUnit;
  int64_t sum = static_cast<int64_t>(s.past / KT + 1) * r;
  static_assert(M / kUnit <= 2, "one or two");
  if (u == 2 && v % 2 == 0) {
    u = 1;
    v /= 2;
    e /= 2;
  }
  if (u == 1) {
    // sum of floor(j / v) over j < x
    auto below = [v](int x) {
      const int q = divided(x, v);
      return static_cast<int64_t>(v) * (static_cast<int64_t>(q) * (q - 1) / 2) + static_cast<int64_t>(q) * (x - q * v);
    };
    sum += below(r + e) - below(e);
  } else {
    // repeats every v tiles, u q more after q times
    const int whole = divided(r, v), rest = r - whole * v, upto = whole > 0 ? v : rest;
    int64_t period = 0;
    for (int i = 0; i < upto; ++i) {
      const int f = divided(u * i + e, v);
      period += f;
      if (i < rest) sum += f;
    }
    sum += whole * period + static_cast<int64_t>(u) * (static_cast<int64_t>(v) * (static_cast<int64_t>(whole) * (whole - 1) / 2) +
                                                      static_cast<int64_t>(whole) * rest);
  }
  return sum;
}
// How a kernel shares out: rows and keys of a tile; what an item costs beside its
// tiles, in tiles; there is a run for every `least` units or a part of them, at most, and
// an item is not cut within `slack` of its ends (a cut costs a join).  `least` and `slack`
// were chosen for batches that fill the SMs; of a few short sequences they leave most idle
// (501 keys, 8 key heads: 10 runs).
template <int M_, int KT_, int COST_, int SLACK_, int LEAST_>
struct Shape {
  static constexpr int M = M_, KT = KT_, cost = COST_, slack = SLACK_, least = LEAST_;
};

// A place among all items' tiles.
struct Place {
  int b, h, r, t;
};

// A CTA's place in its run.
template <typename S>
struct Walk {
  Seq s;
  int b, h, r, R;
  int t, end;   // key tiles of the item in this run
  int len;      // the item's key tiles
  Place stop;   // where the run ends
  int first, pieces, pieces_last;  // of an item that begins before the run: the CTA where it does, and its CTAs; of
                                   // one that ends after it

  __device__ __forceinline__ void enter(const AttnArgs& a) {
    len = key_tiles<S::M, S::KT>(s, a.G, r);
    end = b == stop.b && h == stop.h && r == stop.r ? stop.t : len;
  }
  // the item's first CTA, and how many it has
  __device__ __forceinline__ int first_cta() const { return t > 0 ? first : static_cast<int>(blockIdx.x); }
  __device__ __forceinline__ int cta_count() const { return t > 0 ? pieces : end < len ? pieces_last : 1; }
  // to the next item; false at the run's end
  __device__ __forceinline__ bool next(const AttnArgs& a) {
    if (end < len) return false;
    if (++r == R) {
      r = 0;
      if (++h == a.Hkv) {
        h = 0;
        do {
          if (++b >= a.B) return false;
          s = sequence(a, b, false);
          R = row_tiles<S::M>(s, a.G);
        } while (R == 0);
      }
    }
    t = 0;
    enter(a);
    return end > 0;
  }
};

constexpr int kScratchWords = 64;  // of 8 bytes, for start()

// The run of this CTA; false where it has none.  Every thread calls it; `scratch` (read
// until the next barrier) holds kScratchWords.
template <int THREADS, typename S>
__device__ __forceinline__ bool start(const AttnArgs& a, int64_t* scratch, Walk<S>& w) {
  constexpr int kWarps = THREADS / 32, M = S::M, KT = S::KT;
  static_assert(kWarps <= 32 && kWarps >= 2, "one warp joins the warps' sums, two find the run's ends");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
  auto scan = [&](int64_t v, int64_t& sum) {  // the threads' values before this one's; their sum
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    int64_t before = x - v;
    sum = 0;
#pragma unroll 4
    for (int i = 0; i < kWarps; ++i) {
      const int64_t y = scratch[i];
      if (i < warp) before += y;
      sum += y;
    }
    return before;
  };
  // (twice over the sequences, in one piece of code: their sum, then those that hold
  // the run's ends; of few sequences the second time needs no reading)
  int64_t total = 0, mine = 0, before = 0, base = 0, cut[2] = {0, 0}, run = 0;
  int n = 0, longer = 0;
  auto run_of = [&](int c) { return run + (c < longer); };
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += THREADS) {
      int64_t sum = total;
      if (pass == 0 || a.B > THREADS) {
        const int b = b0 + tid;
        mine = 0;
        if (b < a.B) {
          const Seq s = sequence(a, b, pass == 0 && cta == 0);
          const int R = row_tiles<M>(s, a.G);
          if (R > 0)
            mine = (tiles_before<M, KT>(s, a.G, R - 1) + key_tiles<M, KT>(s, a.G, R - 1) + static_cast<int64_t>(S::cost) * R) * a.Hkv;
        }
        before = scan(mine, sum);
      }
      if (pass == 0) {
        total += sum;
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (base + before <= cut[i] && cut[i] < base + before + mine) {
            scratch[32 + 2 * i] = b0 + tid;
            scratch[33 + 2 * i] = cut[i] - base - before;
          }
        base += sum;
      }
    }
    if (pass == 0) {
      const int64_t most = (total + S::least - 1) / S::least;
      n = static_cast<int>(most < static_cast<int64_t>(gridDim.x) ? most : static_cast<int64_t>(gridDim.x));
      if (cta >= n) return false;
      run = total >> 31 == 0 ? static_cast<int64_t>(divided(static_cast<int>(total), n)) : total / n;
      longer = static_cast<int>(total - run * n);
      cut[0] = run * cta + min(cta, longer);
      cut[1] = cut[0] + run_of(cta);
    }
  }
  __syncthreads();
  // warps 0 and 1: where the run's ends lie
  int* found = reinterpret_cast<int*>(scratch + 40);
  if (warp < 2) {
    const int c = cta + warp;  // the CTA that begins here
    Place p = {a.B, 0, 0, 0};
    int first = cta, pieces = 1, from_b = -1;
    Seq s{};
    if (c < n) {
      from_b = p.b = static_cast<int>(scratch[32 + 2 * warp]);
      int64_t rest = scratch[33 + 2 * warp];
      s = sequence(a, p.b, false);
      int R = row_tiles<M>(s, a.G);
      // the last row tile that starts at or before `rest`: 32 candidates at a time, the
      // first time with the whole head's cost as one more
      int lo = 0, hi = R;    // in [lo, hi)
      int64_t skipped = 0;   // what lies before row tile lo
      bool whole = true;
#pragma unroll 1
      while (whole || hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, r = whole ? R - 1 : min(lo + lane * step, R - 1);
        const int64_t there = tiles_before<M, KT>(s, a.G, r) + static_cast<int64_t>(S::cost) * r;
        if (whole) {
          const int64_t head = there + key_tiles<M, KT>(s, a.G, r) + S::cost;
          for (; rest >= head; ++p.h) rest -= head;
          whole = false;
          continue;
        }
        const int top = 31 - __clz(__ballot_sync(0xffffffffu, lo + lane * step < hi && there <= rest));
        skipped = __shfl_sync(0xffffffffu, there, top);
        lo += top * step;
        hi = min(hi, lo + step);
      }
      p.r = lo;
      const int len = key_tiles<M, KT>(s, a.G, lo);
      const int64_t at = rest - skipped;  // in the item, its cost first
      const int64_t from = S::cost + S::slack, upto = S::cost + len - S::slack;
      if (at < from) {
        p.t = 0;
      } else if (at > upto) {  // the next item's start
        if (++p.r == R) {
          p.r = 0;
          if (++p.h == a.Hkv) {
            p.h = 0;
            do ++p.b;
            while (p.b < a.B && row_tiles<M>(sequence(a, p.b, false), a.G) == 0);
          }
        }
      } else {
        p.t = static_cast<int>(at) - S::cost;
        // the item's other cuts
        int c0 = c, c1 = c;
        for (int64_t x = at; c0 > 1 && x - run_of(c0 - 1) >= from; --c0) x -= run_of(c0 - 1);
        for (int64_t x = at; c1 + 1 < n && x + run_of(c1) <= upto; ++c1) x += run_of(c1);
        first = c0 - 1;
        pieces = c1 - c0 + 2;
      }
    }
    if (lane == 0) {
      int* to = found + 6 * warp;
      to[0] = p.b, to[1] = p.h, to[2] = p.r, to[3] = p.t, to[4] = first, to[5] = pieces;
      if (warp == 0 && p.b < a.B) *reinterpret_cast<Seq*>(found + 12) = p.b == from_b ? s : sequence(a, p.b, false);
    }
  }
  __syncthreads();
  w.b = found[0], w.h = found[1], w.r = found[2], w.t = found[3];
  w.stop = {found[6], found[7], found[8], found[9]};
  w.first = found[4];
  w.pieces = found[5];
  w.pieces_last = found[11];
  if (w.b >= a.B || (w.b == w.stop.b && w.h == w.stop.h && w.r == w.stop.r && w.t == w.stop.t)) return false;
  w.s = *reinterpret_cast<const Seq*>(found + 12);
  w.R = row_tiles<M>(w.s, a.G);
  w.enter(a);
  return true;
}

// How an item's pieces are joined: all at once by the last CTA to finish, or, where
// they are many, by the last one of each kGroup and then the last of those (152
// pieces one after the other took 40 us).  Counters are zero between calls: of all
// pieces or groups, of the first group and of the others, each by a CTA that has no
// other item's (a CTA begins at most one cut item and continues at most one).
constexpr int kDirect = 16, kGroup = 12;
struct Join {
  uint32_t* counter;
  int base, stride, count;  // pieces base, base + stride, ...
  bool last;                // of the item, else of a group
};
__device__ __forceinline__ Join join_of(const AttnArgs& a, int first, int pieces, int me, int level) {
  if (pieces <= kDirect) return {a.tickets + first, 0, 1, pieces, true};
  if (level > 0) return {a.tickets + first, 0, kGroup, (pieces + kGroup - 1) / kGroup, true};
  const int group = me / kGroup, base = group * kGroup;
  return {group == 0 ? a.tickets + kAttnMaxCtas + first : a.tickets + 2 * kAttnMaxCtas + first + base, base, 1,
          min(kGroup, pieces - base), false};
}
// Counts one in; whether it was the last, with what the others wrote before visible.
__device__ __forceinline__ bool count_in(const Join& j) {
  const bool last = atomicAdd(j.counter, 1u) == static_cast<uint32_t>(j.count - 1);
  if (last) *j.counter = 0;
  __threadfence();
  return last;
}

// Rows of tokens that see no key: zeros, and minus infinity as their logarithm.
__device__ __forceinline__ void clear_empty_rows(const AttnArgs& a) {
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const Seq s = sequence(a, b, false);
    const int width = a.Hq * a.D;
    for (int64_t i = threadIdx.x; i < static_cast<int64_t>(s.none) * width; i += blockDim.x)
      a.out[(s.row0 - s.none + i / width) * a.out_stride + i % width] = 0;
    if (a.lse != nullptr)
      for (int64_t i = threadIdx.x; i < static_cast<int64_t>(s.none) * a.Hq; i += blockDim.x)
        a.lse[static_cast<int64_t>(s.row0 - s.none) * a.Hq + i] = -INFINITY;
  }
}

// 2^x; x = -inf gives 0
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// What scores are taken relative to: the row's maximum, lowered where the weights' type
// needs it; of rows without any score yet zero.
__device__ __forceinline__ float reference(float m, float lift = 0.f) { return m == -INFINITY ? 0.f : m - lift; }

// 8-bit caches: what a key's value scale adds to its score where a row's maximum is
// taken, so that weight times scale, which is what becomes f16, is of the same size
// whatever the scales are: the logarithm of the power of two above it.  Weights of small
// scales are large numbers for that, hence at least -80: 2^30 keys' sum stays in float's
// range.  (Scales that are not finite say nothing about the others.)
constexpr float kLeastScale = -80.f;
__device__ __forceinline__ float scale_log2(float v) {
  const int e = static_cast<int>(__float_as_uint(v) >> 23 & 255u);
  return e == 255 ? kLeastScale : fmaxf(static_cast<float>(e - 126), kLeastScale);
}

// A sum of weights times f = 2^d: of an 8-bit cache, which may be large where f
// vanishes, twice by half of the exponent.
template <bool E4M3>
__device__ __forceinline__ float moved(float sum, float d, float f) {
  if (!E4M3) return sum * f;
  const float h = exp2_fast(0.5f * d);
  return sum * h * h;
}

__device__ __forceinline__ float f32_of(uint16_t v, bool f16) {
  return f16 ? __half2float(__ushort_as_half(v)) : __uint_as_float(static_cast<uint32_t>(v) << 16);
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace attn
}  // namespace moe
