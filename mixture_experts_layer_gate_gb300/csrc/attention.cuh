// How the attention kernels share out their work.  An item is a tile of rows (the
// queries of one sequence and key head: row i G + g is query head g of the group,
// new token i) and reads the keys up to its last row's, in tiles of KT keys.  All
// items' tiles, in the order of sequences, key heads and row tiles, are cut into as
// many runs of equal length as there are CTAs, whatever the sequences' lengths are: a
// long context is spread over many SMs and short ones share one.  Lengths are read
// on the device, so a captured call follows them.  An item that lies in several runs
// is joined by the CTA that finishes last, in the order of the runs (the result does
// not depend on which one that is).
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
template <int M, int KT>
__device__ __forceinline__ int64_t head_tiles(const Seq& s, int G) {
  const int R = row_tiles<M>(s, G);
  return R == 0 ? 0 : tiles_before<M, KT>(s, G, R - 1) + key_tiles<M, KT>(s, G, R - 1);
}

// A CTA's place in its run of tiles.
template <int M, int KT>
struct Walk {
  Seq s;
  int b, h, r, R;
  int t, end;        // key tiles of the item in this run
  int len;           // the item's key tiles
  int64_t left;      // tiles of the run from t on

  __device__ __forceinline__ void enter(const AttnArgs& a) {
    len = key_tiles<M, KT>(s, a.G, r);
    end = left < len - t ? t + static_cast<int>(left) : len;
  }
  // to the next item; false at the run's end
  __device__ __forceinline__ bool next(const AttnArgs& a) {
    left -= end - t;
    if (left <= 0) return false;
    if (++r == R) {
      r = 0;
      if (++h == a.Hkv) {
        h = 0;
        do {
          if (++b >= a.B) {  // (lengths that changed under the call)
            left = 0;
            return false;
          }
          s = sequence(a, b, false);
          R = row_tiles<M>(s, a.G);
        } while (R == 0);
      }
    }
    t = 0;
    enter(a);
    return true;
  }
};

struct Shares {
  int64_t run;   // tiles of a CTA, and one more of the first `more` CTAs
  int n, more;   // CTAs with work
  int first;     // the CTA whose run holds the first tile of this run's first item
  __device__ __forceinline__ int64_t run_of(int c) const { return run + (c < more); }
  // CTAs up to the one that holds the last tile of an item of this CTA that begins
  // in the run of `from`, `rest` tiles after this run
  __device__ __forceinline__ int pieces(int from, int64_t rest) const {
    int c = blockIdx.x + 1;
    for (; rest > 0; ++c) rest -= run_of(c);
    return c - from;
  }
};

// The run of this CTA; false where it has none.  Every thread calls it; `scratch`
// (read until the next barrier) holds THREADS / 32 + 4 words of 8 bytes.
template <int M, int KT, int THREADS>
__device__ __forceinline__ bool start(const AttnArgs& a, int64_t* scratch, Walk<M, KT>& w, Shares& sh) {
  constexpr int kWarps = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  // (twice over the sequences, in one piece of code: their sum, then the one that
  // holds the run's first tile; of few sequences the second time needs no reading)
  const int cta = blockIdx.x;
  int64_t total = 0, mine = 0, before = 0, base = 0, lo = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += THREADS) {
      int64_t sum = total;
      if (pass == 0 || a.B > THREADS) {
        const int b = b0 + tid;
        mine = b < a.B ? head_tiles<M, KT>(sequence(a, b, pass == 0 && cta == 0), a.G) * a.Hkv : 0;
        before = scan(mine, sum);
      }
      if (pass == 0) {
        total += sum;
      } else {
        if (base + before <= lo && lo < base + before + mine) {
          scratch[kWarps] = b0 + tid;
          scratch[kWarps + 1] = lo - base - before;
        }
        base += sum;
      }
    }
    if (pass == 0) {
      sh.n = static_cast<int>(total < static_cast<int64_t>(gridDim.x) ? total : static_cast<int64_t>(gridDim.x));
      if (cta >= sh.n) return false;
      sh.run = total >> 31 == 0 ? static_cast<int64_t>(divided(static_cast<int>(total), sh.n)) : total / sh.n;
      sh.more = static_cast<int>(total - sh.run * sh.n);
      lo = sh.run * cta + min(cta, sh.more);
    }
  }
  __syncthreads();
  w.b = static_cast<int>(scratch[kWarps]);
  int64_t rest = scratch[kWarps + 1];
  w.s = sequence(a, w.b, false);
  w.R = row_tiles<M>(w.s, a.G);
  w.h = 0;
  // the last row tile that starts at or before `rest`: 32 candidates at a time, the
  // first time with the whole head's tiles as one more
  int lo_r = 0, hi_r = w.R;  // in [lo_r, hi_r)
  int64_t skipped = 0;       // tiles before row tile lo_r
  bool first = true;
#pragma unroll 1
  while (first || hi_r - lo_r > 1) {
    const int step = (hi_r - lo_r + 31) / 32;
    const int r = first ? w.R - 1 : lo_r + lane * step;
    const int64_t there = tiles_before<M, KT>(w.s, a.G, min(r, w.R - 1));
    if (first) {
      const int64_t per_head = there + key_tiles<M, KT>(w.s, a.G, w.R - 1);
      for (; rest >= per_head; ++w.h) rest -= per_head;
      first = false;
      continue;
    }
    const int top = 31 - __clz(__ballot_sync(0xffffffffu, r < hi_r && there <= rest));
    skipped = __shfl_sync(0xffffffffu, there, top);
    lo_r += top * step;
    hi_r = min(hi_r, lo_r + step);
  }
  w.r = lo_r;
  w.t = static_cast<int>(rest - skipped);
  w.left = sh.run_of(cta);
  sh.first = cta;
  for (int64_t back = w.t; back > 0;) back -= sh.run_of(--sh.first);
  w.enter(a);
  return true;
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
// the maximum that scores are taken relative to: of rows without any score yet zero
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace attn
}  // namespace moe
