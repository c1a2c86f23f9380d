// Attention of few rows (single tokens, drafted tokens: at most 16 rows of a key
// head's queries): every key and value is read once and used by 16 rows, so the bound
// is memory, and the products are mma.sync m16n8k16 (tcgen05's smallest M is 64
// rows).  More rows go through tiles of 16, which is right but reads the keys once a
// tile.
//
// A tile of 128 keys is 16 keys for each of the eight warps.  A warp streams its
// keys and values through a ring of its own (cp.async, several tiles ahead, across
// items) and holds its own running maximum, sum and output, joined when the item
// ends: no warp waits for another inside an item.
//
// One pass over the keys: with m the largest score so far, l = sum 2^(x - m) and O =
// sum 2^(x - m) v, both multiplied by 2^(m - m') when it grows to m'.  Sums are float;
// weights are rounded to the values' 16-bit type before they multiply them (half a
// step of it, as the output's own rounding).
//
// 8-bit cache: codes become f16, which is exact, and so do the queries after a
// power of two brings each row's largest value to 2^14 (what falls below f16's steps is
// under 2^-38 of that).  A key's scale multiplies its score.  A value's scale
// multiplies its weight, relative to the largest one so far rounded up to a power of
// two, so that weights stay in f16's range.
//
// K is permuted inside the head (any order gives the same product) so that a lane's
// 16 adjacent bytes of a key are its fragment; 8-bit values are read along the head and
// paired across keys by byte permutes, which leaves each lane 32 adjacent outputs.
#include "attention.cuh"
#include "stream.cuh"

namespace moe {
namespace {

using namespace attn;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kRows = kAttnFewRows;
constexpr int kKeys = 16;             // of a warp's step
constexpr int kTile = kKeys * kWarps;
constexpr int kMaxDepth = 8;
constexpr size_t kSmem = 232448;

using FewWalk = Walk<Shape<kRows, kTile, 1, 1, 1>>;

__host__ __device__ constexpr int row_bytes(bool e4m3, int dp) { return e4m3 ? dp : 2 * dp; }
// a step's keys and values, and their scales
__host__ __device__ constexpr int stage_bytes(bool e4m3, int dp) {
  return 2 * kKeys * row_bytes(e4m3, dp) + (e4m3 ? 2 * kKeys * 4 : 0);
}
__host__ __device__ constexpr int join_bytes(int dp) { return 4 * kRows * dp * 4; }
constexpr int kMiscBytes = 2 * kWarps * kRows * 4 + kScratchWords * 8;

__device__ __forceinline__ void cp_async16_if(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16u : 0u) : "memory");
}

// Where the 16-byte pieces of a key or value row lie, so that a warp's reads fall into
// different banks: lanes read four pieces of eight keys, or one of eight values
// (16-bit) or eight of four value pairs (8-bit).
template <bool E4M3, int DP>
__device__ __forceinline__ int k_piece(int key, int piece) {
  return row_bytes(E4M3, DP) >= 128 ? piece ^ ((key & 1) << 2) : piece;
}
template <bool E4M3, int DP>
__device__ __forceinline__ int v_piece(int key, int piece) {
  if (!E4M3) return piece ^ (key & 7);
  return DP == 128 ? piece ^ (((key >> 1) & 3) << 1) : piece;
}

__device__ __forceinline__ float f32_of(uint16_t v, bool f16) {
  return f16 ? __half2float(__ushort_as_half(v)) : __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// F16: the products' type (8-bit caches: always), else bf16
template <bool E4M3, bool F16, int DP>
__global__ void __launch_bounds__(kThreads, 1) attention_few_kernel(const AttnArgs a, const int depth) {
  extern __shared__ __align__(128) uint8_t few_smem[];
  constexpr int kRow = row_bytes(E4M3, DP), kPieces = kRow / 16, kStage = stage_bytes(E4M3, DP);
  constexpr int kPerLoad = 32 / kPieces;  // keys that a load of the warp covers
  constexpr int kTiles = DP / 8;          // column tiles of the output
  constexpr int W = DP / 8;               // 8-bit: adjacent values a lane reads of a row
  __shared__ int last;
  float* join = reinterpret_cast<float*>(few_smem);  // [4 or 8][rows][DP]
  float* ms = join + join_bytes(DP) / 4;             // [warp][row]
  float* ls = ms + kWarps * kRows;
  int64_t* scratch = reinterpret_cast<int64_t*>(ls + kWarps * kRows);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(few_smem) + static_cast<uint32_t>((join_bytes(DP) + kMiscBytes + 127) / 128 * 128) +
                        static_cast<uint32_t>(warp * depth * kStage);
  pdl_wait();
  pdl_trigger();
  clear_empty_rows(a);
  FewWalk cur;
  if (!start<kThreads>(a, scratch, cur)) return;

  // ---- loads, ahead of the products
  FewWalk iss = cur;
  bool more = true;
  const bool paged = a.page_table != nullptr;
  const int my_piece = lane % kPieces, my_key = lane / kPieces;
  const bool in_head = my_piece * 16 < a.D * (E4M3 ? 1 : 2);
  const int page_mask = (1 << a.page_shift) - 1;
  // (looked at when the page's keys are loaded, a tile later)
  auto page_of = [&](const FewWalk& w) -> int {
    const int key = w.t * kTile + warp * kKeys;
    return paged && key < w.s.L ? a.page_table[w.b * a.table_stride + (key >> a.page_shift)] : 0;
  };
  int page = page_of(iss), slot_i = 0;
  auto issue = [&] {
    if (more) {
      const int key0 = iss.t * kTile + warp * kKeys;
      const uint32_t dst = ring + static_cast<uint32_t>(slot_i * kStage);
      if (key0 < iss.s.L) {
        const bool good = page >= 0 && page < a.num_pages;
        if (!good && lane == 0) record_error(a.err, kErrBadIndex, static_cast<uint32_t>(iss.b));
        const int64_t place = paged ? (key0 & page_mask) : static_cast<int64_t>(iss.s.row0 + key0);
        const int64_t from = good ? page : 0;
        constexpr int64_t size = E4M3 ? 1 : 2;
        const uint8_t* k = a.kv.k + size * (from * a.kv.k_page + place * a.kv.k_token + iss.h * a.kv.k_head);
        const uint8_t* v = a.kv.v + size * (from * a.kv.v_page + place * a.kv.v_token + iss.h * a.kv.v_head);
#pragma unroll
        for (int i = 0; i < kKeys / kPerLoad; ++i) {
          const int key = i * kPerLoad + my_key;
          const bool there = good && in_head && key0 + key < iss.s.L;
          const int64_t kt = there ? size * key * a.kv.k_token + 16 * my_piece : 0;
          const int64_t vt = there ? size * key * a.kv.v_token + 16 * my_piece : 0;
          cp_async16_if(dst + static_cast<uint32_t>(key * kRow + 16 * k_piece<E4M3, DP>(key, my_piece)),
                        there ? k + kt : a.kv.k, there);
          cp_async16_if(dst + static_cast<uint32_t>((kKeys + key) * kRow + 16 * v_piece<E4M3, DP>(key, my_piece)),
                        there ? v + vt : a.kv.v, there);
        }
        if (E4M3 && lane < 8) {
          const float* s = lane < 4 ? a.kv.k_scale : a.kv.v_scale;
          const int64_t at = ((from * a.Hkv + iss.h) << a.page_shift) + place + 4 * (lane & 3);
          cp_async16_if(dst + static_cast<uint32_t>(2 * kKeys * kRow + 16 * lane), good ? s + at : s, good);
        }
      }
      if (++iss.t == iss.end) more = iss.next(a);
      if (more) page = page_of(iss);
    }
    cp_async_commit();
    if (++slot_i == depth) slot_i = 0;
  };
  for (int i = 0; i < depth - 1; ++i) issue();

  int slot = 0;
  bool going = true;
  while (going) {
    // ---- an item: its rows g and g + 8
    const Seq s = cur.s;
    const int live = min(s.n * a.G - cur.r * kRows, kRows);
    uint4 qf[2][DP / 32];  // of row g + 8 i
    int limit[2];          // the last key that the row sees
    float factor[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool there = g + 8 * i < live;
      const int R = cur.r * kRows + (there ? g + 8 * i : 0);
      const int token = divided(R, a.G), head = cur.h * a.G + R - token * a.G;
      limit[i] = there ? s.past + token : -1;
      factor[i] = a.scale_log2;
      const uint16_t* q = a.q + (s.row0 + token) * a.q_stride + static_cast<int64_t>(head) * a.D;
#pragma unroll
      for (int j = 0; j < DP / 32; ++j) {
        // 16-bit: 8 values at 32 j + 8 c; 8-bit: of 16 values at 64 (j / 2) + 16 c the half j % 2
        const int d = E4M3 ? 64 * (j >> 1) + 16 * c + 8 * (j & 1) : 32 * j + 8 * c;
        qf[i][j] = there && d < a.D ? *reinterpret_cast<const uint4*>(q + d) : make_uint4(0, 0, 0, 0);
      }
      if (E4M3) {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < DP / 32; ++j) {
          const uint32_t w[4] = {qf[i][j].x, qf[i][j].y, qf[i][j].z, qf[i][j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            amax = fmaxf(amax, fmaxf(fabsf(f32_of(static_cast<uint16_t>(w[e]), a.f16)),
                                     fabsf(f32_of(static_cast<uint16_t>(w[e] >> 16), a.f16))));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^(14 - exponent), within float's normal range (no row that is not finite, and none of zeros)
        const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100), 126);
        const bool scaled = amax > 0.f && amax < INFINITY;
        const float up = scaled ? __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23) : 1.f;
        factor[i] = scaled ? factor[i] * __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23) : factor[i];
#pragma unroll
        for (int j = 0; j < DP / 32; ++j) {
          uint32_t* w = &qf[i][j].x;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = pack_half(f32_of(static_cast<uint16_t>(w[k]), a.f16) * up,
                             f32_of(static_cast<uint16_t>(w[k] >> 16), a.f16) * up);
        }
      }
    }
    const int least = s.past + divided(cur.r * kRows, a.G);  // of all rows' limits
    float o[kTiles][4];
#pragma unroll
    for (int j = 0; j < kTiles; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float unit = 0.f, per_unit = 0.f;  // 8-bit: what the values' scales are relative to, and its inverse

    for (int t = cur.t; t < cur.end; ++t) {
      cp_async_wait(depth - 2);
      __syncwarp();
      issue();
      const int key0 = t * kTile + warp * kKeys;
      const uint32_t src = ring + static_cast<uint32_t>(slot * kStage);
      if (++slot == depth) slot = 0;
      if (key0 >= s.L) continue;
      // ---- scores of 16 keys
      float x[2][4] = {};
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const uint32_t row = src + static_cast<uint32_t>((8 * nt + g) * kRow);
        if (!E4M3) {
#pragma unroll
          for (int j = 0; j < DP / 32; ++j) {
            const uint4 b = lds128(row + 16u * static_cast<uint32_t>(k_piece<E4M3, DP>(g, 4 * j + c)));
            mma16816<F16>(x[nt], qf[0][j].x, qf[1][j].x, qf[0][j].y, qf[1][j].y, b.x, b.y);
            mma16816<F16>(x[nt], qf[0][j].z, qf[1][j].z, qf[0][j].w, qf[1][j].w, b.z, b.w);
          }
        } else {
#pragma unroll
          for (int j = 0; j < DP / 64; ++j) {
            const uint4 b = lds128(row + 16u * static_cast<uint32_t>(k_piece<E4M3, DP>(g, 4 * j + c)));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t w = word(b, i);
              const uint4 &u = qf[0][2 * j + (i >> 1)], &v = qf[1][2 * j + (i >> 1)];
              mma16816<true>(x[nt], word(u, 2 * (i & 1)), word(v, 2 * (i & 1)), word(u, 2 * (i & 1) + 1),
                             word(v, 2 * (i & 1) + 1), e4m3x2_f16x2(w & 0xFFFFu), e4m3x2_f16x2(w >> 16));
            }
          }
        }
      }
      float vs[4] = {1.f, 1.f, 1.f, 1.f};  // 8-bit: scales of this lane's keys, 2 c, 2 c + 1, 2 c + 8, 2 c + 9
      float ks[4] = {1.f, 1.f, 1.f, 1.f};
      if (E4M3) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const uint2 u = lds64(src + static_cast<uint32_t>(2 * kKeys * kRow + 4 * (8 * nt + 2 * c)));
          const uint2 v = lds64(src + static_cast<uint32_t>(2 * kKeys * kRow + 4 * (kKeys + 8 * nt + 2 * c)));
          ks[2 * nt] = __uint_as_float(u.x);
          ks[2 * nt + 1] = __uint_as_float(u.y);
          vs[2 * nt] = __uint_as_float(v.x);
          vs[2 * nt + 1] = __uint_as_float(v.y);
        }
      }
      // ---- maxima
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = e >> 1, key = key0 + 8 * nt + 2 * c + (e & 1);
          float z = x[nt][e] * factor[i];
          if (E4M3) z *= ks[2 * nt + (e & 1)];
          x[nt][e] = key <= limit[i] ? z : -INFINITY;
          top[i] = fmaxf(top[i], x[nt][e]);
        }
      float grown = 0.f;  // 8-bit: the unit's new value
      if (E4M3) {
        float most = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key0 + 8 * (e >> 1) + 2 * c + (e & 1) < s.L && fabsf(vs[e]) < INFINITY) most = fmaxf(most, fabsf(vs[e]));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        if (most >= unit) grown = __uint_as_float(min((__float_as_uint(most) & 0x7F800000u) + 0x00800000u, 0x7F000000u));
      }
      float keep[2];
      bool rescale = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
        const float next = fmaxf(m[i], top[i]);
        keep[i] = exp2_fast(m[i] - reference(next));
        rescale = rescale || next != m[i];
        m[i] = next;
      }
      float shrink = 1.f;
      if (E4M3 && grown > unit) {
        shrink = unit / grown;
        unit = grown;
        per_unit = 1.f / grown;
        rescale = true;
      }
      if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[i] *= keep[i];
          keep[i] *= shrink;
        }
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] *= keep[e >> 1];
      }
      // ---- weights
      uint32_t p[2][2];  // [key tile][row]
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float r = reference(m[i]);
          float u = exp2_fast(x[nt][2 * i] - r), v = exp2_fast(x[nt][2 * i + 1] - r);
          l[i] += u + v;
          if (E4M3) {  // (a masked key's weight is zero whatever its scale is)
            const int key = key0 + 8 * nt + 2 * c;
            u = key <= limit[i] ? u * (vs[2 * nt] * per_unit) : 0.f;
            v = key + 1 <= limit[i] ? v * (vs[2 * nt + 1] * per_unit) : 0.f;
          }
          p[nt][i] = F16 ? pack_half(u, v) : pack_bf16x2(u, v);
        }
      // ---- their sum of values
      const bool partly = key0 + kKeys - 1 > least;  // some row does not see some key
      const uint32_t values = src + static_cast<uint32_t>(kKeys * kRow);
      // a value that is not finite must not reach the rows that do not see it (0 *
      // NaN): it is taken out of the product and added to the others below
      uint32_t odd = 0;
      auto tame = [&](uint32_t w) {
        constexpr uint32_t e = F16 ? 0x7C00u : 0x7F80u;
        if ((w & e) == e) {
          odd = 1;
          w &= 0xFFFF0000u;
        }
        if ((w >> 16 & e) == e) {
          odd = 1;
          w &= 0xFFFFu;
        }
        return w;
      };
      if (!E4M3) {
        const int row = (lane >> 3 & 1) * 8 + (lane & 7);
#pragma unroll
        for (int j = 0; j < kTiles / 2; ++j) {
          uint4 b = ldmatrix_x4_trans(values + static_cast<uint32_t>(row * kRow + 16 * v_piece<E4M3, DP>(row, 2 * j + (lane >> 4))));
          if (partly) b = make_uint4(tame(b.x), tame(b.y), tame(b.z), tame(b.w));
          mma16816<F16>(o[2 * j], p[0][0], p[0][1], p[1][0], p[1][1], b.x, b.y);
          mma16816<F16>(o[2 * j + 1], p[0][0], p[0][1], p[1][0], p[1][1], b.z, b.w);
        }
      } else {
        uint32_t code[4][W / 4];  // rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9 at W g
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = 8 * (k >> 1) + 2 * c + (k & 1);
          if (DP == 128) {
            const uint4 u = lds128(values + static_cast<uint32_t>(key * kRow + 16 * v_piece<E4M3, DP>(key, g)));
#pragma unroll
            for (int i = 0; i < W / 4; ++i) code[k][i] = word(u, i);
          } else {
            const uint2 u = lds64(values + static_cast<uint32_t>(key * kRow + 8 * g));
            code[k][0] = u.x;
            code[k][1] = u.y;
          }
        }
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
          const uint32_t lo[2] = {__byte_perm(code[0][i], code[1][i], 0x5140), __byte_perm(code[0][i], code[1][i], 0x7362)};
          const uint32_t hi[2] = {__byte_perm(code[2][i], code[3][i], 0x5140), __byte_perm(code[2][i], code[3][i], 0x7362)};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t b0 = e4m3x2_f16x2(e & 1 ? lo[e >> 1] >> 16 : lo[e >> 1] & 0xFFFFu);
            uint32_t b1 = e4m3x2_f16x2(e & 1 ? hi[e >> 1] >> 16 : hi[e >> 1] & 0xFFFFu);
            if (partly) {
              b0 = tame(b0);
              b1 = tame(b1);
            }
            mma16816<true>(o[4 * i + e], p[0][0], p[0][1], p[1][0], p[1][1], b0, b1);
          }
        }
      }
      if (partly && __any_sync(0xffffffffu, odd)) {
#pragma unroll 1
        for (int key = 0; key < kKeys; ++key) {
#pragma unroll
          for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int d = E4M3 ? W * (2 * c + e) + j : 8 * j + 2 * c + e;
              float v;
              if (E4M3) {
                const uint32_t at = values + static_cast<uint32_t>(
                    DP == 128 ? key * kRow + 16 * v_piece<E4M3, DP>(key, d >> 4) + (d & 15) : key * kRow + d);
                uint16_t q;
                asm volatile("ld.shared.u8 %0, [%1];" : "=h"(q) : "r"(at) : "memory");
                v = (q & 0x7F) == 0x7F ? NAN : 0.f;
              } else {
                uint16_t q;
                asm volatile("ld.shared.u16 %0, [%1];"
                             : "=h"(q)
                             : "r"(values + static_cast<uint32_t>(key * kRow + 16 * v_piece<E4M3, DP>(key, d >> 3) + 2 * (d & 7)))
                             : "memory");
                v = f32_of(q, F16);
              }
              if (!(fabsf(v) < INFINITY)) {
                if (key0 + key <= limit[0]) o[j][e] += v;
                if (key0 + key <= limit[1]) o[j][2 + e] += v;
              }
            }
        }
      }
    }

    // ---- the warps' sums joined
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    if (E4M3) {
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] *= unit;
    }
    auto column = [&](int j, int e) { return E4M3 ? W * (2 * c + e) + j : 8 * j + 2 * c + e; };
    // eight columns of a row stay adjacent; rows lie in different banks
    auto place = [&](int buf, int row, int d, int per) { return join + (buf * per + row) * DP + (d ^ ((row & 3) << 3)); };
    auto put = [&](int buf, int per) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = g + 8 * i;
        if (row < live) {
#pragma unroll
          for (int j = 0; j < kTiles; ++j) {
            if (E4M3) {
              *place(buf, row, column(j, 0), per) = o[j][2 * i];
              *place(buf, row, column(j, 1), per) = o[j][2 * i + 1];
            } else {
              *reinterpret_cast<float2*>(place(buf, row, column(j, 0), per)) = make_float2(o[j][2 * i], o[j][2 * i + 1]);
            }
          }
          if (c == 0) {
            ms[buf * kRows + row] = m[i];
            ls[buf * kRows + row] = l[i];
          }
        }
      }
    };
    const bool two = live > 8;  // four buffers of 16 rows, or eight of 8
    const int per = two ? 16 : 8, bufs = two ? 4 : 8;
    __syncthreads();  // the last item's sums have been read
    if (two) {
      if (warp >= 4) put(warp - 4, per);
      __syncthreads();
      if (warp < 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = g + 8 * i;
          if (row < live) {
            const float om = ms[warp * kRows + row], both = fmaxf(m[i], om), r = reference(both);
            const float mine = exp2_fast(m[i] - r), other = exp2_fast(om - r);
            l[i] = l[i] * mine + ls[warp * kRows + row] * other;
            m[i] = both;
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                o[j][2 * i + e] = o[j][2 * i + e] * mine + *place(warp, row, column(j, e), per) * other;
          }
        }
      }
      __syncthreads();
      if (warp < 4) put(warp, per);
    } else {
      put(warp, per);
    }
    __syncthreads();
    constexpr int kChunks = DP / 8;  // threads of a row, eight columns each
    const int row = tid / kChunks, d0 = 8 * (tid % kChunks);
    const bool mine = row < live;
    float v[8], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    if (mine) {
      for (int i = 0; i < bufs; ++i) top = fmaxf(top, ms[i * kRows + row]);
      const float r = reference(top);
      for (int i = 0; i < bufs; ++i) {
        const float f = exp2_fast(ms[i * kRows + row] - r);
        sum += ls[i * kRows + row] * f;
        const float* from = place(i, row, d0, per);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = fmaf(from[j], f, v[j]);
      }
    }
    bool write = true;
    if (cur.end - cur.t < cur.len) {
      // the item lies in several runs: the last one to finish joins them
      const int first = cur.first_cta(), pieces = cur.cta_count();
      constexpr size_t kPiece = attn_piece_bytes(kRows, DP) / 4;
      auto piece = [&](int i) { return a.partial + (2 * (first + i) + (i == 0 ? 1 : 0)) * kPiece; };
      float* to = piece(static_cast<int>(blockIdx.x) - first);
      if (mine) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          __stcg(reinterpret_cast<float4*>(to + row * DP + d0) + j, make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
        if (d0 == 0) {
          __stcg(to + kRows * DP + 2 * row, top);
          __stcg(to + kRows * DP + 2 * row + 1, sum);
        }
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        last = atomicAdd(a.tickets + first, 1u) == static_cast<uint32_t>(pieces - 1);
        if (last) a.tickets[first] = 0;
        __threadfence();
      }
      __syncthreads();
      write = last != 0;
      if (write && mine) {
        top = -INFINITY;
        for (int i = 0; i < pieces; ++i) top = fmaxf(top, __ldcg(piece(i) + kRows * DP + 2 * row));
        const float r = reference(top);
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll 2
        for (int i = 0; i < pieces; ++i) {
          const float* from = piece(i);
          const float f = exp2_fast(__ldcg(from + kRows * DP + 2 * row) - r);
          sum = fmaf(__ldcg(from + kRows * DP + 2 * row + 1), f, sum);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float4 u = __ldcg(reinterpret_cast<const float4*>(from + row * DP + d0) + j);
            v[4 * j] = fmaf(u.x, f, v[4 * j]);
            v[4 * j + 1] = fmaf(u.y, f, v[4 * j + 1]);
            v[4 * j + 2] = fmaf(u.z, f, v[4 * j + 2]);
            v[4 * j + 3] = fmaf(u.w, f, v[4 * j + 3]);
          }
        }
      }
    }
    if (write && mine) {
      const int R = cur.r * kRows + row;
      const int token = divided(R, a.G), head = cur.h * a.G + R - token * a.G;
      if (d0 < a.D) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = a.f16 ? pack_half(v[2 * j] / sum, v[2 * j + 1] / sum) : pack_bf16x2(v[2 * j] / sum, v[2 * j + 1] / sum);
        *reinterpret_cast<uint4*>(a.out + (s.row0 + token) * a.out_stride + static_cast<int64_t>(head) * a.D + d0) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (d0 == 0 && a.lse != nullptr)
        a.lse[static_cast<int64_t>(s.row0 + token) * a.Hq + head] = (top + log2_fast(sum)) * 0.69314718055994531f;
    }
    going = cur.next(a);
  }
}

template <bool E4M3, bool F16, int DP>
cudaError_t launch(const AttnArgs& a, int sms, cudaStream_t s) {
  auto kernel = attention_few_kernel<E4M3, F16, DP>;
  static int configured[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64 || configured[dev] == 0) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem) - 1024);
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  const size_t fixed = (join_bytes(DP) + kMiscBytes + 127) / 128 * 128;
  const int most = static_cast<int>((kSmem - 1024 - fixed) / (kWarps * stage_bytes(E4M3, DP)));
  const int depth = most < kMaxDepth ? most : kMaxDepth;
  return launch_pdl(kernel, dim3(sms < kAttnMaxCtas ? sms : kAttnMaxCtas), dim3(kThreads),
                    fixed + static_cast<size_t>(kWarps) * depth * stage_bytes(E4M3, DP), s, a, depth);
}

template <bool E4M3, bool F16>
cudaError_t launch(const AttnArgs& a, int sms, cudaStream_t s) {
  return a.D <= 64 ? launch<E4M3, F16, 64>(a, sms, s) : launch<E4M3, F16, 128>(a, sms, s);
}

}  // namespace

cudaError_t launch_attention_few(const AttnArgs& a, int sms, cudaStream_t s) {
  if (a.e4m3) return launch<true, true>(a, sms, s);
  return a.f16 ? launch<false, true>(a, sms, s) : launch<false, false>(a, sms, s);
}

}  // namespace moe
