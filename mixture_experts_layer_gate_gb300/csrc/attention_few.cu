// Attention of few rows (single tokens, drafted tokens: at most 16 rows of a key
// head's queries): every key and value is read once and used by all rows, so the bound
// is memory, and the products are mma.sync m16n8k16 with 16 keys, or 16 places of the
// head, as M and 8 rows as N (tcgen05's smallest M is 64).  More rows go through tiles
// of 16, which is right but reads the keys once a tile.
//
// A tile is 16 keys for each warp.  A warp streams its keys and values through a ring
// of its own (cp.async, some tiles ahead, across items) and holds its own running
// maximum, sum and output, joined when the item ends: no warp waits for another inside
// an item.
//
// One pass over the keys: with m the largest score so far, l = sum 2^(x - m) and O =
// sum 2^(x - m) v, both multiplied by 2^(m - m') when it grows to m'.  Sums are float;
// weights are rounded to the values' 16-bit type before they multiply them (half a
// step of it, as the output's own rounding).  In f16 they are 2^14 times that: relative to
// m itself those under 2^-14 lost bits and those under 2^-25 all of them, which shows
// beside a key that takes nearly all of the weight and adds nothing.
//
// 8-bit cache: codes become f16, which is exact, and so do the queries after a
// power of two brings each row's largest value to 2^14 (what falls below f16's steps is
// under 2^-38 of that).  A key's scale multiplies its score.  A value's scale
// multiplies its weight, and m is then the largest score plus logarithm of the scale that
// the row sees (scale_log2), so that their product stays in f16's range; l is relative to
// the same m.  A largest scale of all keys instead took the weights of rows that do not
// see it, or give it no weight, into f16's subnormals.
//
// K is permuted inside the head (any order gives the same product) so that a lane's
// 16 adjacent bytes of a key are its fragment; 8-bit values are read along the head and
// paired across keys by byte permutes, which leaves each lane 16 adjacent outputs.
// Weights, made with a key a lane, become the second product's fragment by one
// transposition of 8 x 8 each.
//
// In a graph, 32 query and 8 key heads of 128: 256 sequences of 2000 keys 317 us, 98%
// of the measured copy's bandwidth; 64 sequences of 100 to 16384 142 us, 89%; with
// queries as M (16 rows whatever there are) 343 and 155.  e4m3: 256 of 2000 232 us =
// 4.7 TB/s, bound by the four instructions that a code's conversion takes.
#include "attention.cuh"
#include "stream.cuh"

namespace moe {
namespace {

using namespace attn;

constexpr int kMostRows = kAttnFewRows;
constexpr int kKeys = 16;  // of a warp's step
constexpr int kMaxDepth = 8;
constexpr size_t kSmem = 232448 - 1024;

// How far under the maximum f16 weights' reference lies: they reach 2^14.
template <bool F16>
constexpr float kLift = F16 ? 14.f : 0.f;

// Warps of a CTA: 8-bit keys take more instructions a byte, and up to 8 rows leave the
// registers for 16 warps.
template <bool E4M3, int NT>
constexpr int kWarpsOf = E4M3 && NT == 1 ? 16 : 8;

__host__ __device__ constexpr int row_bytes(bool e4m3, int dp) { return e4m3 ? dp : 2 * dp; }
// a step's keys and values, and their scales
__host__ __device__ constexpr int stage_bytes(bool e4m3, int dp) {
  return 2 * kKeys * row_bytes(e4m3, dp) + (e4m3 ? 2 * kKeys * 4 : 0);
}
// 64 rows of sums: of 8 warps with 8 rows, or 4 with 16 (twice, where there are more)
__host__ __device__ constexpr int join_bytes(int dp) { return 64 * dp * 4; }
constexpr int kStatBytes = 2 * 64 * 4;
constexpr int kMiscBytes = kStatBytes + kScratchWords * 8;

__device__ __forceinline__ void cp_async16_if(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16u : 0u) : "memory");
}
// Of an 8 x 8 matrix of 16-bit values, (row g, columns 2 c and 2 c + 1) a lane: the
// transposed one.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
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

// F16: the products' type (8-bit caches: always), else bf16.  NT: column tiles of 8 rows.
template <bool E4M3, bool F16, int DP, int NT>
__global__ void __launch_bounds__(32 * kWarpsOf<E4M3, NT>, 1) attention_few_kernel(const AttnArgs a, const int depth) {
  extern __shared__ __align__(128) uint8_t few_smem[];
  constexpr int kWarps = kWarpsOf<E4M3, NT>, kThreads = 32 * kWarps, kTile = kKeys * kWarps, kRows = 8 * NT;
  constexpr int kRow = row_bytes(E4M3, DP), kPieces = kRow / 16, kStage = stage_bytes(E4M3, DP);
  constexpr int kPerLoad = 32 / kPieces;  // keys that a load of the warp covers
  constexpr int MT = DP / 16;             // row tiles of the output: 16 places of the head
  constexpr int W = DP / 8;               // 8-bit: adjacent values a lane reads of a row
  using FewWalk = Walk<Shape<kRows, kTile, 1, 2, 4>>;
  __shared__ int last;
  float* join = reinterpret_cast<float*>(few_smem);  // [buffer][row][DP]
  float* ms = join + join_bytes(DP) / 4;             // [buffer][row]
  float* ls = ms + 64;
  int64_t* scratch = reinterpret_cast<int64_t*>(ls + 64);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(few_smem) + static_cast<uint32_t>((join_bytes(DP) + kMiscBytes + 127) / 128 * 128) +
                        static_cast<uint32_t>(warp * depth * kStage);
  pdl_wait();
  pdl_trigger();
  FewWalk cur;
  if (!start<kThreads>(a, scratch, cur)) {
    clear_empty_rows(a);
    return;
  }

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
  // this lane's first key and piece of the item's head
  constexpr int64_t size = E4M3 ? 1 : 2;
  const uint8_t *k_head, *v_head;
  auto enter = [&] {
    k_head = a.kv.k + size * (my_key * a.kv.k_token + iss.h * a.kv.k_head) + 16 * my_piece;
    v_head = a.kv.v + size * (my_key * a.kv.v_token + iss.h * a.kv.v_head) + 16 * my_piece;
  };
  enter();
  const int64_t k_step = size * kPerLoad * a.kv.k_token, v_step = size * kPerLoad * a.kv.v_token;
  auto issue = [&] {
    if (more) {
      const int key0 = iss.t * kTile + warp * kKeys;
      const uint32_t dst = ring + static_cast<uint32_t>(slot_i * kStage);
      if (key0 < iss.s.L) {
        const bool good = page >= 0 && page < a.num_pages;
        if (!good && lane == 0) record_error(a.err, kErrBadIndex, static_cast<uint32_t>(iss.b));
        const int64_t place = paged ? (key0 & page_mask) : static_cast<int64_t>(iss.s.row0 + key0);
        const int64_t from = good ? page : 0;
        const uint8_t* k = k_head + size * (from * a.kv.k_page + place * a.kv.k_token);
        const uint8_t* v = v_head + size * (from * a.kv.v_page + place * a.kv.v_token);
        auto k_at = [&](int i) {
          const int key = i * kPerLoad + my_key;
          return dst + static_cast<uint32_t>(key * kRow + 16 * k_piece<E4M3, DP>(key, my_piece));
        };
        auto v_at = [&](int i) {
          const int key = i * kPerLoad + my_key;
          return dst + static_cast<uint32_t>((kKeys + key) * kRow + 16 * v_piece<E4M3, DP>(key, my_piece));
        };
        if (good && key0 + kKeys <= iss.s.L && a.D == DP) {
#pragma unroll
          for (int i = 0; i < kKeys / kPerLoad; ++i, k += k_step, v += v_step) {
            cp_async16(k_at(i), k);
            cp_async16(v_at(i), v);
          }
        } else {
          const int there = good && in_head ? iss.s.L - key0 - my_key : 0;  // keys of this lane's column of loads
#pragma unroll 1
          for (int i = 0; i < kKeys / kPerLoad; ++i, k += k_step, v += v_step) {
            const bool in = i * kPerLoad < there;
            cp_async16_if(k_at(i), in ? k : a.kv.k, in);
            cp_async16_if(v_at(i), in ? v : a.kv.v, in);
          }
        }
        if (E4M3 && lane < 8) {
          const float* s = lane < 4 ? a.kv.k_scale : a.kv.v_scale;
          const int64_t at = ((from * a.Hkv + iss.h) << a.page_shift) + place + 4 * (lane & 3);
          cp_async16_if(dst + static_cast<uint32_t>(2 * kKeys * kRow + 16 * lane), good ? s + at : s, good);
        }
      }
      if (++iss.t == iss.end) {
        more = iss.next(a);
        enter();
      }
      if (more) page = page_of(iss);
    }
    cp_async_commit();
    if (++slot_i == depth) slot_i = 0;
  };
  for (int i = 0; i < depth - 1; ++i) issue();

  int slot = 0;
  bool going = true;
  while (going) {
    // ---- an item.  As fragments of the first product a lane holds row g (of each
    // tile), everywhere else rows 2 c and 2 c + 1.
    const Seq s = cur.s;
    const int live = min(s.n * a.G - cur.r * kRows, kRows);
    uint4 qf[NT][DP / 32];
    int limit[NT][2];  // the last key that the row sees
    float factor[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool there = 8 * nt + g < live;
      const int R = cur.r * kRows + (there ? 8 * nt + g : 0);
      const int token = divided(R, a.G), head = cur.h * a.G + R - token * a.G;
      const int sees = there ? s.past + token : -1;
      float f = a.scale_log2;
      const uint16_t* q = a.q + (s.row0 + token) * a.q_stride + static_cast<int64_t>(head) * a.D;
#pragma unroll
      for (int j = 0; j < DP / 32; ++j) {
        // 16-bit: 8 values at 32 j + 8 c; 8-bit: of 16 values at 64 (j / 2) + 16 c the half j % 2
        const int d = E4M3 ? 64 * (j >> 1) + 16 * c + 8 * (j & 1) : 32 * j + 8 * c;
        qf[nt][j] = there && d < a.D ? *reinterpret_cast<const uint4*>(q + d) : make_uint4(0, 0, 0, 0);
      }
      if (E4M3) {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < DP / 32; ++j) {
          const uint32_t w[4] = {qf[nt][j].x, qf[nt][j].y, qf[nt][j].z, qf[nt][j].w};
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
        if (scaled) f *= __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
#pragma unroll
        for (int j = 0; j < DP / 32; ++j) {
          uint32_t* w = &qf[nt][j].x;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = pack_half(f32_of(static_cast<uint16_t>(w[k]), a.f16) * up,
                             f32_of(static_cast<uint16_t>(w[k] >> 16), a.f16) * up);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // (row 2 c + i is row g of lane 4 (2 c + i))
        limit[nt][i] = __shfl_sync(0xffffffffu, sees, 4 * (2 * c + i));
        factor[nt][i] = __shfl_sync(0xffffffffu, f, 4 * (2 * c + i));
      }
    }
    const int least = s.past + divided(cur.r * kRows, a.G);  // of all rows' limits
    float o[MT][NT][4];  // places (16-bit: 16 j + g, + 8; 8-bit: W g + 2 j, + 1) of rows 2 c, 2 c + 1
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][nt][e] = 0.f;
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[nt][i] = -INFINITY;
        l[nt][i] = 0.f;
      }

    for (int t = cur.t; t < cur.end; ++t) {
      cp_async_wait(depth - 2);
      __syncwarp();
      issue();
      const int key0 = t * kTile + warp * kKeys;
      const uint32_t src = ring + static_cast<uint32_t>(slot * kStage);
      if (++slot == depth) slot = 0;
      if (key0 >= s.L) continue;
      // ---- scores of keys g and g + 8
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nt][e] = 0.f;
      const uint32_t row_a = src + static_cast<uint32_t>(g * kRow), row_b = row_a + static_cast<uint32_t>(8 * kRow);
      if (!E4M3) {
#pragma unroll
        for (int j = 0; j < DP / 32; ++j) {
          const uint32_t at = 16u * static_cast<uint32_t>(k_piece<E4M3, DP>(g, 4 * j + c));
          const uint4 u = lds128(row_a + at), v = lds128(row_b + at);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816<F16>(x[nt], u.x, v.x, u.y, v.y, qf[nt][j].x, qf[nt][j].y);
            mma16816<F16>(x[nt], u.z, v.z, u.w, v.w, qf[nt][j].z, qf[nt][j].w);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < DP / 64; ++j) {
          const uint32_t at = 16u * static_cast<uint32_t>(k_piece<E4M3, DP>(g, 4 * j + c));
          const uint4 u = lds128(row_a + at), v = lds128(row_b + at);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t p = word(u, i), q = word(v, i);
            const uint32_t a0 = e4m3x2_f16x2(p & 0xFFFFu), a1 = e4m3x2_f16x2(q & 0xFFFFu), a2 = e4m3x2_f16x2(p >> 16),
                           a3 = e4m3x2_f16x2(q >> 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint4& b = qf[nt][2 * j + (i >> 1)];
              mma16816<true>(x[nt], a0, a1, a2, a3, word(b, 2 * (i & 1)), word(b, 2 * (i & 1) + 1));
            }
          }
        }
      }
      float ks[2] = {1.f, 1.f}, vs[2] = {1.f, 1.f}, more_by[2] = {0.f, 0.f};  // 8-bit: of keys g, g + 8
      if (E4M3) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t u, v;
          const uint32_t at = src + static_cast<uint32_t>(2 * kKeys * kRow + 4 * (8 * i + g));
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(u) : "r"(at) : "memory");
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at + 4 * kKeys) : "memory");
          ks[i] = __uint_as_float(u);
          vs[i] = __uint_as_float(v);
          more_by[i] = scale_log2(vs[i]);
        }
      }
      // ---- maxima
      float keep[NT][2];
      bool rescale = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float z = x[nt][2 * k + i] * factor[nt][i];
            if (E4M3) z *= ks[k];
            x[nt][2 * k + i] = key0 + 8 * k + g <= limit[nt][i] ? z : -INFINITY;
          }
          float top = E4M3 ? fmaxf(x[nt][i] + more_by[0], x[nt][2 + i] + more_by[1]) : fmaxf(x[nt][i], x[nt][2 + i]);
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
          const float next = fmaxf(m[nt][i], top);
          const float shift = m[nt][i] - reference(next);
          keep[nt][i] = exp2_fast(E4M3 ? 0.5f * shift : shift);
          rescale = rescale || next != m[nt][i];
          m[nt][i] = next;
        }
      if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            l[nt][i] *= keep[nt][i];
            if (E4M3) {  // (l may be large: twice half of the exponent)
              l[nt][i] *= keep[nt][i];
              keep[nt][i] *= keep[nt][i];
            }
          }
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][nt][e] *= keep[nt][e & 1];
      }
      // ---- weights
      uint32_t p[NT][2];  // keys 2 c, 2 c + 1 (+ 8) of row g
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float u = exp2_fast(x[nt][2 * k] - reference(m[nt][0], kLift<F16>));
          float v = exp2_fast(x[nt][2 * k + 1] - reference(m[nt][1], kLift<F16>));
          l[nt][0] += u;
          l[nt][1] += v;
          if (E4M3) {  // (a masked key's weight is zero whatever its scale is)
            u = key0 + 8 * k + g <= limit[nt][0] ? u * vs[k] : 0.f;
            v = key0 + 8 * k + g <= limit[nt][1] ? v * vs[k] : 0.f;
          }
          p[nt][k] = transposed(F16 ? pack_half(u, v) : pack_bf16x2(u, v));
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
      auto add = [&](int j, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
        if (partly) a0 = tame(a0), a1 = tame(a1), a2 = tame(a2), a3 = tame(a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816<F16>(o[j][nt], a0, a1, a2, a3, p[nt][0], p[nt][1]);
      };
      if (!E4M3) {
        // matrices: places 0-7 and 8-15 of keys 0-7, then of keys 8-15
        const int key = (lane >> 4) * 8 + (lane & 7);
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const uint4 b = ldmatrix_x4_trans(
              values + static_cast<uint32_t>(key * kRow + 16 * v_piece<E4M3, DP>(key, 2 * j + (lane >> 3 & 1))));
          add(j, b.x, b.y, b.z, b.w);
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
        for (int i = 0; i < W / 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // places W g + 4 i + 2 e and the next
            const uint32_t sel = e == 0 ? 0x5140 : 0x7362;
            const uint32_t lo = __byte_perm(code[0][i], code[1][i], sel), hi = __byte_perm(code[2][i], code[3][i], sel);
            add(2 * i + e, e4m3x2_f16x2(lo & 0xFFFFu), e4m3x2_f16x2(lo >> 16), e4m3x2_f16x2(hi & 0xFFFFu), e4m3x2_f16x2(hi >> 16));
          }
      }
      if (partly && __any_sync(0xffffffffu, odd)) {
#pragma unroll 1
        for (int key = 0; key < kKeys; ++key) {
#pragma unroll
          for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int d = E4M3 ? W * g + 2 * j + e : 16 * j + 8 * e + g;
              float v;
              uint16_t q;
              if (E4M3) {
                const uint32_t at = values + static_cast<uint32_t>(
                    DP == 128 ? key * kRow + 16 * v_piece<E4M3, DP>(key, d >> 4) + (d & 15) : key * kRow + d);
                asm volatile("ld.shared.u8 %0, [%1];" : "=h"(q) : "r"(at) : "memory");
                v = (q & 0x7F) == 0x7F ? NAN : 0.f;
              } else {
                asm volatile("ld.shared.u16 %0, [%1];"
                             : "=h"(q)
                             : "r"(values + static_cast<uint32_t>(key * kRow + 16 * v_piece<E4M3, DP>(key, d >> 3) + 2 * (d & 7)))
                             : "memory");
                v = f32_of(q, F16);
              }
              if (!(fabsf(v) < INFINITY)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int i = 0; i < 2; ++i)
                    if (key0 + key <= limit[nt][i]) o[j][nt][2 * e + i] += v;
              }
            }
        }
      }
    }

    // ---- the warps' sums joined
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], w);
    constexpr int kBufs = 64 / kRows;          // buffers of kRows rows
    constexpr int kTurns = kWarps / kBufs;     // 1, or 2: the second half of the warps first
    static_assert(kTurns == 1 || kTurns == 2, "each warp has a buffer, or half of them");
    // eight places of a row stay adjacent; the rows of four lanes lie in different banks
    auto at = [&](int buf, int row, int d) { return join + (buf * kRows + row) * DP + (d ^ ((row >> 1 & 3) << 3)); };
    auto put = [&](int buf) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 8 * nt + 2 * c + i;
          if (row < live) {
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              if (E4M3) {
                *reinterpret_cast<float2*>(at(buf, row, W * g + 2 * j)) = make_float2(o[j][nt][i], o[j][nt][2 + i]);
              } else {
                *at(buf, row, 16 * j + g) = o[j][nt][i];
                *at(buf, row, 16 * j + 8 + g) = o[j][nt][2 + i];
              }
            }
            if (g == 0) {
              ms[buf * kRows + row] = m[nt][i];
              ls[buf * kRows + row] = l[nt][i];
            }
          }
        }
    };
    __syncthreads();  // the last item's sums have been read
    if (kTurns == 2) {
      if (warp >= kBufs) put(warp - kBufs);
      __syncthreads();
      if (warp < kBufs) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int row = 8 * nt + 2 * c + i;
            if (row < live) {
              const float om = ms[warp * kRows + row], both = fmaxf(m[nt][i], om), r = reference(both);
              const float mine = exp2_fast(m[nt][i] - r), other = exp2_fast(om - r);
              l[nt][i] = moved<E4M3>(l[nt][i], m[nt][i] - r, mine) + moved<E4M3>(ls[warp * kRows + row], om - r, other);
              m[nt][i] = both;
#pragma unroll
              for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int d = E4M3 ? W * g + 2 * j + e : 16 * j + 8 * e + g;
                  o[j][nt][2 * e + i] = o[j][nt][2 * e + i] * mine + *at(warp, row, d) * other;
                }
            }
          }
      }
      __syncthreads();
    }
    if (warp < kBufs) put(warp);
    __syncthreads();
    constexpr int kChunks = DP / 8;  // threads of a row, eight places each
    const int row = tid / kChunks, d0 = 8 * (tid % kChunks);
    const bool mine = row < live;
    float v[8], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    if (mine) {
#pragma unroll
      for (int i = 0; i < kBufs; ++i) top = fmaxf(top, ms[i * kRows + row]);
      const float r = reference(top);
#pragma unroll
      for (int i = 0; i < kBufs; ++i) {
        const float f = exp2_fast(ms[i * kRows + row] - r);
        sum += moved<E4M3>(ls[i * kRows + row], ms[i * kRows + row] - r, f);
        const float* from = at(i, row, d0);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = fmaf(from[j], f, v[j]);
      }
    }
    bool write = true;
    if (cur.end - cur.t < cur.len) {
      // the item lies in several runs: the last one to finish joins them
      const int first = cur.first_cta(), pieces = cur.cta_count();
      constexpr size_t kPiece = attn_piece_bytes(kMostRows, DP) / 4;
      auto piece = [&](int i) { return a.partial + (2 * (first + i) + (i == 0 ? 1 : 0)) * kPiece; };
      const int me = static_cast<int>(blockIdx.x) - first;
      write = false;
      int to = me;  // the piece that this CTA writes
#pragma unroll 1
      for (int level = 0; !write; ++level) {
        float* p = piece(to);
        if (mine) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            __stcg(reinterpret_cast<float4*>(p + row * DP + d0) + j, make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
          if (d0 == 0) __stcg(reinterpret_cast<float2*>(p + kMostRows * DP + 2 * row), make_float2(top, sum));
        }
        const Join j = join_of(a, first, pieces, me, level);
        __threadfence();
        __syncthreads();
        if (tid == 0) last = count_in(j);
        __syncthreads();
        if (last == 0) break;
        if (mine) {
          top = -INFINITY;
#pragma unroll 8
          for (int i = 0; i < j.count; ++i)
            top = fmaxf(top, __ldcg(piece(j.base + i * j.stride) + kMostRows * DP + 2 * row));
          const float r = reference(top);
          sum = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll 8
          for (int i = 0; i < j.count; ++i) {
            const float* from = piece(j.base + i * j.stride);
            const float2 stat = __ldcg(reinterpret_cast<const float2*>(from + kMostRows * DP + 2 * row));
            const float4 u = __ldcg(reinterpret_cast<const float4*>(from + row * DP + d0));
            const float4 z = __ldcg(reinterpret_cast<const float4*>(from + row * DP + d0) + 1);
            const float f = exp2_fast(stat.x - r);
            sum += moved<E4M3>(stat.y, stat.x - r, f);
            v[0] = fmaf(u.x, f, v[0]);
            v[1] = fmaf(u.y, f, v[1]);
            v[2] = fmaf(u.z, f, v[2]);
            v[3] = fmaf(u.w, f, v[3]);
            v[4] = fmaf(z.x, f, v[4]);
            v[5] = fmaf(z.y, f, v[5]);
            v[6] = fmaf(z.z, f, v[6]);
            v[7] = fmaf(z.w, f, v[7]);
          }
        }
        write = j.last;
        to = j.base;
        __syncthreads();  // (all have read the group's pieces before its sum takes the first one's place)
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
        a.lse[static_cast<int64_t>(s.row0 + token) * a.Hq + head] = (top - kLift<F16> + log2_fast(sum)) * 0.69314718055994531f;
    }
    going = cur.next(a);
  }
  clear_empty_rows(a);
}

template <bool E4M3, bool F16, int DP, int NT>
cudaError_t launch(const AttnArgs& a, int sms, cudaStream_t s) {
  auto kernel = attention_few_kernel<E4M3, F16, DP, NT>;
  constexpr int kWarps = kWarpsOf<E4M3, NT>;
  static int configured[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64 || configured[dev] == 0) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  const size_t fixed = (join_bytes(DP) + kMiscBytes + 127) / 128 * 128;
  const int most = static_cast<int>((kSmem - fixed) / (kWarps * stage_bytes(E4M3, DP)));
  const int depth = most < kMaxDepth ? most : kMaxDepth;
  return launch_pdl(kernel, dim3(sms < kAttnMaxCtas ? sms : kAttnMaxCtas), dim3(32 * kWarps),
                    fixed + static_cast<size_t>(kWarps) * depth * stage_bytes(E4M3, DP), s, a, depth);
}

template <bool E4M3, bool F16, int DP>
cudaError_t launch(const AttnArgs& a, int rows, int sms, cudaStream_t s) {
  return rows <= 8 ? launch<E4M3, F16, DP, 1>(a, sms, s) : launch<E4M3, F16, DP, 2>(a, sms, s);
}

template <bool E4M3, bool F16>
cudaError_t launch(const AttnArgs& a, int rows, int sms, cudaStream_t s) {
  return a.D <= 64 ? launch<E4M3, F16, 64>(a, rows, sms, s) : launch<E4M3, F16, 128>(a, rows, sms, s);
}

}  // namespace

cudaError_t launch_attention_few(const AttnArgs& a, int rows, int sms, cudaStream_t s) {
  if (a.e4m3) return launch<true, true>(a, rows, sms, s);
  return a.f16 ? launch<false, true>(a, rows, sms, s) : launch<false, false>(a, rows, sms, s);
}

}  // namespace moe
