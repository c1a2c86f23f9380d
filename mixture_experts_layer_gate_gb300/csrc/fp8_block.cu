// Product of e4m3 operands with a scale per block of 128 (moe_gemm_fp8_block,
// moe_gemm_fp8_block_swiglu): out[m, n] = sum_b a_scale[m, b] w_scale[n / 128, b]
// sum_{k in b} a[m, k] w[n, k].  A k-block of the dense kernel is a scale block,
// so each accumulator is one block's product and is joined to the sums in
// registers with one multiply-add per value.
#include "dense.cuh"

namespace moe {
namespace {

struct Choice {
  int bn, pair, P;
};

// Tiles, pairs and the split of K.  Large batches: CTA pairs on 256 x 256 tiles.
// Else the width and split that spread the tile's weights over the SMs.
Choice choose(const Fp8GemmArgs& g, bool swiglu, int KB, int sms) {
  const int cols = g.N;
  const int bn_full = swiglu ? 128 : 256;
  const int mt = (g.M + 127) / 128;
  const long long pair_tiles = static_cast<long long>((g.M + 255) / 256) * ((cols + bn_full - 1) / bn_full);
  if (g.M > 128 && pair_tiles * 2 >= sms * 3 / 4) return {256, 1, 1};
  Choice best{256, 0, 1};
  double best_time = 1e30;
  for (int bn : {32, 64, 128, 256}) {
    if (swiglu && bn != 256) continue;
    const long long tiles = static_cast<long long>(mt) * ((cols + (swiglu ? 128 : bn) - 1) / (swiglu ? 128 : bn));
    for (int P : {1, 2, 4, 8}) {
      if (P > KB) continue;
      const long long waves = (tiles * P + sms - 1) / sms;
      const double load = 128.0 * (bn + std::min(128, g.M)) / 48.0;  // cycles to load a k-block
      const double time = static_cast<double>(waves) * (((KB + P - 1) / P) * std::max(load, 2.0 * bn) + 1500.0) +
                          (P > 1 ? 1200.0 + 4.0 * P * std::min(128, g.M) / P : 0.0);
      if (time < best_time * 0.999) {
        best_time = time;
        best = {bn, 0, P};
      }
    }
  }
  return best;
}

}  // namespace

cudaError_t launch_fp8_block(const Fp8GemmArgs& g, cudaStream_t s) {
  const bool swiglu = g.codes != nullptr;
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  const int KB = (g.K + 127) / 128;
  const Choice c = choose(g, swiglu, KB, di.sms);
  dense::Params p = {};
  p.a_scale = g.a_scale;
  p.w_scale = g.w_scale;
  p.out = g.out;
  p.codes = g.codes;
  p.scales = g.scales;
  p.err = g.err;
  p.a_scale_stride = g.a_scale_stride;
  p.out_stride = g.out_stride;
  p.M = g.M;
  p.N = g.N;
  p.KB = KB;
  p.group = 1;
  p.P = c.P;
  p.out_dtype = g.out_dtype;
  p.accumulate = g.accumulate;
  const int64_t osz = g.out_dtype == 2 ? 4 : 2;
  p.vec = reinterpret_cast<uintptr_t>(g.out) % 16 == 0 && g.out_stride * osz % 16 == 0;
  p.vec_scale = reinterpret_cast<uintptr_t>(g.a_scale) % 16 == 0 && g.a_scale_stride % 4 == 0 && c.P == 1;
  return dense::plan_and_launch<dense::kE4M3>(p, c.bn, c.pair, swiglu, g.a, g.a_stride, g.w, g.w_stride,
                                              swiglu ? 2 * g.N : g.N, g.K, di.sms, s);
}

}  // namespace moe
