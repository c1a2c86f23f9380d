// Product of e4m3 operands with a scale per block of 128 (moe_gemm_fp8_block,
// moe_gemm_fp8_block_swiglu): out[m, n] = sum_b a_scale[m, b] w_scale[n / 128, b]
// sum_{k in b} a[m, k] w[n, k].  A k-block of the dense kernel is a scale block,
// so each accumulator is one block's product and is joined to the sums in
// registers with one multiply-add per value.  Measured in a graph: SwiGLU, M = 4096,
// K = 7168, N = 2048 103 us = 2.3 PFLOP/s; M = 4096, K = 2048, N = 7168 51 us = 2.3
// PFLOP/s, added to out 62 us (bound by the joining warps, which take ~800 cycles
// for a k-block of a CTA pair, its MMAs ~690, and by the last round of tiles).
#include "dense.cuh"

namespace moe {
cudaError_t launch_fp8_block(const Fp8GemmArgs& g, cudaStream_t s) {
  const bool swiglu = g.codes != nullptr;
  if (fp8_few_fits(g)) return launch_fp8_few(g, s);
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  const int KB = (g.K + 127) / 128;
  const dense::Choice c = dense::choose(g.M, g.N, KB, swiglu, true, di.sms);
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
