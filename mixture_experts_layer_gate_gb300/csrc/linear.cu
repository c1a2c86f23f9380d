// 16-bit product with bias, activation and residual in its epilogue (moe_linear):
// out = act(x w^T + bias) + residual, on the dense kernel with 16-bit operands.
// The sums are in registers when the tile ends, so bias and activation are applied
// there, and the residual's boxes are fetched by TMA before that.  An accumulator takes
// 2048 of K and is joined in float while the next one fills: the tensor core cuts off what
// its own sum does not hold, so that sums of one sign are 2.4e-6 off after 2048, 7.9e-6
// after 4096, 2.5e-5 after 8192 and 6.5e-5 after 16384 (f32 output; the times are the same).
// In a graph, M = N = K = 4096 78 us = 1.76 PFLOP/s, 91% of cuBLAS's rate
// alone, with a residual 83; N = 6144 114 us.  CTA pairs: single CTAs of 128 by 256
// took 91 us, bound by their reads from L2.  Up to 8 rows go through a kernel that
// streams the weights (linear_few.cu).
#include "dense.cuh"

namespace moe {

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  if (a.M <= kLinearFewRows) return launch_linear_few(a, s);
  dense::EpilogueParams p = {};
  p.out = a.out;
  p.old = a.residual;
  p.bias = a.bias;
  p.err = a.err;
  p.out_stride = a.out_stride;
  p.old_stride = a.residual_stride;
  p.M = a.M;
  p.N = a.N;
  p.KB = (a.K + 63) / 64;
  p.group = std::min(p.KB, kLinearRun / 64);
  p.fmt = a.f16 ? 0 : 1;
  p.out_dtype = a.out_dtype;
  p.accumulate = a.residual != nullptr;
  constexpr float kTwice = 1.5957691216057308f;  // 2 sqrt(2 / pi)
  p.act[0] = a.act == 4 ? 0.f : a.act == 0 ? -INFINITY : a.act == 1 ? 1.f : kTwice;
  p.act[1] = a.act == 3 ? 0.044715f * kTwice : 0.f;
  p.vec_bias = reinterpret_cast<uintptr_t>(a.bias) % 8 == 0;
  const int64_t osz = a.out_dtype == 2 ? 4 : 2;
  auto wide = [&](const void* q, int64_t stride) {
    return reinterpret_cast<uintptr_t>(q) % 16 == 0 && stride * osz % 16 == 0;
  };
  p.vec = wide(a.out, a.out_stride) && (a.residual == nullptr || wide(a.residual, a.residual_stride));
  const dense::Choice c = dense::choose(a.M, a.N, p.KB, false, false, di.sms, true);
  p.P = c.P;
  auto launch = [&](auto epi) {
    return dense::plan_and_launch<dense::kHalf, decltype(epi)::value>(p, c.bn, c.pair, false, a.x, a.x_stride, a.w,
                                                                      a.w_stride, a.N, a.K, di.sms, s);
  };
  if (a.act == 0 || a.act == 4) return launch(std::integral_constant<int, 1>());
  if (a.act == 2) return launch(std::integral_constant<int, 3>());
  return launch(std::integral_constant<int, 2>());
}

}  // namespace moe
