// Router scores (moe_router_logits): logits[t, e] = sum_h x[t, h] w[e, h], in
// float, on the dense kernel with 16-bit operands.
#include "dense.cuh"

namespace moe {

cudaError_t launch_router(const RouterArgs& a, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  dense::Params p = {};
  p.out = a.logits;
  p.err = a.err;
  p.out_stride = a.E;
  p.M = a.T;
  p.N = a.E;
  p.KB = (a.H + 63) / 64;
  p.group = 16;
  p.out_dtype = 2;
  p.fmt = a.dtype == 0 ? 1 : 0;
  p.vec = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.E % 4 == 0;
  const dense::Choice c = dense::choose(a.T, a.E, p.KB, false, false, di.sms);
  p.P = c.P;
  return dense::plan_and_launch<dense::kHalf>(p, c.bn, c.pair, false, a.x, a.x_stride, a.w, a.w_stride, a.E, a.H, di.sms,
                                              s);
}

}  // namespace moe
