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
  const int mt = (a.T + 127) / 128;
  int bn = 32;
  while (bn < 256 && static_cast<long long>(mt) * ((a.E + bn - 1) / bn) * 8 > di.sms) bn *= 2;
  const long long tiles = static_cast<long long>(mt) * ((a.E + bn - 1) / bn);
  p.P = 8;
  while (p.P > 1 && (tiles * p.P > di.sms || p.P > p.KB)) p.P /= 2;
  return dense::plan_and_launch<dense::kHalf>(p, bn, false, false, a.x, a.x_stride, a.w, a.w_stride, a.E, a.H, di.sms,
                                              s);
}

}  // namespace moe
