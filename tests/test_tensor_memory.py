"""Tensor memory is allocated without a time limit, so no two CTAs that take some may share an SM: of two clusters on two
streams each could hold columns that the other waits for.  Shared memory sees to that: each asks for over half of it."""
import random
import subprocess

import pytest
import torch

import mixture_experts_layer_gate_gb300 as moe
from mixture_experts_layer_gate_gb300 import build
from tests.test_operators import gen, product_inputs, randn

SM_BYTES, RESERVED = 228 * 1024, 1024  # of an SM; of each CTA besides what it asks for
PROGRAM = r"""
#include <cstdio>
#include "dense.cuh"
using namespace moe::dense;
template <int KIND, bool SWIGLU>
void all() {
  for (int bn = 32; bn <= 256; bn *= 2)
    for (int pair = 0; pair < 2; ++pair)
      for (int P = 1; P <= 8; P *= 2)
        for (int M = 8; M <= 128; M += 40) {
          if ((SWIGLU || pair) && bn != 256) continue;
          if (pair && P > 1) continue;
          Params p = {};  // the shortest ring
          p.stages = 1, p.M = M, p.P = P, p.arows = pair ? 128 : M, p.boxes = 2;
          std::printf("%d %d %d %d %d %d %zu\n", KIND, SWIGLU, bn, pair, P, M, smem_bytes<KIND, SWIGLU>(p, bn, pair));
        }
}
int main() {
  all<kE4M3, false>();
  all<kE4M3, true>();
  all<kHalf, false>();
}
"""


def shares_an_sm(a, b):
    return a + RESERVED + b + RESERVED <= SM_BYTES


@pytest.fixture(scope="module")
def dense(tmp_path_factory):
    """Shared memory that each variant of the dense kernel asks for with the shortest ring."""
    d = tmp_path_factory.mktemp("dense")
    (d / "plan.cu").write_text(PROGRAM)
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", build.CSRC, "-I",
                    build.ROOT + "/include", str(d / "plan.cu"), "-o", str(d / "plan"), "-cudart", "static"],
                   check=True, capture_output=True)
    out = subprocess.run([str(d / "plan")], check=True, capture_output=True, text=True).stdout
    rows = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert len(rows) > 100
    return rows


def test_no_two_ctas_of_the_dense_kernel_share_an_sm(dense):
    least = min(dense, key=lambda r: r[-1])
    assert not shares_an_sm(least[-1], least[-1]), least


def test_no_cta_of_a_grouped_product_shares_an_sm(dense):
    rng = random.Random(5)
    least = min(r[-1] for r in dense)
    worst = 1 << 30
    for _ in range(3000):
        E = rng.choice([1, 2, 8, 16, 64, 128, 256, 1024])
        p = moe.problem(rng.choice([1, 2, 8, 33, 100, 256, 1000, 4096, 20000]), rng.randint(1, 64) * 128,
                        rng.randint(1, 64) * 128, E, rng.randint(1, min(E, 8)),
                        wdtype=rng.choice(["bf16", "fp8", "int4", "int8", "int4_paired"]))
        plan = moe.get_plan(p, 152)
        worst = min(worst, plan.smem_up, plan.smem_down)
    assert not shares_an_sm(worst, worst) and not shares_an_sm(worst, least)
    with moe.tuning(stages=2):
        plan = moe.get_plan(moe.problem(1, 1024, 1024, 8, 2), 152)
        assert not shares_an_sm(plan.smem_up, least) and not shares_an_sm(plan.smem_down, least)


@pytest.mark.gpu
def test_products_of_two_streams_at_once():
    """Split products of different widths from two streams, each with its workspace."""
    dev = torch.device("cuda:0")
    x, w = randn(gen(1), 64, 4096).to(torch.bfloat16).to(dev), randn(gen(2), 60, 4096).to(torch.bfloat16).to(dev)
    a, sa, b, sb = [t.to(dev) for t in product_inputs(64, 1024, 1024, 3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [moe.alloc_op_workspace(dev) for _ in range(2)]
    logits, want = torch.empty(64, 60, device=dev), torch.empty(64, 60, device=dev)
    codes = [torch.empty(64, 512, dtype=torch.uint8, device=dev) for _ in range(2)]
    scales = [torch.empty(64, 4, device=dev) for _ in range(2)]
    r, g = moe.router_problem(64, 4096, 60), moe.fp8_gemm_problem(64, 512, 1024)
    moe.router_logits(r, x, w, want, ws[0])
    moe.gemm_fp8_block_swiglu(g, a, sa, b, sb, codes[0], scales[0], ws[0])
    torch.cuda.synchronize()
    for _ in range(100):
        moe.router_logits(r, x, w, logits, ws[0], streams[0].cuda_stream)
        moe.gemm_fp8_block_swiglu(g, a, sa, b, sb, codes[1], scales[1], ws[1], streams[1].cuda_stream)
    torch.cuda.synchronize()
    assert moe.get_device_error(ws[0]) == 0 and moe.get_device_error(ws[1]) == 0
    assert torch.equal(logits, want) and torch.equal(codes[0], codes[1]) and torch.equal(scales[0], scales[1])
