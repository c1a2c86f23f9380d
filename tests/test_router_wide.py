"""Router scores of large batches against many experts with short rows: tiles of 256 columns with 16-bit operands."""
import subprocess

import pytest
import torch

import mixture_experts_layer_gate_gb300 as moe
from mixture_experts_layer_gate_gb300 import build
from tests import op_reference as ref
from tests.test_operators import gen, randn

# T, H, E: whole tiles and cut ones, E that takes 16-byte stores and E that does not, several tiles a CTA
SIZES = [(4096, 256, 1024), (4864, 128, 1024), (4096, 256, 1000), (4100, 72, 1021), (9727, 136, 769)]
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "dense.cuh"
int main(int n, char** v) {
  for (int i = 1; i + 2 < n; i += 3)
    std::printf("%d\n", moe::dense::choose(std::atoi(v[i]), std::atoi(v[i + 2]), (std::atoi(v[i + 1]) + 63) / 64, false,
                                           false, 152).bn);
}
"""


def test_these_sizes_take_the_widest_tiles(tmp_path):
    (tmp_path / "choose.cu").write_text(PROGRAM)
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", build.CSRC, "-I",
                    build.ROOT + "/include", str(tmp_path / "choose.cu"), "-o", str(tmp_path / "choose"), "-cudart",
                    "static"], check=True, capture_output=True)
    args = [str(v) for size in SIZES for v in size]
    out = subprocess.run([str(tmp_path / "choose"), *args], check=True, capture_output=True, text=True).stdout
    assert out.split() == ["256"] * len(SIZES)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,E", SIZES)
@pytest.mark.parametrize("dtype,off", [(torch.bfloat16, 0), (torch.float16, 1)])
def test_router_of_the_widest_tiles(T, H, E, dtype, off):
    dev = torch.device("cuda:0")
    g = gen(T + E)
    x, w = randn(g, T, H).to(dtype), (0.1 * randn(g, E, H)).to(dtype)
    whole = torch.full((off + T * E + 1,), 7.0, device=dev)
    logits = whole[off:off + T * E].view(T, E)  # off 1: not on a 16-byte boundary
    ws = moe.alloc_op_workspace(dev)
    r = moe.router_problem(T, H, E, dtype="bf16" if dtype == torch.bfloat16 else "f16")
    moe.router_logits(r, x.to(dev), w.to(dev), logits, ws)
    assert moe.get_device_error(ws) == 0
    want, tol = ref.router(x, w)
    ref.check(logits, want, tol, "logits")
    assert bool((whole[:off] == 7.0).all()) and float(whole[-1]) == 7.0
