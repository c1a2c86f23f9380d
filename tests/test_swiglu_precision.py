"""SwiGLU of a few rows to a float's last bits, also where the exponential is far from 1."""
import pytest
import torch

import mixture_experts_layer_gate_gb300 as moe


@pytest.mark.gpu
@pytest.mark.parametrize("gate", [-80.0, -60.0, -20.0, -1.0, 0.5, 10.0, 60.0])
@pytest.mark.parametrize("M", [1, 8])
def test_scales_of_far_gates(gate, M):
    dev = torch.device("cuda:0")
    N, K, up = 128, 16, 3.0
    one = lambda *s, v=0x38: torch.full(s, v, dtype=torch.uint8, device=dev)  # noqa: E731
    w = torch.cat([one(N, K, v=0x38 if gate > 0 else 0xB8), one(N, K)])
    w_scale = torch.tensor([[abs(gate) / K], [up / K]], device=dev)  # both products are exact
    ws = moe.alloc_op_workspace(dev)
    codes, scales = torch.zeros(M, N, dtype=torch.uint8, device=dev), torch.zeros(M, 1, device=dev)
    moe.gemm_fp8_block_swiglu(moe.fp8_gemm_problem(M, N, K), one(M, K), torch.ones(M, 1, device=dev), w, w_scale, codes,
                              scales, ws)
    assert moe.get_device_error(ws) == 0
    g = float(torch.tensor(abs(gate) / K)) * K * (1 if gate > 0 else -1)
    u = float(torch.tensor(up / K)) * K
    want = abs(g / (1.0 + float(torch.exp(torch.tensor(-g, dtype=torch.float64)))) * u) / 448.0
    # expf: 2 units in the last place (4 halves); its sum with 1, the quotient, the product and the scale one half each
    assert bool(((scales.double().cpu() - want).abs() <= 8 * 2.0 ** -24 * want).all())
    assert bool((codes == (0x7E if g > 0 else 0xFE)).all())
