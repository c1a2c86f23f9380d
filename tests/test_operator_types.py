"""Types of the tensors that the operators around the layer are given: another type of the same size is refused."""
import pytest
import torch

import mixture_experts_layer_gate_gb300 as moe
from tests.test_operators import few_weights, product_inputs

gpu = pytest.mark.gpu
SAME_SIZE = {torch.bfloat16: (torch.float16, torch.int16), torch.float32: (torch.int32,),
             torch.uint8: (torch.int8, torch.bool, torch.float8_e5m2), torch.float16: (torch.bfloat16,)}


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    from mixture_experts_layer_gate_gb300 import build
    if not os.path.exists(moe.LIB_PATH) or not os.path.exists(build.OPS):
        build.build()
    return moe.load()


def calls(device):
    """(name, function, its tensors) of every operator, ready to run."""
    new = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device=device)  # noqa: E731
    u8, f32 = torch.uint8, torch.float32
    ws = torch.zeros(1 << 20, dtype=u8, device=device)
    x, logits = new(4, 256), new(4, 8, t=f32)
    p = moe.problem(4, 256, 128, 8, 2, scoring="sigmoid")
    w = moe.Weights(*[None if t is None else t.to(device) for t in few_weights(p, False, 1)])
    a, sa, b, sb = [t.to(device) for t in product_inputs(4, 256, 256, 1)]
    h = moe.norm_problem(4, 256, dtype="f16", weight_dtype="f32")
    return [
        ("norm", lambda **k: moe.add_rms_norm(moe.norm_problem(4, 256, quant="block"), **k),
         dict(x=x, weight=new(256), residual=new(4, 256), residual_out=new(4, 256), y=new(4, 256),
              codes=new(4, 256, t=u8), scales=new(4, 2, t=f32))),
        ("norm f16", lambda **k: moe.add_rms_norm(h, **k),
         dict(x=new(4, 256, t=torch.float16), weight=new(256, t=f32), y=new(4, 256, t=torch.float16))),
        ("router", lambda **k: moe.router_logits(moe.router_problem(4, 256, 8), ws=ws, **k),
         dict(x=x, w=new(8, 256), logits=logits)),
        ("gemm", lambda **k: moe.gemm_fp8_block(moe.fp8_gemm_problem(4, 256, 256), ws=ws, **k),
         dict(a=a, a_scale=sa, w=b, w_scale=sb, out=new(4, 256))),
        ("swiglu", lambda **k: moe.gemm_fp8_block_swiglu(moe.fp8_gemm_problem(4, 128, 256), ws=ws, **k),
         dict(a=a, a_scale=sa, w13=b, w13_scale=sb, codes=new(4, 128, t=u8), scales=new(4, 1, t=f32))),
        ("few", lambda **k: moe.forward_few(p, w, ws=ws, **k),
         dict(x=x, logits=logits, bias=new(8, t=f32), out=new(4, 256))),
    ]


def refused(device, message):
    for name, call, tensors in calls(device):
        for arg, t in tensors.items():
            for other in SAME_SIZE[t.dtype]:
                with pytest.raises(ValueError, match=f"^{arg}: .*{message(t.dtype)}"):
                    call(**dict(tensors, **{arg: t.view(other)}))


def test_tensors_that_are_not_on_a_gpu():
    for name, call, tensors in calls("cpu"):
        with pytest.raises(ValueError, match="on the current CUDA device"):
            call(**tensors)


@gpu
def test_another_type_of_the_same_size():
    names = {torch.bfloat16: "BFloat16", torch.float32: "Float", torch.float16: "Half", torch.uint8: "Byte or Float8_e4m3fn"}
    refused("cuda:0", names.__getitem__)
    for name, call, tensors in calls("cuda:0"):
        call(**tensors)
        call(**{k: t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t for k, t in tensors.items()})
    torch.cuda.synchronize()


@gpu
@pytest.mark.parametrize("which", ["x", "norm_weight", "router_weight"])
def test_block_refuses_half_precision(which):
    dev = torch.device("cuda:0")
    H, I, E = 256, 128, 8
    bf = lambda *s: torch.ones(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    t = dict(x=bf(4, H), norm_weight=bf(H), router_weight=bf(E, H))
    t[which] = t[which].half()
    b = moe.MoEBlock(H, I, E, 2, moe.Weights(bf(E, 2 * I, H), bf(E, H, I)), t["norm_weight"], t["router_weight"], None, 8, dev)
    with pytest.raises(ValueError):
        b(t["x"])
