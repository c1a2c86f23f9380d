"""AttentionBlock's memory between calls and across streams: its cache lives as long as a given stream's kernels need it,
errors of a workspace that was outgrown are not lost, and one that an aborted call left is made usable again."""
import pytest
import torch

import mixture_experts_layer_gate_gb300 as moe
from mixture_experts_layer_gate_gb300 import binding
from tests.test_attention_block import D, H, HKV, HQ, PAGE, Pages, make, weights
from tests.test_block_streams import FakeStreams, cpu_block
from tests.test_operators import dev, gen, lib, randn  # noqa: F401  (fixtures among them)

gpu = pytest.mark.gpu
BAD_INDEX, TIMEOUT = 5, 6


def cpu_attention(monkeypatch, current=16):
    block = make(weights(gen(1), "cpu"), "cpu")
    fake = FakeStreams(monkeypatch, current)
    for name in ("linear", "qk_norm_rope", "paged_attention", "prompt_attention"):
        def op(*a, name=name, **kw):
            fake.log.append((name, fake.current))
            if name.endswith("attention"):
                fake.passed.append(next(t for t in a if isinstance(t, torch.Tensor) and t.dtype == torch.uint8
                                        and t.dim() == 1 and t.numel() > 4096))
        monkeypatch.setattr(binding, name, op)

    def error(ws, stream=None):  # a workspace's first word, cleared
        head = ws[:8].view(torch.int32)
        e = int(head[0])
        head.zero_()
        return e

    monkeypatch.setattr(binding, "get_device_error", error)
    return block, fake


def step(block, T, max_q, cache, stream=None):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    return block(x, x, i32(T), torch.tensor([0, T], dtype=torch.int32), max_q, cache, i32(T), i32(1, 4), i32(1), stream=stream)


@pytest.mark.parametrize("cache_dtype", ["bf16", "e4m3"])
def test_cache_is_kept_for_the_given_stream(lib, monkeypatch, cache_dtype):
    cache = moe.KVCache(4, PAGE, HKV, D, "cpu", cache_dtype=cache_dtype)
    block, fake = cpu_attention(monkeypatch)
    step(block, 3, 3, cache, stream=48)
    assert {s for n, s in fake.log if n != "zeros"} == {48}  # (the inputs' zeros are the caller's)
    held = [t for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]
    assert {(t.data_ptr(), 48) for t in held} <= set(fake.recorded)
    fake.recorded.clear()
    step(block, 3, 3, cache, stream=16)  # the current one
    step(block, 3, 3, cache)
    assert not fake.recorded


def test_cache_is_kept_by_a_decoder_layer(lib, monkeypatch):
    cache = moe.KVCache(4, PAGE, HKV, D, "cpu")
    block, fake = cpu_attention(monkeypatch)
    layer = moe.DecoderLayer(block, lambda x, residual, stream=None: (x, residual))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    x = torch.zeros(3, H, dtype=torch.bfloat16)
    layer(x, x, i32(3), torch.tensor([0, 3], dtype=torch.int32), 3, stream=48, cache=cache, slots=i32(3),
          page_table=i32(1, 4), kv_len=i32(1))
    assert {(cache.k.data_ptr(), 48), (cache.v.data_ptr(), 48)} <= set(fake.recorded)


def test_errors_of_an_outgrown_workspace_are_found(lib, monkeypatch):
    cache = moe.KVCache(4, PAGE, HKV, D, "cpu")
    block, fake = cpu_attention(monkeypatch)
    step(block, 1, 1, cache)
    fake.passed[-1][:8].view(torch.int32)[0] = BAD_INDEX
    step(block, 90, 90, cache)
    assert fake.passed[0] is not fake.passed[1]
    assert block.device_error() == BAD_INDEX and block.device_error() == 0


def test_errors_of_an_outgrown_expert_workspace_are_found(lib, monkeypatch):
    """The same of MoEBlock, few tokens and many; of several outgrown ones the first error is the one that counts."""
    for small, large in ((1, 3), (9, 40)):
        with monkeypatch.context() as m:
            block = cpu_block(small, shared=False)
            _, fake = cpu_attention(m)
            bf = lambda n: torch.zeros(n, 256, dtype=torch.bfloat16)  # noqa: E731
            for i, n in enumerate((small, large, large + 2)):
                block(bf(n))
                fake.passed[-1][:8].view(torch.int32)[0] = (BAD_INDEX, TIMEOUT, 0)[i]
            assert block.device_error() == BAD_INDEX and block.device_error() == 0, small


@pytest.mark.parametrize("captured", [False, True])
def test_a_workspace_is_zeroed_after_an_error(lib, monkeypatch, captured):
    cache = moe.KVCache(4, PAGE, HKV, D, "cpu")
    block, fake = cpu_attention(monkeypatch)
    fake.capturing = captured
    step(block, 1, 1, cache)
    fake.capturing = False
    ws = fake.passed[-1]
    for error in (TIMEOUT, BAD_INDEX):  # (a timeout after another error is not recorded)
        ws.fill_(1)
        ws[:8].view(torch.int32)[0] = error
        assert block.device_error() == error and not bool(ws.any())


@gpu
def test_errors_of_an_outgrown_workspace_on_the_device(dev):
    g = gen(21)
    block = make(weights(g, dev), dev)
    cache, pages = moe.KVCache(8, PAGE, HKV, D, dev), Pages(g, 8, 1)
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device=dev)  # noqa: E731
    x = randn(g, 40, H).bfloat16().to(dev)
    slots = pages.append(0, 41)
    block(x[:1], None, i32([0]), i32([0, 1]), 1, cache, i32(slots[:1]), i32([[-7] * 12]), i32([1]))
    block(x, None, i32(list(range(1, 41))), i32([0, 40]), 40, cache, i32(slots[1:]), pages.table(dev), i32([41]))
    assert block.device_error() == BAD_INDEX and block.device_error() == 0


@gpu
def test_results_after_a_timeout_was_reported(dev):
    """The code and counters that an aborted call leaves, written by the host: once reported, calls are right again."""
    g = gen(22)
    w = weights(g, dev)
    blocks = [make(w, dev) for _ in range(2)]
    n = 3000
    cache, pages = moe.KVCache(200, PAGE, HKV, D, dev), Pages(g, 200, 1)
    slots = pages.append(0, n)
    for t in (cache.k, cache.v):
        t.copy_(randn(g, 200, PAGE, HKV, D))
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device=dev)  # noqa: E731
    x = randn(g, 1, H).bfloat16().to(dev)
    call = lambda b: b(x, None, i32([n - 1]), i32([0, 1]), 1, cache, i32(slots[-1:]), pages.table(dev, 200), i32([n]))  # noqa: E731
    want = call(blocks[0])[0]
    call(blocks[1])
    ws = blocks[1].attention_ws
    ws[256:256 + 2048].view(torch.int32).fill_(77)
    ws[:4].view(torch.int32).fill_(TIMEOUT)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert blocks[1].device_error(side.cuda_stream) == TIMEOUT
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(call(blocks[1])[0], want) and blocks[1].device_error() == 0
