"""AttentionBlock's memory between calls and across streams: its cache lives as long as a given stream's kernels need it."""
import pytest
import torch

import mixture_experts_layer_gate_gb300 as moe
from mixture_experts_layer_gate_gb300 import binding
from tests.test_attention_block import D, H, HKV, PAGE, make, weights
from tests.test_block_streams import FakeStreams
from tests.test_operators import gen, lib  # noqa: F401  (a fixture)


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
