"""MoEBlock and MoELayer on a stream that they are given and in captured graphs: what a call allocates belongs to the
stream of its kernels, and a workspace lives as long as a graph that uses it."""
import contextlib
import weakref

import pytest
import torch

import mixture_experts_layer_gate_gb300 as moe
from mixture_experts_layer_gate_gb300 import binding, block
from tests.test_operators import codes_of, few_weights, gen, randn

gpu = pytest.mark.gpu


class FakeStreams:
    """Stands in for PyTorch's streams, allocations and the kernels, on the CPU: notes on which stream each runs."""

    def __init__(self, monkeypatch, caller):
        self.current, self.log, self.recorded, self.capturing, self.passed = caller, [], [], False, []
        fake = self

        class Stream:
            def __init__(self, handle, device=None):
                self.cuda_stream = handle

        @contextlib.contextmanager
        def switch(s):
            before, fake.current = fake.current, s.cuda_stream
            yield
            fake.current = before

        empty, zeros = torch.empty, torch.zeros
        monkeypatch.setattr(torch, "empty", lambda *a, **k: (self.log.append(("empty", self.current)), empty(*a, **k))[1])
        monkeypatch.setattr(torch, "zeros", lambda *a, **k: (self.log.append(("zeros", self.current)), zeros(*a, **k))[1])
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(self.current))
        monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
        monkeypatch.setattr(torch.cuda, "stream", switch)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.capturing)
        monkeypatch.setattr(torch.Tensor, "record_stream",
                            lambda t, s: self.recorded.append((t.data_ptr(), s.cuda_stream)))
        monkeypatch.setattr(binding, "_stream", lambda s: self.current if s is None else int(s))
        at = {"add_rms_norm": 8, "router_logits": 5, "gemm_fp8_block": 7, "gemm_fp8_block_swiglu": 8, "forward_few": 7,
              "forward": 7}  # where each takes its stream
        for name, i in at.items():
            def op(*a, name=name, i=i, stream=None):
                given = a[i] if len(a) > i else stream
                self.log.append((name, self.current if given is None else int(given)))
                if name.startswith("forward"):
                    self.passed.append(a[6])  # its workspace
            monkeypatch.setattr(binding, name, op)


def cpu_block(max_tokens, shared=True):
    H, I, E = 256, 128, 8
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    by = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    sh = moe.SharedExpert(by(2 * I, H), torch.ones(2, 2), by(H, I), torch.ones(2, 1)) if shared else None
    return moe.MoEBlock(H, I, E, 2, moe.Weights(bf(E, 2 * I, H), bf(E, H, I)), bf(H), bf(E, H), sh, max_tokens, "cpu")


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    from mixture_experts_layer_gate_gb300 import build
    if not os.path.exists(moe.LIB_PATH) or not os.path.exists(build.OPS):
        build.build()
    return moe.load()


@pytest.mark.parametrize("T", [3, 20])
@pytest.mark.parametrize("max_tokens", [0, 64])
@pytest.mark.parametrize("stream", [None, 16, 48])
def test_block_allocates_on_the_stream_of_its_kernels(monkeypatch, T, max_tokens, stream):
    b = cpu_block(max_tokens)
    x, r = (torch.zeros(T, 256, dtype=torch.bfloat16) for _ in range(2))
    fake = FakeStreams(monkeypatch, 16)
    out, total = b(x, r, stream=stream)
    used = 16 if stream is None else stream
    assert {s for _, s in fake.log} == {used}, fake.log
    assert {"add_rms_norm", "router_logits", "forward_few" if T <= 8 else "forward", "gemm_fp8_block", "empty"} <= \
        {n for n, _ in fake.log}
    assert fake.current == 16
    if used != 16:  # what crosses streams is kept for both
        assert {(x.data_ptr(), 48), (r.data_ptr(), 48), (out.data_ptr(), 16), (total.data_ptr(), 16)} <= set(fake.recorded)


@pytest.mark.parametrize("given", [True, False])
def test_layer_allocates_on_the_stream_of_its_kernels(monkeypatch, given):
    H, I, E = 256, 128, 8
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    layer = moe.MoELayer(H, I, E, 2, moe.Weights(bf(E, 2 * I, H), bf(E, H, I)), 1, "cpu")
    fake = FakeStreams(monkeypatch, 16)
    x, logits = bf(40, H), torch.empty(40, E)
    fake.log.clear()
    out = bf(40, H) if given else None
    fake.log.clear()
    got = layer(x, logits, None, out, stream=48)
    assert fake.log and {s for _, s in fake.log} == {48}, fake.log
    assert got.shape == (40, H) and (out is None or got is out)


@pytest.mark.parametrize("T", [3, 20])
def test_workspaces_live_as_long_as_the_graphs_that_use_them(monkeypatch, T):
    """Capture a small batch, then call a larger one: the graph's workspace stays.  Captured while too small: the zero
    fill belongs to the graph, so a later call does not take that workspace for a zeroed one."""
    bf = lambda n: torch.zeros(n, 256, dtype=torch.bfloat16)  # noqa: E731
    small = 1 if T <= 8 else 9
    b = cpu_block(small, shared=False)
    fake = FakeStreams(monkeypatch, 16)
    fake.capturing = True
    b(bf(small))
    fake.capturing = False
    graphs = weakref.ref(fake.passed.pop())
    b(bf(T))                                   # grows
    assert graphs() is not None and fake.passed.pop() is not graphs()
    fake.capturing = True
    b(bf(T + 5 if T <= 8 else 2 * T))          # too small again, within a capture
    fake.capturing = False
    graphs = weakref.ref(fake.passed.pop())
    b(bf(T + 5 if T <= 8 else 2 * T))
    assert graphs() is not None and fake.passed.pop() is not graphs()
    before = len(b.kept) + len(b.layer.kept)
    for n in range(2 * T + 1, 2 * T + 4):      # without a capture outgrown ones go
        b(bf(n))
    assert len(b.kept) + len(b.layer.kept) == before


@gpu
@pytest.mark.parametrize("T", [3, 20])
def test_block_on_a_given_stream_while_the_current_one_allocates_and_writes(T):
    dev = torch.device("cuda:0")
    H, I, E, k = 2048, 512, 16, 4
    g = gen(T)
    rand = lambda *s: torch.rand(s, generator=g)  # noqa: E731
    p = moe.problem(T, H, I, E, k, wdtype="int8")
    wd = moe.Weights(*[None if t is None else t.to(dev) for t in few_weights(p, False, 7)])
    sh = (codes_of(g, 2 * I, H), rand(2 * I // 128, H // 128) * 4e-4, codes_of(g, H, I), rand(H // 128, I // 128) * 4e-4)
    b = moe.MoEBlock(H, I, E, k, wd, torch.ones(H, dtype=torch.bfloat16, device=dev),
                     (0.05 * randn(g, E, H)).to(torch.bfloat16).to(dev), moe.SharedExpert(*[t.to(dev) for t in sh]), 64, dev,
                     wdtype="int8")
    xs = [randn(gen(i), T, H).to(torch.bfloat16).to(dev) for i in range(6)]
    want = [tuple(t.clone() for t in b(x, x)) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    noise = []
    big = torch.randn(4096, 4096, device=dev)
    got = []
    for x in xs:
        big = (big @ big) * 1e-4  # the current stream is busy, and writes to whatever the allocator hands out
        got.append(b(x, x, stream=side.cuda_stream))
        for n in (T * H * 2, T * H, T * I, T * E * 4, T * H // 32, T * I // 32):
            noise.append(torch.full((n,), 0x7F, dtype=torch.uint8, device=dev))
            noise.pop()
    torch.cuda.synchronize()
    assert b.device_error() == 0
    for (out, total), (o, t) in zip(got, want):
        assert torch.equal(out, o) and torch.equal(total, t)


@gpu
@pytest.mark.parametrize("small,large", [(1, 8), (9, 300)])
def test_a_graph_replays_after_the_workspace_has_grown(small, large):
    dev = torch.device("cuda:0")
    H, I, E, k = 512, 256, 16, 4
    p = moe.problem(large, H, I, E, k, wdtype="int8")
    wd = moe.Weights(*[None if t is None else t.to(dev) for t in few_weights(p, False, 7)])
    nw, rw = torch.ones(H, dtype=torch.bfloat16, device=dev), (0.05 * randn(gen(1), E, H)).to(torch.bfloat16).to(dev)
    b, other = (moe.MoEBlock(H, I, E, k, wd, nw, rw, None, n, dev, wdtype="int8") for n in (0, large))
    x, y = (randn(gen(n), n, H).to(torch.bfloat16).to(dev) for n in (small, large))
    graphs = []
    other(x)  # the kernels' first launches, outside of a capture
    torch.cuda.synchronize()
    for eager in (False, True):  # the first capture grows the workspace itself, the second uses the eager one
        if eager:
            want, _ = b(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, b(x)[0]))
    large_want = b(y)[0].clone()
    junk = [torch.full((1 << 16,), 0x7F, dtype=torch.uint8, device=dev) for _ in range(64)]
    torch.cuda.synchronize()
    for graph, out in graphs:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all(bool((j == 0x7F).all()) for j in junk)
    assert torch.equal(b(y)[0], large_want) and b.device_error() == 0
