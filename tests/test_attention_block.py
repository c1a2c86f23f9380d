"""AttentionBlock and DecoderLayer: prompts in chunks and single tokens through a paged cache, as one would use them,
against a plain form in 64 bits and against the whole prompt at once; streams and graphs."""
import pytest
import torch

import mixture_experts_layer_gate_gb300 as moe
from tests import attention_reference as att
from tests import op_reference as ref
from tests.test_operators import dev, few_weights, gen, randn  # noqa: F401  (a fixture among them)

gpu = pytest.mark.gpu
H, HQ, HKV, D, PAGE = 512, 8, 2, 64, 16


def weights(g, dev, norms=True, bias=True):
    bf = lambda t: t.bfloat16()  # noqa: E731
    w = dict(wqkv=bf(randn(g, (HQ + 2 * HKV) * D, H) * H ** -0.5), wo=bf(randn(g, H, HQ * D) * (HQ * D) ** -0.5),
             norm_weight=bf(1 + 0.1 * randn(g, H)))
    if bias:
        w["bias"] = bf(0.3 * randn(g, (HQ + 2 * HKV) * D))
    if norms:
        w["q_norm"], w["k_norm"] = bf(1 + 0.1 * randn(g, D)), bf(1 + 0.1 * randn(g, D))
    return w


def make(w, dev, **kw):
    return moe.AttentionBlock(H, HQ, HKV, D, turns=moe.rope_table(kw.get("rot", D), device=dev), device=dev,
                              **{n: t.to(dev) for n, t in w.items()}, **kw)


def rounded(v):
    return v.float().bfloat16().double()


def plain(w, x, residual, positions, past_kv, e4m3=False, layout="half", rot=D):
    """One sequence's new tokens in 64 bits, with the block's roundings to bf16: out, residual + x, and its keys and
    values with those before them."""
    s = x.double() + (residual.double() if residual is not None else 0)
    y = rounded(s / torch.sqrt((s * s).mean(dim=1, keepdim=True) + 1e-6) * w["norm_weight"].double())
    qkv = y @ w["wqkv"].double().T
    if "bias" in w:
        qkv = qkv + w["bias"].double()
    q, k, v = rounded(qkv).split((HQ * D, HKV * D, HKV * D), dim=1)
    n, freq = x.shape[0], att.frequencies(rot)
    turn = lambda t, weight: att.norm_rotate(t.reshape(n, -1, D), weight, positions, freq, layout == "interleaved",  # noqa: E731
                                             1e-6, 1.0)[0]
    q, k, v = rounded(turn(q, w.get("q_norm"))), turn(k, w.get("k_norm")), v.reshape(n, HKV, D)
    if e4m3:
        def codes(t):
            scale = t.abs().amax(dim=2, keepdim=True) / 448
            return ref.e4m3_round(t / scale) * scale
        k, v = codes(k), codes(v)
    else:
        k = rounded(k)
    k, v = (torch.cat([a, c]) if a is not None else c for a, c in zip(past_kv, (k, v)))
    o = att.attend(q, k, v, k.shape[0] - n, D ** -0.5, 0.0)[0]
    return rounded(rounded(o.reshape(n, -1)) @ w["wo"].double().T), rounded(s), (k, v)


def near(got, want, roundings, what):
    """Each rounding to bf16 (2^-8 of a value at most, e4m3 2^-4) reaches out through maps that keep relative sizes; two
    results that round the same values differ by as much where a value lies next to a border."""
    got, want = got.cpu().double(), want.double()
    assert bool(torch.isfinite(got).all()), what
    off = float((got - want).norm() / want.norm())
    assert off <= roundings, (what, off, roundings)


class Pages:
    """Slots and page tables of growing sequences, pages handed out in a shuffled order."""

    def __init__(self, g, n, sequences):
        self.free = torch.randperm(n, generator=g).tolist()
        self.pages, self.lens = [[] for _ in range(sequences)], [0] * sequences

    def append(self, b, n):
        slots = []
        for j in range(self.lens[b], self.lens[b] + n):
            if j // PAGE == len(self.pages[b]):
                self.pages[b].append(self.free.pop())
            slots.append(self.pages[b][j // PAGE] * PAGE + j % PAGE)
        self.lens[b] += n
        return slots

    def table(self, dev, columns=12):
        t = torch.full((len(self.pages), columns), -1, dtype=torch.int32)
        for b, p in enumerate(self.pages):
            t[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        return t.to(dev)


@gpu
@pytest.mark.parametrize("cache_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout,rot,norms,bias", [("half", D, True, True), ("interleaved", 32, False, False)])
def test_chunks_and_single_tokens(dev, cache_dtype, layout, rot, norms, bias):
    """Steps of a server: a chunk beside single tokens, a drafted few, a sequence that sits a step out, a padded row."""
    g = gen(11)
    w = weights(g, dev, norms, bias)
    block = make(w, dev, layout=layout, rot=rot)
    cache = moe.KVCache(40, PAGE, HKV, D, dev, cache_dtype=cache_dtype)
    pages, past = Pages(g, 40, 3), [(None, None)] * 3
    bound = 6 * 2.0 ** -8 + (2 * 2.0 ** -4 * 0.6 if cache_dtype == "e4m3" else 0)  # (rms of e4m3's steps: 0.6 of half a one)
    for step, new in enumerate(([50, 1, 0], [30, 1, 7], [1, 1, 1], [3, 0, 1], [1, 90, 2])):
        T = sum(new) + 1
        x, residual = randn(g, T, H).bfloat16(), (2 * randn(g, T, H)).bfloat16()
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        positions = torch.tensor([p for b in range(3) for p in range(pages.lens[b], pages.lens[b] + new[b])] + [0],
                                 dtype=torch.int32)
        slots = torch.tensor([s for b in range(3) for s in pages.append(b, new[b])] + [-1], dtype=torch.int32)
        out, total = block(x.to(dev), residual.to(dev), positions.to(dev), torch.tensor(cu, dtype=torch.int32, device=dev),
                           max(new), cache, slots.to(dev), pages.table(dev),
                           torch.tensor(pages.lens, dtype=torch.int32, device=dev))
        assert block.device_error() == 0
        for b in range(3):
            rows = slice(cu[b], cu[b + 1])
            if not new[b]:
                continue
            want, s, past[b] = plain(w, x[rows], residual[rows], positions[rows], past[b], cache_dtype == "e4m3", layout, rot)
            assert torch.equal(total[rows].cpu().double(), s)
            # (the cache holds what the block computed, a border's width off the plain form's)
            near(out[rows], want, bound, f"step {step} sequence {b}")


@gpu
def test_whole_prompts(dev):
    g = gen(12)
    w = weights(g, dev)
    block = make(w, dev)
    lens = [33, 1, 120]
    T = sum(lens)
    x = randn(g, T, H).bfloat16()
    cu = torch.tensor([0, 33, 34, 154], dtype=torch.int32)
    positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens])
    out, total = block(x.to(dev), None, positions.to(dev), cu.to(dev), max(lens))
    assert block.device_error() == 0 and torch.equal(total.cpu(), x)
    for b in range(3):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        want, _, _ = plain(w, x[rows], None, positions[rows], (None, None))
        near(out[rows], want, 6 * 2.0 ** -8, f"prompt {b}")


@gpu
@pytest.mark.parametrize("new", [1, 5])
def test_captured_step_follows_its_inputs(dev, new):
    """A decode step captured once and replayed as the context grows gives what eager calls give."""
    g = gen(13)
    w = weights(g, dev)
    eager, captured = make(w, dev), make(w, dev)
    caches = [moe.KVCache(30, PAGE, HKV, D, dev) for _ in range(2)]
    pages = Pages(g, 30, 2)
    x = randn(g, 2 * 37, H).bfloat16().to(dev)
    pos = torch.arange(37, dtype=torch.int32).repeat(2).to(dev)
    slots = torch.tensor(pages.append(0, 37) + pages.append(1, 37), dtype=torch.int32, device=dev)
    cu = torch.tensor([0, 37, 74], dtype=torch.int32, device=dev)
    lens = torch.tensor(pages.lens, dtype=torch.int32, device=dev)
    for b, c in zip((eager, captured), caches):
        b(x, None, pos, cu, 37, c, slots, pages.table(dev), lens)
    s = dict(x=torch.zeros(2 * new, H, dtype=torch.bfloat16, device=dev), pos=torch.zeros(2 * new, dtype=torch.int32, device=dev),
             slots=torch.full((2 * new,), -1, dtype=torch.int32, device=dev), table=pages.table(dev),
             lens=torch.full((2,), 37 + new, dtype=torch.int32, device=dev))
    cu = torch.tensor([0, new, 2 * new], dtype=torch.int32, device=dev)
    graph = torch.cuda.CUDAGraph()
    call = lambda b, c: b(s["x"], s["x"], s["pos"], cu, new, c, s["slots"], s["table"], s["lens"])  # noqa: E731
    call(captured, caches[1])  # (its workspaces; stores nothing)
    with torch.cuda.graph(graph):
        out, total = call(captured, caches[1])
    for _ in range(4):
        s["x"].copy_(randn(g, 2 * new, H).bfloat16())
        s["pos"].copy_(torch.tensor([p for b in range(2) for p in range(pages.lens[b], pages.lens[b] + new)], dtype=torch.int32))
        s["slots"].copy_(torch.tensor(pages.append(0, new) + pages.append(1, new), dtype=torch.int32))
        s["table"].copy_(pages.table("cpu"))
        s["lens"].copy_(torch.tensor(pages.lens, dtype=torch.int32))
        graph.replay()
        want = call(eager, caches[0])
        assert torch.equal(out, want[0]) and torch.equal(total, want[1])
    assert torch.equal(caches[0].k[pages.pages[0][0]], caches[1].k[pages.pages[0][0]])


@gpu
def test_on_a_given_stream(dev):
    g = gen(14)
    block = make(weights(g, dev), dev)
    x = randn(g, 60, H).bfloat16().to(dev)
    cu, pos = torch.tensor([0, 60], dtype=torch.int32, device=dev), torch.arange(60, dtype=torch.int32, device=dev)
    want, _ = block(x, x, pos, cu, 60)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, total = block(x, x, pos, cu, 60, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want) and block.device_error() == 0


@gpu
def test_decoder_layer(dev):
    """Attention, then experts: a prompt in two chunks gives what the whole prompt gives."""
    g = gen(15)
    E, I, k = 8, 256, 2
    w13, w2 = few_weights(moe.problem(1, H, I, E, k), False, 15)[:2]
    router = (randn(g, E, H) * H ** -0.5).bfloat16().to(dev)
    experts = moe.Weights(w13.to(dev), w2.to(dev))
    layer = moe.DecoderLayer(make(weights(g, dev), dev),
                             moe.MoEBlock(H, I, E, k, experts, torch.ones(H, dtype=torch.bfloat16, device=dev), router,
                                          None, 128, dev))
    n = 70
    x = randn(g, n, H).bfloat16().to(dev)
    pos = torch.arange(n, dtype=torch.int32, device=dev)
    whole, total = layer(x, x, pos, torch.tensor([0, n], dtype=torch.int32, device=dev), n)
    cache, pages, parts = moe.KVCache(8, PAGE, HKV, D, dev), Pages(g, 8, 1), []
    for lo, hi in ((0, 45), (45, 69), (69, 70)):
        slots = torch.tensor(pages.append(0, hi - lo), dtype=torch.int32, device=dev)
        parts.append(layer(x[lo:hi], x[lo:hi], pos[lo:hi], torch.tensor([0, hi - lo], dtype=torch.int32, device=dev), hi - lo,
                           cache=cache, slots=slots, page_table=pages.table(dev),
                           kv_len=torch.tensor([hi], dtype=torch.int32, device=dev)))
    assert layer.device_error() == 0
    # (the residual stream: the router of a token whose scores tie within a rounding may choose another expert)
    near(torch.cat([t for _, t in parts]), total.cpu(), 4 * 2.0 ** -8, "residual")


def test_cache_refuses_other_types():
    with pytest.raises(ValueError):
        moe.KVCache(1, 16, 1, 64, "cpu", cache_dtype="f16")
    c = moe.KVCache(3, 16, 2, 64, "cpu", cache_dtype="e4m3")
    assert c.k.shape == (3, 16, 2, 64) and c.k_scale.shape == (3, 2, 16) and c.v.stride() == (2048, 64, 1024, 1)
