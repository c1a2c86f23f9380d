"""moe_paged_attention and moe_prompt_attention: refusals (no GPU), and the operators against their plain 64-bit form at
the lengths, masks and values where they can go wrong."""
import ctypes
import math

import pytest
import torch

import mixture_experts_layer_gate_gb300 as moe
from tests import attention_reference as att
from tests import op_reference as ref
from tests.test_operators import dev, gen, lib, randn, wide  # noqa: F401  (fixtures among them)
from tests.test_rope import kv

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
INVALID, UNSUPPORTED, WORKSPACE, BAD_INDEX = 1, 2, 3, 5
P = 4096  # an address that is never dereferenced: the checks come before any launch


# ------------------------------------------------------------------ refusals (CPU)


def paged(T=3, B=2, Hq=8, Hkv=4, D=64, max_q=2, page_size=16, num_pages=7, max_pages=5, **kw):
    return moe.attention_problem(T, B, Hq, Hkv, D, max_q, page_size=page_size, num_pages=num_pages, max_pages=max_pages,
                                 **kw)


def call(lib, p, q=P, qs=None, cache=None, pt=P, pts=5, cu=P, kl=P, out=P, os=None, lse=None, ws=P, ws_bytes=1 << 40):
    nq = p.Hq * p.D if p is not None else 0
    own = lambda s, n: n if s is None else s  # noqa: E731
    return lib.moe_paged_attention(ctypes.byref(p) if p is not None else None, q, own(qs, nq),
                                   ctypes.byref(cache if cache is not None else kv()), pt, pts, cu, kl, out, own(os, nq),
                                   lse, ws, ws_bytes, None)


def call_prompt(lib, p, q=P, qs=None, k=P, ks=None, v=P, vs=None, cu=P, out=P, os=None, lse=None, ws=P, ws_bytes=1 << 40):
    nq, nk = p.Hq * p.D, p.Hkv * p.D
    own = lambda s, n: n if s is None else s  # noqa: E731
    return lib.moe_prompt_attention(ctypes.byref(p), q, own(qs, nq), k, own(ks, nk), v, own(vs, nk), cu, out, own(os, nq),
                                    lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [dict(q=None), dict(pt=None), dict(cu=None), dict(kl=None), dict(out=None), dict(q=P + 8),
                                dict(out=P + 2), dict(pt=P + 2), dict(cu=P + 1), dict(kl=P + 3), dict(lse=P + 2),
                                dict(qs=504), dict(qs=516), dict(os=511), dict(pts=4), dict(cache=kv(k=None)),
                                dict(cache=kv(v=P + 8)), dict(cache=kv(ks=P, vs=P)), dict(cache=kv(token=60)),
                                dict(cache=kv(head=68)), dict(cache=kv(page=0))])
def test_refuses_arguments(lib, kw):
    assert call(lib, paged(), **kw) == INVALID


def test_refuses_problems(lib):
    assert ctypes.sizeof(moe.AttentionProblem) == 48
    assert call(lib, None) == INVALID
    for bad in (dict(T=-1), dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=6), dict(D=0), dict(D=60), dict(max_q=0),
                dict(dtype=2), dict(cache_dtype=2), dict(page_size=8), dict(page_size=24), dict(num_pages=0),
                dict(max_pages=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=3e38)):
        p = paged()
        for n, v in bad.items():
            setattr(p, n, v)
        assert call(lib, p) == INVALID, bad
    for bad in (dict(D=136), dict(Hq=8192), dict(max_pages=1 << 27), dict(T=(1 << 28) + 1)):
        p = paged()
        for n, v in bad.items():
            setattr(p, n, v)
        big = kv(page=1 << 20, token=1 << 14, head=256)
        assert call(lib, p, cache=big, pts=1 << 28) == UNSUPPORTED, bad
    p = paged()
    need = moe.attention_workspace_size(p)
    assert call(lib, p, ws=None) == WORKSPACE and call(lib, p, ws_bytes=need - 1) == WORKSPACE
    assert call(lib, p, ws=P + 64) == WORKSPACE
    assert call(lib, paged(T=0)) == 0 and call(lib, paged(B=0)) == 0
    # 8-bit: both scales, whole 16-byte rows
    assert call(lib, paged(cache_dtype="e4m3")) == INVALID
    assert call(lib, paged(D=72, cache_dtype="e4m3"), cache=kv(ks=P, vs=P, page=1 << 12, token=288, head=72)) == INVALID
    # a prompt has no cache
    p = moe.attention_problem(3, 2, 8, 4, 64, 2)
    assert call(lib, p) == INVALID
    for kw in (dict(q=None), dict(k=None), dict(v=P + 2), dict(ks=200), dict(vs=260), dict(cu=None), dict(out=P + 8)):
        assert call_prompt(lib, p, **kw) == INVALID, kw
    assert call_prompt(lib, paged()) == INVALID
    assert call_prompt(lib, moe.attention_problem(3, 2, 8, 4, 64, 2, cache_dtype="e4m3")) == INVALID
    assert call_prompt(lib, moe.attention_problem(0, 2, 8, 4, 64, 2)) == 0
    bad = paged()
    bad.scale = 0.0
    assert moe.attention_workspace_size(bad) == 0
    with pytest.raises(moe.MoEError):
        moe.alloc_attention_workspace(bad, "cpu")


# ------------------------------------------------------------------ against the 64-bit form


def build(dev, new, kv_len, Hq, Hkv, D, dtype, cache, page, order, seed=0, spare=3, junk=math.nan, scale=None):
    """A call's inputs, with junk wherever nothing may be read, and float64 keys and values of each sequence."""
    g = gen(seed * 131 + sum(new) + sum(kv_len))
    dt, B, T = DT[dtype], len(new), sum(new) + spare
    q = randn(g, T, Hq * D).to(dt)
    need = [-(-n // page) for n in kv_len]
    pages, columns = sum(need) + 2, max(need + [1]) + 1
    at = torch.randperm(pages, generator=g).int()
    table = torch.full((B, columns), 2 ** 31 - 1, dtype=torch.int32)
    shape = (pages, page, Hkv, D)
    if cache == "e4m3":
        codes = [torch.randint(0, 256, shape, generator=g, dtype=torch.uint8) for _ in range(2)]
        for c in codes:
            c[(c & 127) == 127] = 5  # no NaN among what is read
            c[(c & 127) > 0x60] &= 0xBF  # (fewer of the largest, so that weights are spread)
        scales = [(torch.rand(pages, Hkv, page, generator=g) + 0.1) * f for f in (0.02, 0.3)]
        full = [ref.e4m3_values(c) * s.double().transpose(1, 2)[..., None] for c, s in zip(codes, scales)]
    else:
        codes = [randn(g, *shape).to(dt) for _ in range(2)]
        scales = [None, None]
        full = [c.double() for c in codes]
    used, first, keys = torch.zeros(pages, page, dtype=torch.bool), 0, []
    for b, n in enumerate(kv_len):
        mine = at[first:first + need[b]]
        table[b, :need[b]] = mine
        first += need[b]
        keys.append([f[mine.long()].reshape(-1, Hkv, D)[:n] for f in full])
        for j in range(n):
            used[mine[j // page], j % page] = True
    for c, s in zip(codes, scales):
        if cache == "e4m3":
            c[~used] = 0x7F
            s.transpose(1, 2)[~used] = junk
        else:
            c[~used] = junk
    place = lambda c: (c if order == "token" else c.transpose(1, 2).contiguous()).to(dev)  # noqa: E731
    caches = [place(c) if order == "token" else place(c).transpose(1, 2) for c in codes]
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32)
    problem = moe.attention_problem(T, B, Hq, Hkv, D, max(new + [1]), dtype=dtype, cache_dtype=cache, page_size=page,
                                    num_pages=pages, max_pages=columns, scale=scale)
    args = dict(q=wide(q, 8, dev), k_cache=caches[0], v_cache=caches[1], page_table=table.to(dev), cu_q=cu.to(dev),
                kv_len=torch.tensor(kv_len, dtype=torch.int32, device=dev),
                k_scale=None if scales[0] is None else scales[0].to(dev),
                v_scale=None if scales[1] is None else scales[1].to(dev))
    return problem, args, q, keys, cu, [None if s is None else float(s[torch.isfinite(s)].max()) for s in scales]


def run(problem, args, dev, ws=None, lse=True, fill=7.0):
    dt = args["q"].dtype
    out = wide(torch.full((problem.T, problem.Hq * problem.D), fill).to(dt), 8, dev, fill=fill)
    lse = torch.full((problem.T, problem.Hq), fill, device=dev) if lse else None
    ws = ws if ws is not None else moe.alloc_attention_workspace(problem, dev)
    moe.paged_attention(problem, args["q"], args["k_cache"], args["v_cache"], args["page_table"], args["cu_q"],
                        args["kv_len"], out, ws, k_scale=args["k_scale"], v_scale=args["v_scale"], lse=lse)
    return out, lse, ws


def compare(problem, out, lse, q, keys, cu, dtype, cache, unit):
    Hq, D, T = problem.Hq, problem.D, problem.T
    p_type = torch.float16 if cache == "e4m3" else DT[dtype]
    rel, tiny = ref.half_step(DT[dtype])
    for b, (k, v) in enumerate(keys):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        n, L = rows.stop - rows.start, k.shape[0]
        if n == 0:
            continue
        want, wl, dout, dl = att.attend(q[rows].double().view(n, Hq, D), k, v, L - n, problem.scale,
                                        ref.half_step(p_type)[0], unit if cache == "e4m3" else None)
        ref.check(out[rows].reshape(n, Hq, D), want, dout + (want.abs() + dout) * rel + tiny, f"out {b}")
        got = lse[rows].cpu().double()
        empty = torch.isinf(wl)
        assert bool((got[empty] == -math.inf).all())
        assert bool(((got - wl).abs() <= dl)[~empty].all()), (b, (got - wl).abs()[~empty].max(), dl[~empty].max())
    last = int(cu[-1])
    assert bool((out[last:] == 7.0).all()) and bool((lse[last:] == 7.0).all())
    base = torch.as_strided(out, (T, Hq * D + 16), (out.stride(0), 1), out.storage_offset() - 8)
    assert bool((base[:, :8] == 7.0).all()) and bool((base[:, Hq * D + 8:] == 7.0).all())


CASES = [  # new tokens, lengths, Hq, Hkv, D, dtype, cache, page, order
    ([1], [1], 8, 8, 128, "bf16", "bf16", 16, "token"),
    ([1, 1, 1], [500, 17, 128], 32, 8, 128, "bf16", "bf16", 16, "token"),
    ([1, 1, 1, 1], [1, 3000, 0, 129], 28, 4, 128, "bf16", "e4m3", 64, "head"),
    ([1] * 70, [1 + 37 * i % 400 for i in range(70)], 4, 1, 64, "f16", "f16", 32, "head"),
    ([2, 0, 5, 1, 3], [40, 9, 5, 700, 2], 8, 4, 128, "bf16", "bf16", 16, "head"),       # a row that sees nothing
    ([4, 2, 1], [1000, 1999, 300], 10, 2, 128, "f16", "e4m3", 32, "token"),
    ([3, 3], [66, 1], 5, 1, 72, "f16", "f16", 16, "token"),
    ([1, 1], [16000, 5], 16, 1, 128, "bf16", "bf16", 128, "head"),                       # one key head over all SMs
    ([1, 8], [200, 90], 2, 2, 8, "bf16", "bf16", 16, "token"),
    ([2, 2], [333, 20], 8, 1, 80, "bf16", "e4m3", 16, "token"),
    ([1, 1], [256, 1024], 64, 2, 96, "f16", "e4m3", 256, "head"),
    # more rows than one small tile: chunks of prompts
    ([17, 1, 40], [17, 77, 300], 8, 2, 128, "bf16", "bf16", 16, "token"),
    ([130], [130], 4, 4, 64, "f16", "f16", 32, "head"),
    ([100, 33, 0, 1], [700, 33, 50, 1200], 14, 2, 128, "bf16", "e4m3", 64, "head"),
    ([70, 5], [50, 900], 6, 2, 128, "f16", "f16", 16, "token"),                          # 20 rows that see nothing
    ([260], [400], 5, 1, 128, "bf16", "bf16", 128, "token"),
    ([65, 64, 63], [65, 192, 511], 8, 1, 48, "bf16", "bf16", 16, "head"),
    ([129, 2], [129, 258], 3, 1, 112, "f16", "e4m3", 16, "head"),
    # one item over many SMs: pieces joined in groups
    ([1], [30000], 4, 1, 64, "bf16", "bf16", 64, "head"),
    ([2, 1], [40000, 100], 8, 1, 64, "f16", "e4m3", 256, "head"),
    ([3], [30011], 16, 1, 64, "bf16", "e4m3", 64, "token"),
    ([7, 2], [29000, 5000], 13, 1, 128, "bf16", "bf16", 64, "head"),
    # the narrowest heads, and odd groups, in tiles of 128 rows
    ([40, 3], [40, 200], 2, 2, 8, "bf16", "bf16", 16, "token"),
    ([33], [150], 4, 2, 16, "f16", "e4m3", 32, "token"),
    ([9, 5], [300, 77], 71, 1, 64, "bf16", "bf16", 16, "head"),
    ([1, 3], [130, 60], 142, 2, 32, "f16", "e4m3", 16, "head"),
]


@gpu
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_matches_plain(dev, case):
    new, kv_len, Hq, Hkv, D, dtype, cache, page, order = case
    problem, args, q, keys, cu, unit = build(dev, *case)
    out, lse, ws = run(problem, args, dev)
    assert moe.get_device_error(ws) == 0
    compare(problem, out, lse, q, keys, cu, dtype, cache, unit[1])
    # again on the same workspace, without lse: the same bits
    again, _, _ = run(problem, args, dev, ws=ws, lse=False)
    assert torch.equal(out, again)


PROMPTS = [  # lengths, Hq, Hkv, D, dtype
    ([1], 4, 2, 128, "bf16"),
    ([3, 0, 2, 1], 8, 4, 64, "f16"),
    ([130, 1, 257], 6, 2, 72, "f16"),
    ([300], 8, 8, 128, "bf16"),
    ([40, 129, 128, 5], 7, 1, 128, "bf16"),
    ([513], 5, 1, 40, "f16"),
]


@gpu
@pytest.mark.parametrize("case", PROMPTS, ids=[str(i) for i in range(len(PROMPTS))])
def test_prompt_matches_plain(dev, case):
    new, Hq, Hkv, D, dtype = case
    g, dt, T = gen(sum(new)), DT[dtype], sum(new) + 4
    q, k, v = (randn(g, T, h * D).to(dt) for h in (Hq, Hkv, Hkv))
    k[sum(new):], v[sum(new):] = math.nan, math.nan
    qkv = torch.cat([q, k, v], dim=1).to(dev).split((Hq * D, Hkv * D, Hkv * D), dim=1)
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32)
    problem = moe.attention_problem(T, len(new), Hq, Hkv, D, max(new), dtype=dtype)
    out = wide(torch.full((T, Hq * D), 7.0).to(dt), 8, dev, fill=7.0)
    lse, ws = torch.full((T, Hq), 7.0, device=dev), moe.alloc_attention_workspace(problem, dev)
    moe.prompt_attention(problem, *qkv, cu.to(dev), out, ws, lse=lse)
    assert moe.get_device_error(ws) == 0
    keys = [[t[cu[b]:cu[b + 1]].double().view(-1, Hkv, D) for t in (k, v)] for b in range(len(new))]
    compare(problem, out, lse, q, keys, cu, dtype, dtype, None)


def big_scores(q, factor):
    q.mul_(factor)


@gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 3, 150])
def test_far_scores(dev, cache, new):
    """Scores of some hundreds on both sides of zero, growing along the keys: the maximum changes all the time."""
    L, D = 600, 128
    problem, args, q, keys, cu, unit = build(dev, [new], [L], 4, 2, D, "bf16", cache, 16, "token", spare=0)
    q.mul_(0)
    q.view(new, 4, D)[:, :, 0] = 8.0
    ramp = torch.linspace(-60, 60, L).bfloat16().double()
    if cache == "e4m3":
        ks = args["k_scale"]
        kc = args["k_cache"]
        kc.zero_()
        kc[:, :, :, 0] = 0x38  # 1.0
        scale = torch.zeros_like(ks)
        for j in range(L):
            scale[int(args["page_table"][0, j // 16]), :, j % 16] = float(ramp[j])
        args["k_scale"] = scale
    else:
        args["k_cache"].zero_()
        for j in range(L):
            args["k_cache"][int(args["page_table"][0, j // 16]), j % 16, :, 0] = float(ramp[j])
    keys[0][0] = torch.zeros(L, 2, D, dtype=torch.float64)
    keys[0][0][:, :, 0] = ramp[:, None].float().double()
    args["q"] = q.to(dev)
    problem.scale = 1.0
    out, lse, ws = run(problem, args, dev)
    compare(problem, out, lse, q, keys, cu, "bf16", cache, unit[1])


@gpu
@pytest.mark.parametrize("cache", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("new,L", [(1, 40), (4, 200), (5, 5), (100, 300), (200, 200)])
def test_what_is_not_seen_does_not_matter(dev, cache, new, L):
    """Keys and values that are NaN or infinite reach only the rows that see them."""
    dtype = "f16" if cache == "f16" else "bf16"
    D = 64 if cache == "f16" else 128
    problem, args, q, keys, cu, unit = build(dev, [new], [L], 4, 2, D, dtype, cache, 16, "head", spare=0)
    clean, clean_lse, _ = run(problem, args, dev)
    at = L - 1 - new // 2  # seen by the later half of the new tokens
    page, place = int(args["page_table"][0, at // 16]), at % 16
    first = new - 1 - new // 2  # the first new token that sees it
    for bad in (math.nan, math.inf, -math.inf):
        broken = {n: (t.clone() if isinstance(t, torch.Tensor) and n.endswith(("cache", "scale")) else t)
                  for n, t in args.items()}
        if cache == "e4m3":
            if math.isnan(bad):
                broken["v_cache"][page, place, 1, 5] = 0x7F
                broken["k_cache"][page, place, 0, 5] = 0xFF
            else:
                broken["v_scale"][page, 1, place] = bad
                broken["k_scale"][page, 0, place] = bad
        else:
            broken["v_cache"][page, place, 1, 5] = bad
            broken["k_cache"][page, place, 0, 5] = bad
        out, lse, _ = run(problem, broken, dev)
        if cache == "e4m3" and math.isinf(bad):
            # the broken scale is not what the others are relative to: weights under f16's normal range round elsewhere
            assert bool(((out[:first] - clean[:first]).abs() <= clean[:first].abs() * 2.0 ** -7 + 2.0 ** -10).all())
        else:
            assert torch.equal(out[:first], clean[:first])
        assert torch.equal(lse[:first], clean_lse[:first])
        o = out.reshape(new, 4, D)
        c = clean.reshape(new, 4, D)
        # heads 2 and 3 read value head 1: only its broken value
        assert not bool(torch.isfinite(o[first:, 2:, 5]).any())
        if cache != "e4m3" or math.isnan(bad):
            others = [d for d in range(D) if d != 5]
            assert torch.equal(o[first:, 2:][:, :, others], c[first:, 2:][:, :, others])
        # heads 0 and 1 read key head 0: a score that is NaN or infinite
        seen = o[first:, :2].float()
        ok = seen.isnan() if math.isnan(bad) else seen.isnan() | (seen - c[first:, :2].float()).isfinite()
        assert bool(ok.all())


@gpu
@pytest.mark.parametrize("new", [2, 64])
def test_bad_pages_and_lengths(dev, new):
    """Recorded, not followed; the other sequences keep their results."""
    case = ([new, new, new], [500, 300, 90], 4, 2, 64, "bf16", "bf16", 16, "token")
    problem, args, q, keys, cu, _ = build(dev, *case)
    good, good_lse, _ = run(problem, args, dev)
    rows = slice(0, new), slice(2 * new, 3 * new)
    for what, bad in (("page_table", -1), ("page_table", 2 ** 31 - 1), ("page_table", problem.num_pages),
                      ("kv_len", -5), ("kv_len", 2 ** 31 - 1)):
        broken = dict(args)
        broken[what] = args[what].clone()
        if what == "page_table":
            broken[what][1, 7] = bad
        else:
            broken[what][1] = bad
        out, lse, ws = run(problem, broken, dev)
        assert moe.get_device_error(ws) == BAD_INDEX, (what, bad)
        for r in rows:
            ref.check(out[r], good[r].cpu().double(), good[r].cpu().double().abs() * 2.0 ** -6 + 2.0 ** -6, what)
        assert bool((out[3 * new:] == 7.0).all())
        run(problem, args, dev, ws=ws)
        assert moe.get_device_error(ws) == 0
    for cu_bad in ([0, new, -1, 3 * new], [0, new, 3 * new + 100, 3 * new], [-3, new, 2 * new, 3 * new]):
        broken = dict(args, cu_q=torch.tensor(cu_bad, dtype=torch.int32, device=dev))
        _, _, ws = run(problem, broken, dev)
        assert moe.get_device_error(ws) == BAD_INDEX


@gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 50])
def test_offsets_past_32_bits(dev, cache, new):
    """A cache of more than 2^32 elements: its last pages."""
    Hkv, D, page = 8, 128, 128
    pages = 2 ** 32 // (Hkv * D * page) + 5
    dt = torch.uint8 if cache == "e4m3" else torch.bfloat16
    L, Hq, g = 300, 16, gen(5)
    kc, vc = (torch.empty(pages, page, Hkv, D, dtype=dt, device=dev) for _ in range(2))
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32)
    ks = vs = None
    kv64 = []
    for c in (kc, vc):
        for p in table[0].tolist():
            if cache == "e4m3":
                c[p] = torch.randint(0, 0x50, (page, Hkv, D), generator=g, dtype=torch.uint8).to(dev)
            else:
                c[p] = randn(g, page, Hkv, D).bfloat16().to(dev)
        rows = torch.cat([c[p] for p in table[0].tolist()]).cpu()[:L]
        kv64.append(ref.e4m3_values(rows) * 0.5 if cache == "e4m3" else rows.double())
    if cache == "e4m3":
        ks, vs = (torch.full((pages, Hkv, page), 0.5, device=dev) for _ in range(2))
    q = randn(g, new, Hq * D).bfloat16()
    problem = moe.attention_problem(new, 1, Hq, Hkv, D, new, cache_dtype=cache, page_size=page, num_pages=pages, max_pages=3)
    cu = torch.tensor([0, new], dtype=torch.int32)
    args = dict(q=q.to(dev), k_cache=kc, v_cache=vc, page_table=table.to(dev), cu_q=cu.to(dev),
                kv_len=torch.tensor([L], dtype=torch.int32, device=dev), k_scale=ks, v_scale=vs)
    out, lse, ws = run(problem, args, dev)
    assert moe.get_device_error(ws) == 0
    compare(problem, out, lse, q, [kv64], cu, "bf16", cache, 0.5)


@gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 40])
def test_captured_calls_follow_the_lengths(dev, cache, new):
    case = ([new, new], [900, 140], 8, 2, 128, "bf16", cache, 16, "head")
    problem, args, q, keys, cu, unit = build(dev, *case, spare=0)
    ws = moe.alloc_attention_workspace(problem, dev)
    out = torch.zeros(problem.T, problem.Hq * problem.D, dtype=torch.bfloat16, device=dev)
    lse = torch.zeros(problem.T, problem.Hq, device=dev)

    def go(stream=None):
        moe.paged_attention(problem, args["q"], args["k_cache"], args["v_cache"], args["page_table"], args["cu_q"],
                            args["kv_len"], out, ws, k_scale=args["k_scale"], v_scale=args["v_scale"], lse=lse,
                            stream=stream)

    graph = torch.cuda.CUDAGraph()
    go()
    with torch.cuda.graph(graph):
        go()
    for lens in ([900, 140], [41, 99], [700, 130]):
        args["kv_len"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        got = out.clone()
        cut = [[t[:n] for t in pair] for pair, n in zip(keys, lens)]
        compare(problem, wide(got.cpu(), 8, dev, fill=7.0), lse, q, cut, cu, "bf16", cache, unit[1])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        go(side.cuda_stream)
        side.synchronize()
        assert torch.equal(out, got)


@gpu
@pytest.mark.parametrize("new", [1, 20])
def test_more_sequences_than_threads(dev, new):
    B = 1100
    case = ([new if i % 97 == 5 else 1 if i % 3 else 0 for i in range(B)], [i * 7 % 90 if i % 97 != 5 else 20 + i % 70 for i in range(B)],
            2, 1, 16, "bf16", "bf16", 16, "token")
    case[1][::3] = [n if m else 3 for n, m in zip(case[1][::3], case[0][::3])]
    problem, args, q, keys, cu, _ = build(dev, *case)
    out, lse, ws = run(problem, args, dev)
    assert moe.get_device_error(ws) == 0
    compare(problem, out, lse, q, keys, cu, "bf16", "bf16", None)


@gpu
def test_more_new_tokens_than_promised(dev):
    """max_q chooses the kernel: one too small costs time, not results."""
    case = ([40, 1], [90, 33], 4, 1, 64, "bf16", "bf16", 16, "token")
    problem, args, q, keys, cu, _ = build(dev, *case)
    problem.max_q = 1
    out, lse, ws = run(problem, args, dev)
    assert moe.get_device_error(ws) == 0
    compare(problem, out, lse, q, keys, cu, "bf16", "bf16", None)


@gpu
def test_two_streams_at_once(dev):
    """Calls on two streams, each with its own workspace."""
    cases = [([1] * 20, [3000 - 100 * i for i in range(20)], 8, 2, 128, "bf16", "bf16", 16, "token"),
             ([200], [1500], 8, 2, 128, "bf16", "e4m3", 16, "token")]
    made = [build(dev, *c) for c in cases]
    want = [run(m[0], m[1], dev)[0] for m in made]
    wss = [moe.alloc_attention_workspace(m[0], dev) for m in made]
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (s, m) in enumerate(zip(streams, made)):
            with torch.cuda.stream(s):
                got[i].append(run(m[0], m[1], dev, ws=wss[i])[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


@gpu
def test_python_refusals(dev):
    case = ([1, 1], [30, 20], 4, 2, 64, "bf16", "bf16", 16, "token")
    problem, args, *_ = build(dev, *case)
    ws = moe.alloc_attention_workspace(problem, dev)
    out = torch.zeros(problem.T, problem.Hq * problem.D, dtype=torch.bfloat16, device=dev)

    def go(**kw):
        a = {**args, "out": out, "lse": None, "ws": ws, **kw}
        moe.paged_attention(problem, a["q"], a["k_cache"], a["v_cache"], a["page_table"], a["cu_q"], a["kv_len"],
                            a["out"], a["ws"], k_scale=a["k_scale"], v_scale=a["v_scale"], lse=a["lse"])

    go()
    for bad in (dict(q=args["q"].half()), dict(q=args["q"].cpu()), dict(k_cache=args["k_cache"][1:]),
                dict(v_cache=args["v_cache"].transpose(2, 3)), dict(page_table=args["page_table"].long()),
                dict(page_table=args["page_table"][:, 1:]), dict(cu_q=args["cu_q"][1:]), dict(kv_len=args["kv_len"].cpu()),
                dict(lse=torch.zeros(problem.T, 1, device=dev)), dict(out=out.float())):
        with pytest.raises((ValueError, TypeError)):
            go(**bad)
    for bad in (dict(k_cache=None, v_cache=None), dict(ws=ws[:-1]), dict(k_scale=torch.zeros(problem.num_pages, 2, 16, device=dev))):
        with pytest.raises(moe.MoEError):
            go(**bad)
    with pytest.raises(moe.MoEError):
        moe.prompt_attention(problem, args["q"], args["q"][:, :128], args["q"][:, :128], args["cu_q"], out, ws)
