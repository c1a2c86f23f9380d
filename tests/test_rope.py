"""moe_qk_norm_rope: refusals (no GPU), tables, and the operator against its plain 64-bit form."""
import ctypes
import math

import pytest
import torch

import mixture_experts_layer_gate_gb300 as moe
from mixture_experts_layer_gate_gb300 import binding
from tests import attention_reference as att
from tests import op_reference as ref
from tests.test_operators import dev, far, gen, lib, randn, wide  # noqa: F401  (fixtures among them)

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
INVALID, UNSUPPORTED, WORKSPACE, BAD_INDEX = 1, 2, 3, 5
P = 4096  # an address that is never dereferenced: the checks come before any launch


# ------------------------------------------------------------------ refusals and tables (CPU)


def test_struct_layouts():
    assert ctypes.sizeof(moe.RopeProblem) == 52
    assert ctypes.sizeof(binding.KvStruct) == 80


def kv(k=P, v=P, ks=None, vs=None, page=64 * 4 * 16, token=64 * 4, head=64):
    return binding.KvStruct(k, v, ks, vs, page, token, head, page, token, head)


def call(lib, r, q=P, k=P, v=P, pos=P, turns=P, qw=None, kw=None, qo=P, ko=None, cache=None, slots=P, ws=P, ws_bytes=256,
         qs=None, ks=None, vs=None, qos=None, kos=None):
    nq, nk = (r.Hq * r.D, r.Hkv * r.D) if r is not None else (0, 0)
    own = lambda s, n: n if s is None else s  # noqa: E731
    return lib.moe_qk_norm_rope(ctypes.byref(r) if r is not None else None, q, own(qs, nq), k, own(ks, nk), v,
                                own(vs, nk), pos, turns, qw, kw, qo, own(qos, nq), ko, own(kos, nk),
                                ctypes.byref(cache) if cache is not None else None, slots, ws, ws_bytes, None)


def cached(T=3, D=64, **kw):
    return moe.rope_problem(T, 8, 4, D, page_size=16, num_pages=7, **kw)


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(pos=None), dict(turns=None),
                                dict(qo=None), dict(slots=None), dict(q=P + 2), dict(pos=P + 2), dict(turns=P + 4),
                                dict(qw=P + 8), dict(slots=P + 1), dict(qs=511), dict(qs=516), dict(vs=248),
                                dict(ko=P + 2), dict(ko=P, kos=260), dict(qos=520), dict(cache=kv(k=None)),
                                dict(cache=kv(v=P + 8)), dict(cache=kv(ks=P, vs=P)), dict(cache=kv(token=8)),
                                dict(cache=kv(head=68)), dict(cache=kv(page=-64))])
def test_refuses_arguments(lib, kw):
    kw = {"cache": kv(), **kw}
    assert call(lib, cached(), **kw) == INVALID


def test_refuses_problems(lib):
    assert call(lib, None) == INVALID
    for bad in (dict(Hq=0), dict(Hkv=0), dict(D=0), dict(D=60), dict(rot=7), dict(rot=66), dict(rot=-2), dict(T=-1),
                dict(interleaved=2), dict(dtype=2), dict(weight_dtype=1), dict(eps=-1.0), dict(eps=math.nan),
                dict(magnitude=math.inf), dict(cache_dtype=2), dict(page_size=8), dict(page_size=48), dict(num_pages=0),
                dict(page_size=2048)):
        r = cached()
        for n, v in bad.items():
            setattr(r, n, v)
        assert call(lib, r, cache=kv()) == INVALID, bad
    for bad in (dict(D=264), dict(Hq=5000), dict(num_pages=1 << 28)):
        r = cached()
        for n, v in bad.items():
            setattr(r, n, v)
        assert call(lib, r, cache=kv()) == UNSUPPORTED, bad
    assert call(lib, cached(), cache=kv(), ws=None) == WORKSPACE
    assert call(lib, cached(), cache=kv(), ws_bytes=255) == WORKSPACE
    # no cache: the keys have to go somewhere, and page_size says that there is none
    r = moe.rope_problem(3, 8, 4, 64)
    assert call(lib, r) == INVALID
    assert call(lib, cached(), ko=P) == INVALID
    # 8-bit rows are whole 16-byte pieces, and need both scales
    assert call(lib, cached(cache_dtype="e4m3"), cache=kv(ks=P)) == INVALID
    assert call(lib, cached(cache_dtype="e4m3"), cache=kv(ks=P, vs=P + 4)) == INVALID
    r = cached(D=72, cache_dtype="e4m3")
    assert call(lib, r, cache=kv(ks=P, vs=P, page=72 * 64, token=72 * 4, head=72)) == INVALID
    # nothing to do
    assert call(lib, cached(T=0), cache=kv()) == 0
    with pytest.raises(ValueError):
        moe.rope_problem(1, 1, 1, 64, dtype="bf16", cache_dtype="f16")
    with pytest.raises(KeyError):
        moe.rope_problem(1, 1, 1, 64, layout="other")


def test_table():
    for kw in (dict(), dict(theta=500000.0), dict(factor=4.0), dict(factor=8.0, original=8192, low=1.0, high=4.0)):
        table = moe.rope_table(64, **kw)
        want = att.frequencies(64, **kw) / (2 * math.pi)
        got = torch.tensor([(int(t) % 2 ** 64) / 2.0 ** 64 for t in table], dtype=torch.float64)
        assert table.dtype == torch.int64 and table.shape == (32,)
        assert torch.all((got - want).abs() <= want * 2.0 ** -50 + 2.0 ** -63)
    # frequencies of one's own: a whole turn is none, a negative one turns backwards
    t = moe.rope_table(6, inv_freq=[2 * math.pi, -math.pi / 2, math.pi])
    assert [int(x) for x in t] == [0, -2 ** 62, -2 ** 63]
    assert moe.rope_table(0).shape == (0,)
    for bad in (dict(rot=7), dict(rot=-2), dict(rot=4, factor=0.0), dict(rot=4, inv_freq=[1.0]),
                dict(rot=4, inv_freq=[1.0, math.inf])):
        with pytest.raises(ValueError):
            moe.rope_table(**bad)


# ------------------------------------------------------------------ against the 64-bit form


def make_cache(pages, page, heads, D, dtype, order, device):
    shape = (pages, page, heads, D) if order == "token" else (pages, heads, page, D)
    c = torch.randint(0, 255, (*shape, dtype.itemsize), dtype=torch.uint8).to(device).view(dtype).view(shape)
    return c if order == "token" else c.transpose(1, 2)


CASES = [  # T, Hq, Hkv, D, rot, layout, dtype, norm, cache, page, order
    (1, 32, 8, 128, 128, "half", "bf16", "f32", "bf16", 16, "token"),
    (16, 28, 4, 128, 128, "half", "bf16", "bf16", "e4m3", 64, "token"),
    (333, 8, 8, 64, 32, "interleaved", "f16", "f16", "f16", 32, "head"),
    (70, 7, 1, 80, 24, "half", "bf16", None, "bf16", 16, "head"),      # halves of 12: not whole chunks
    (5, 3, 3, 256, 256, "half", "f16", "f32", "e4m3", 16, "head"),
    (37, 5, 1, 16, 2, "half", "bf16", "bf16", "e4m3", 256, "token"),
    (2, 1, 1, 8, 8, "interleaved", "f16", "f32", "f16", 16, "token"),
    (9, 40, 8, 128, 0, "half", "bf16", "f32", "e4m3", 128, "head"),    # no rotation
    (700, 12, 4, 96, 96, "half", "f16", None, "e4m3", 64, "token"),
    (64, 6, 2, 104, 102, "interleaved", "bf16", "f32", "bf16", 1024, "token"),
    (11, 4, 2, 64, 62, "half", "f16", "f16", None, 0, ""),             # no cache
]


@gpu
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("in_place", [False, True])
def test_matches_plain(dev, case, in_place):
    T, Hq, Hkv, D, rot, layout, dtype, norm, cache, page, order = case
    dt, g = DT[dtype], gen(T * 7 + D)
    x = [randn(g, T, n * D).to(dt) for n in (Hq, Hkv, Hkv)]
    x[0][0, :D] = 0  # an empty head
    x[2][T // 2, -D:] = 0
    weights = [None, None] if norm is None else [(1 + 0.2 * randn(g, D)).to(DT[norm]) for _ in range(2)]
    pos = torch.randint(0, 2_000_000, (T,), generator=g, dtype=torch.int32)
    pos[0] = 2 ** 31 - 1
    kw = dict(theta=10000.0, factor=16.0, original=4096, low=1.0, high=32.0)
    turns, magnitude = moe.rope_table(rot, device=dev, **kw), 1.25
    q, k, v = (wide(t, 8, dev) for t in x)
    new = lambda t: torch.empty(t.shape, dtype=t.dtype, device=dev)  # noqa: E731
    qo, ko = (q, k) if in_place else (new(q), new(k))
    pages = 0 if cache is None else -(-T // page) + 1
    args, want_cache = {}, None
    if cache is not None:
        cdt = torch.uint8 if cache == "e4m3" else dt
        kc, vc = (make_cache(pages, page, Hkv, D, cdt, order, dev) for _ in range(2))
        slots = torch.randperm(pages * page, generator=g)[:T].int()
        slots[T // 3] = -1 if T > 1 else slots[0]
        args = dict(v=v, k_cache=kc, v_cache=vc, slots=slots.to(dev))
        if cache == "e4m3":
            args["k_scale"], args["v_scale"] = (torch.full((pages, Hkv, page), 7.0, device=dev) for _ in range(2))
        want_cache = [t.clone() for t in (kc, vc)]
    r = moe.rope_problem(T, Hq, Hkv, D, rot=rot, layout=layout, dtype=dtype, weight_dtype=norm, magnitude=magnitude,
                         cache_dtype=cache, page_size=page, num_pages=pages)
    ws = moe.alloc_op_workspace(dev)
    moe.qk_norm_rope(r, q, k, pos.to(dev), turns, qo, ws, k_out=None if in_place and cache else ko,
                     q_weight=None if norm is None else weights[0].to(dev),
                     k_weight=None if norm is None else weights[1].to(dev), **args)
    assert moe.get_device_error(ws) == 0
    freq = att.frequencies(rot, **kw)
    heads = [t.view(T, -1, D) for t in x]
    full = [att.norm_rotate(h, w, pos, freq, layout == "interleaved", r.eps, magnitude)
            for h, w in zip(heads, weights)]
    full.append((heads[2].double(), torch.zeros_like(heads[2].double())))
    rel, tiny = ref.half_step(dt)
    for got, (val, dv), name in ((qo, full[0], "q"), (ko, full[1], "k")):
        if name == "k" and in_place and cache:
            continue
        ref.check(got.view(T, -1, D) if not in_place else got.reshape(T, -1, D), val, dv + (val.abs() + dv) * rel + tiny,
                  name)
    if cache is None:
        return
    stored = (slots >= 0).nonzero()[:, 0]
    at = slots[stored].long()
    for i, name in ((1, "k"), (2, "v")):
        c, before = args[name + "_cache"], want_cache[i - 1]
        val, dv = full[i][0][stored], full[i][1][stored]
        got = c[at // page, at % page]  # [n, Hkv, D]
        if cache == "e4m3":
            scales = args[name + "_scale"][at // page, :, at % page]  # [n, Hkv]
            ref.check_quantised(got.reshape(-1, D), scales.reshape(-1, 1), val.reshape(-1, D), dv.reshape(-1, D), D,
                                name)
            assert int((args[name + "_scale"] != 7.0).sum()) <= len(stored) * Hkv
        else:
            ref.check(got, val, dv + (val.abs() + dv) * rel + tiny, name)
        # what lies between the slots stays
        rest = torch.ones(pages * page, dtype=torch.bool)
        rest[at] = False
        flat = lambda t: t.reshape(pages * page, -1).contiguous().view(torch.uint8)  # noqa: E731
        assert torch.equal(flat(c).cpu()[rest], flat(before).cpu()[rest])


@gpu
def test_bad_slots_are_recorded(dev):
    T, H, D, page, pages = 4, 2, 64, 16, 2
    q, k, v = (torch.ones(T, H * D, dtype=torch.bfloat16, device=dev) for _ in range(3))
    kc, vc = (torch.zeros(pages, page, H, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    r = moe.rope_problem(T, H, H, D, page_size=page, num_pages=pages)
    ws = moe.alloc_op_workspace(dev)
    slots = torch.tensor([pages * page, 2 ** 31 - 1, -2 ** 31, 5], dtype=torch.int32, device=dev)
    moe.qk_norm_rope(r, q, k, torch.zeros(T, dtype=torch.int32, device=dev), moe.rope_table(D, device=dev), q.clone(),
                     ws, v=v, k_cache=kc, v_cache=vc, slots=slots)
    assert moe.get_device_error(ws) == BAD_INDEX
    assert float(vc.sum()) == H * D and float(vc[0, 5].sum()) == H * D


@gpu
def test_values_that_are_not_finite(dev):
    """A NaN or infinity stays in its head."""
    T, H, D, page = 3, 4, 128, 16
    g = gen(3)
    x = [randn(g, T, H * D).to(torch.bfloat16) for _ in range(3)]
    x[1][1, D + 3] = math.nan
    x[2][2, 2 * D + 5] = math.inf
    r = moe.rope_problem(T, H, H, D, cache_dtype="e4m3", page_size=page, num_pages=1)
    kc, vc = (torch.zeros(1, page, H, D, dtype=torch.uint8, device=dev) for _ in range(2))
    ks, vs = (torch.zeros(1, H, page, device=dev) for _ in range(2))
    q, k, v = (t.to(dev) for t in x)
    w = torch.ones(D, dtype=torch.bfloat16, device=dev)
    moe.qk_norm_rope(r, q, k, torch.arange(T, dtype=torch.int32, device=dev), moe.rope_table(D, device=dev), q,
                     moe.alloc_op_workspace(dev), v=v, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs,
                     slots=torch.arange(T, dtype=torch.int32, device=dev), q_weight=w, k_weight=w)
    nan = ref.e4m3_values(kc[0, :T]).isnan()
    assert bool(nan[1, 1].all()) and int(nan.sum()) == D
    assert ks[0, 1, 1].isnan() and int(ks.isnan().sum()) == 1
    assert vs[0, 2, 2].isinf() and int(vs.isinf().sum()) == 1
    nan = ref.e4m3_values(vc[0, :T]).isnan()
    assert int(nan.sum()) == 1 and bool(nan[2, 2, 5])


@gpu
def test_python_refusals(dev):
    T, H, D = 2, 2, 64
    r = moe.rope_problem(T, H, H, D, page_size=16, num_pages=2)
    q = torch.ones(T, H * D, dtype=torch.bfloat16, device=dev)
    kc = torch.zeros(2, 16, H, D, dtype=torch.bfloat16, device=dev)
    ok = dict(v=q, k_cache=kc, v_cache=kc.clone(), slots=torch.zeros(T, dtype=torch.int32, device=dev))
    pos, turns, ws = torch.zeros(T, dtype=torch.int32, device=dev), moe.rope_table(D, device=dev), moe.alloc_op_workspace(dev)
    for bad in (dict(k_cache=kc.half()), dict(k_cache=kc[:1]), dict(v_cache=kc.transpose(1, 3)), dict(k_cache=kc.cpu()),
                dict(slots=ok["slots"].long()), dict(k_scale=torch.zeros(2, H, 16)), dict(v=q.float()),
                dict(k_cache=None, v_cache=None, k_scale=torch.zeros(2, H, 16, device=dev))):
        with pytest.raises((ValueError, TypeError)):
            moe.qk_norm_rope(r, q, q.clone(), pos, turns, q.clone(), ws, **{**ok, **bad})
    for args in ((q, q, pos.long(), turns), (q, q, pos, turns[:-1]), (q[:, ::2], q, pos, turns)):
        with pytest.raises(ValueError):
            moe.qk_norm_rope(r, *args, q.clone(), ws, **ok)
    with pytest.raises(moe.MoEError):  # no place for the keys
        moe.qk_norm_rope(moe.rope_problem(T, H, H, D), q, q, pos, turns, q.clone(), ws)
