"""The paged key-value cache operators on the GPU against plain 64-bit forms (attn_ref.py)."""
import ctypes
import math
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_ref  # noqa: E402

pytestmark = pytest.mark.gpu

F16, Q8_0 = 7, 1


@pytest.fixture(scope="module")
def syn():
    import torch
    assert torch.cuda.is_available()
    from gguf_block_quantized_gb300 import syn
    yield syn
    torch.cuda.synchronize()
    assert syn.device_status() == syn.OK


def make_cache(syn, rng, t, kv, dim, page, lens, garbage=np.nan, extra=3):
    """A cache with random rows for sequences of the given lengths in shuffled pages; every row
    that belongs to no sequence holds `garbage`.  -> (cache, pages tensor, [(k, v) float64])."""
    import torch
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + extra
    order = rng.permutation(n_pages)
    most = max(1, max(need))
    table = np.full((len(lens), most), -1, np.int32)
    shape = (n_pages, kv, page, dim)
    vals = [np.full(shape, garbage, np.float32) for _ in range(2)]
    mean = [rng.standard_normal((kv, dim)).astype(np.float32) for _ in range(2)]
    at = 0
    for s, n in enumerate(lens):
        mine = order[at:at + need[s]]
        at += need[s]
        table[s, :need[s]] = mine
        for x, mu in zip(vals, mean):
            for i, pg in enumerate(mine):
                m = min(page, n - i * page)
                x[pg, :, :m] = (rng.standard_normal((kv, m, dim)) + mu[:, None]).astype(np.float32)
    if t == F16:
        pools = [torch.from_numpy(x.astype(np.float16)).cuda() for x in vals]
        exact = [x.astype(np.float16).astype(np.float64) for x in vals]
    else:
        pools, exact = [], []
        for x in vals:
            b = x.reshape(n_pages, kv, page, dim // 32, 32)
            with np.errstate(invalid="ignore"):
                d = (np.abs(b).max(-1) / 127).astype(np.float16)
                c = np.nan_to_num(np.clip(np.rint(b / d[..., None].astype(np.float32)), -127, 127)).astype(np.int8)
            raw = np.concatenate([c.reshape(n_pages, kv, -1).view(np.uint8), d.reshape(n_pages, kv, -1).view(np.uint8)], -1)
            pools.append(torch.from_numpy(np.ascontiguousarray(raw)).cuda())
            exact.append((c.astype(np.float64) * d.astype(np.float64)[..., None]).reshape(shape))
    cache = syn.KVCache(t, kv, dim, page, *pools)
    seqs = []
    for s, n in enumerate(lens):
        mine = table[s, :need[s]]
        seqs.append(tuple(x[mine].transpose(0, 2, 1, 3).reshape(-1, kv, dim)[:n] if n else np.zeros((0, kv, dim))
                          for x in exact))
    return cache, torch.from_numpy(table).cuda(), seqs


def options(rng, lens, new, heads, cap=0.0, window=0, prefix=False, slopes=False, docs=False):
    """(keyword arguments of the calls, per-sequence arrays for the reference)."""
    import torch
    rows = [np.arange(n - m, n) for n, m in zip(lens, new)]
    pre = np.array([rng.integers(0, n + 2) if prefix else 0 for n in lens], np.int32)
    first = [np.array([rng.integers(-1, max(1, p) + 1) if docs else 0 for p in r], np.int32) for r in rows]
    sl = (2.0 ** (-8.0 * (np.arange(heads) + 1) / heads)).astype(np.float32) if slopes else None
    kw = {"cap": cap, "window": window,
          "prefix": torch.from_numpy(pre).cuda() if prefix else None,
          "first": torch.from_numpy(np.concatenate(first) if first else np.zeros(0, np.int32)).cuda() if docs else None,
          "slopes": torch.from_numpy(sl).cuda() if slopes else None}
    return kw, rows, first, pre, sl


def reference(q, seqs, rows, first, pre, window, scale, cap, slopes):
    outs, sizes, at = [], [], 0
    for s, (k, v) in enumerate(seqs):
        n = len(rows[s])
        o, b = attn_ref.attention(q[at:at + n], k, v, rows[s], first[s], min(int(pre[s]), len(k)), window, scale, cap, slopes)
        outs.append(o)
        sizes.append(b)
        at += n
    return np.concatenate(outs), np.concatenate(sizes)


# Decode: the scores are sums of exact products with at most a few fp32 roundings of the running
# sum, itself at most A = sum |q_i k_i| * scale; a score error e changes the output by at most
# 2 e max|v|.  2^-20 (1 + A) max|v| leaves 4 to 8 roundings of 2^-23 for each.  An fp16 output
# adds half a unit of its last place.
def decode_bound(size, out, f16):
    return 2.0 ** -20 * size + (np.abs(out) * 2.0 ** -11 + 2.0 ** -24 if f16 else 0)


LENS = [1, 0, 15, 16, 17, 63, 64, 65, 200, 7, 1000, 129]


@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("heads,kv,dim,page", [(8, 2, 64, 16), (4, 4, 32, 8), (12, 1, 96, 32), (8, 1, 128, 64),
                                               (20, 2, 128, 8), (3, 1, 160, 16), (16, 2, 256, 128), (24, 1, 64, 256),
                                               (40, 1, 256, 8)])
def test_decode_shapes(syn, t, heads, kv, dim, page):
    import torch
    rng = np.random.default_rng([t, heads, kv, dim, page])
    cache, pages, seqs = make_cache(syn, rng, t, kv, dim, page, LENS)
    q = rng.standard_normal((len(LENS), heads, dim)).astype(np.float16)
    kw, rows, first, pre, sl = options(rng, LENS, [min(1, n) for n in LENS], heads)
    rows = [np.array([n - 1]) for n in LENS]
    first = [np.zeros(1, np.int32) for _ in LENS]
    ref, size = reference(q, seqs, rows, first, pre, 0, dim ** -0.5, 0.0, None)
    lens = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    for dt in (torch.float32, torch.float16):
        out = torch.full((len(LENS), heads, dim), float("nan"), dtype=dt, device="cuda")
        got = syn.attn_decode(cache, torch.from_numpy(q).cuda(), pages, lens, out, **kw).double().cpu().numpy()
        assert (np.abs(got - ref) <= decode_bound(size, ref, dt == torch.float16)).all()
        assert (got[1] == 0).all()  # no keys: zeros
    assert syn.device_status() == syn.OK


@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("opt", [{"cap": 5.0}, {"window": 37}, {"window": 1}, {"slopes": True}, {"docs": True},
                                 {"window": 40, "prefix": True}, {"cap": 20.0, "window": 100, "prefix": True,
                                                                  "slopes": True, "docs": True}])
def test_decode_options(syn, t, opt):
    import torch
    heads, kv, dim, page = 8, 2, 64, 16
    rng = np.random.default_rng([t, 5])
    lens = LENS + [500, 333, 90]
    cache, pages, seqs = make_cache(syn, rng, t, kv, dim, page, lens)
    q = (2 * rng.standard_normal((len(lens), heads, dim))).astype(np.float16)
    one = [1] * len(lens)
    kw, rows, first, pre, sl = options(rng, lens, one, heads, **opt)
    ref, size = reference(q, seqs, rows, first, pre, kw["window"], 0.3, kw["cap"], sl)
    got = syn.attn_decode(cache, torch.from_numpy(q).cuda(), pages, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                          scale=0.3, **kw).double().cpu().numpy()
    assert (np.abs(got - ref) <= decode_bound(size, ref, False)).all()


@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("limit", [0, 5])
def test_decode_split_long(syn, t, limit):
    """A long sequence beside short ones: its partials are joined over many CTAs; twice with the
    same bits (the join is in order), and once with few SMs."""
    import torch
    heads, kv, dim, page = 8, 2, 128, 32
    rng = np.random.default_rng([t, 9])
    lens = [20011, 1, 300]
    cache, pages, seqs = make_cache(syn, rng, t, kv, dim, page, lens)
    q = rng.standard_normal((3, heads, dim)).astype(np.float16)
    ref, size = reference(q, seqs, [np.array([n - 1]) for n in lens], [np.zeros(1)] * 3, [0] * 3, 0, dim ** -0.5, 0.0, None)
    qd, ld = torch.from_numpy(q).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    old = syn.set_sm_limit(limit)
    try:
        a = syn.attn_decode(cache, qd, pages, ld)
        b = syn.attn_decode(cache, qd, pages, ld)
    finally:
        syn.set_sm_limit(old)
    assert torch.equal(a, b)
    assert (np.abs(a.double().cpu().numpy() - ref) <= decode_bound(size, ref, False)).all()


def test_decode_many_sequences(syn):
    """More sequences than one launch takes."""
    import torch
    rng = np.random.default_rng(3)
    heads, kv, dim, page = 4, 1, 32, 8
    lens = [int(n) for n in rng.integers(0, 40, 2500)]
    cache, pages, seqs = make_cache(syn, rng, F16, kv, dim, page, lens)
    q = rng.standard_normal((len(lens), heads, dim)).astype(np.float16)
    first = rng.integers(0, 3, len(lens)).astype(np.int32)
    ref, size = reference(q, seqs, [np.array([n - 1]) for n in lens], [first[i:i + 1] for i in range(len(lens))],
                          [0] * len(lens), 0, dim ** -0.5, 0.0, None)
    got = syn.attn_decode(cache, torch.from_numpy(q).cuda(), pages, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                          first=torch.from_numpy(first).cuda()).double().cpu().numpy()
    assert (np.abs(got - ref) <= decode_bound(size, ref, False)).all()


def test_decode_deterministic_mode(syn):
    """In deterministic mode a sequence's output has the same bits alone and in a batch."""
    import torch
    rng = np.random.default_rng(4)
    heads, kv, dim, page = 8, 2, 128, 16
    lens = [700, 3, 4000, 0, 129]
    cache, pages, _ = make_cache(syn, rng, Q8_0, kv, dim, page, lens)
    q = torch.from_numpy(rng.standard_normal((5, heads, dim)).astype(np.float16)).cuda()
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    free = syn.attn_decode(cache, q, pages, ld)
    old = syn.set_deterministic(True)
    try:
        whole = syn.attn_decode(cache, q, pages, ld)
        lim = syn.set_sm_limit(3)
        few = syn.attn_decode(cache, q, pages, ld)
        syn.set_sm_limit(lim)
        for s in range(5):
            one = syn.attn_decode(cache, q[s:s + 1].contiguous(), pages[s:s + 1].contiguous(), ld[s:s + 1].contiguous())
            assert torch.equal(one[0], whole[s])
    finally:
        syn.set_deterministic(old)
    assert torch.equal(few, whole)
    assert (whole - free).abs().max().item() < 1e-4


def test_decode_strides_streams_and_graphs(syn):
    """q and out as slices of wider buffers, K and V pools interleaved in one allocation, another
    stream than the current one, and a captured graph replayed on longer lengths."""
    import torch
    rng = np.random.default_rng(6)
    heads, kv, dim, page = 8, 2, 64, 16
    lens = [50, 131, 9]
    cache, pages, seqs = make_cache(syn, rng, F16, kv, dim, page, lens, garbage=np.inf)
    both = torch.stack([cache.k, cache.v], 1)
    mixed = syn.KVCache(F16, kv, dim, page, both[:, 0], both[:, 1])
    assert mixed.desc.page_stride == 2 * kv * page * dim * 2
    wide = torch.randn((3, heads + 4, dim), device="cuda").half()
    wide_out = torch.zeros((3, heads + 8, dim), device="cuda")
    q = wide[:, 2:2 + heads]
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ref, size = reference(q.cpu().numpy(), seqs, [np.array([n - 1]) for n in lens], [np.zeros(1)] * 3, [0] * 3, 0,
                          dim ** -0.5, 0.0, None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    step = syn.prepare_attn_decode(mixed, q, pages, ld, wide_out[:, 3:3 + heads], stream=side)
    step()
    side.synchronize()
    got = wide_out[:, 3:3 + heads].double().cpu().numpy()
    assert (np.abs(got - ref) <= decode_bound(size, ref, False)).all()
    assert (wide_out[:, :3] == 0).all() and (wide_out[:, 3 + heads:] == 0).all()
    # a graph captured at short lengths, replayed at the full ones
    ld.copy_(torch.tensor([1, 1, 0], dtype=torch.int32))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    ld.copy_(torch.tensor(lens, dtype=torch.int32))
    wide_out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(wide_out[:, 3:3 + heads].double().cpu().numpy(), got)


def test_bad_page_is_not_followed(syn):
    """A page id outside the pool is skipped and reported; the other sequences are right."""
    import torch
    rng = np.random.default_rng(8)
    heads, kv, dim, page = 4, 2, 64, 16
    lens = [40, 40]
    cache, pages, seqs = make_cache(syn, rng, F16, kv, dim, page, lens)
    q = rng.standard_normal((2, heads, dim)).astype(np.float16)
    ref, size = reference(q, seqs, [np.array([39])] * 2, [np.zeros(1)] * 2, [0] * 2, 0, dim ** -0.5, 0.0, None)
    assert syn.device_status() == syn.OK
    for bad in (-5, 10 ** 6):
        p = pages.clone()
        p[0, 1] = bad
        got = syn.attn_decode(cache, torch.from_numpy(q).cuda(), p, torch.tensor(lens, dtype=torch.int32, device="cuda"))
        assert syn.device_status(clear=True) == syn.ERR_BOUNDS
        assert (np.abs(got[1].double().cpu().numpy() - ref[1]) <= decode_bound(size[1], ref[1], False)).all()
    assert syn.device_status() == syn.OK


# ---- append and read -----------------------------------------------------------------------

# The angle is exact to 2^-24 turns (3.8e-7 radians) and sine, cosine and the two products to a
# few 2^-24: 2^-20 of the pair's size bounds them; fp16 adds half a unit of its last place.
@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("heads,kv,dim,page,n,rot,layout,axes", [
    (4, 2, 64, 16, 33, 64, 1, 1), (4, 2, 64, 16, 1, 64, 0, 1), (0, 1, 32, 8, 5, 0, 0, 1), (6, 3, 96, 32, 70, 72, 1, 3),
    (5, 1, 128, 64, 17, 96, 0, 1), (32, 8, 128, 64, 40, 128, 1, 1), (3, 3, 160, 8, 9, 80, 1, 2), (2, 1, 256, 128, 300, 256, 0, 1),
    (40, 40, 256, 16, 3, 24, 1, 3)])
@pytest.mark.parametrize("fused", [False, True])
def test_append(syn, t, heads, kv, dim, page, n, rot, layout, axes, fused):
    import torch
    import oracle
    rng = np.random.default_rng([heads, kv, dim, n, rot])
    x = rng.standard_normal((n, heads + 2 * kv, dim)).astype(np.float32)
    x *= np.exp(rng.uniform(-3, 3, (n, 1, 1))).astype(np.float32)
    if n > 3:
        x[2, heads:] = 0  # zero rows: zero scale
    xd = torch.from_numpy(x).cuda()
    q, k, v = xd[:, :heads], xd[:, heads:heads + kv], xd[:, heads + kv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = rng.integers(-1000, 2 ** 31 - 1, (axes, n)).astype(np.int32)
    pos[:, : n // 2] %= 5000
    axis = rng.integers(0, axes, rot // 2).astype(np.uint8) if axes > 1 else None
    factors = rng.uniform(0.5, 8, rot // 2).astype(np.float32)
    n_pages = n // page + 3
    slots = rng.permutation(n_pages * page)[:n].astype(np.int64)
    if n > 2:
        slots[1] = -1
    cache = syn.KVCache.empty(t, kv, dim, page, n_pages)
    cache.k.fill_(1), cache.v.fill_(1)
    rope = syn.Rope(rot, 10000.0, 0.5, factors, layout, axis, 1.25)
    got = syn.kv_append(cache, rope, k, v, torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda(),
                        q if heads else None)
    rk, rv = syn.kv_read(cache, torch.from_numpy(slots).cuda())
    want = attn_ref.rotate(x, pos, rot, 10000.0, layout, axis, 0.5, factors, 1.25)
    pair = np.abs(x).max(-1, keepdims=True).astype(np.float64) * 2.0 ** -20 * 2 * 1.25
    half = lambda y: np.abs(y) * 2.0 ** -11 + 2.0 ** -24  # noqa: E731
    if heads:
        assert (np.abs(got.double().cpu().numpy() - want[:, :heads]) <= pair[:, :heads] + half(want[:, :heads])).all()
    else:
        assert got is None
    kept = slots >= 0
    wk, xv, pair = want[:, heads:heads + kv], x[:, heads + kv:], pair[:, heads:heads + kv]
    gk, gv = rk.double().cpu().numpy(), rv.double().cpu().numpy()
    assert (gk[~kept] == 0).all() and (gv[~kept] == 0).all()
    if t == F16:
        assert (np.abs(gk - wk) <= pair + half(wk))[kept].all()
        assert np.array_equal(rv.cpu().numpy()[kept], xv.astype(np.float16)[kept])
        untouched = np.ones(n_pages * page, bool)
        untouched[slots[kept]] = False
        flat = cache.k.transpose(1, 2).reshape(n_pages * page, kv, dim).cpu().numpy()
        assert (flat[untouched] == 1).all()
    else:
        # k: within half a step of its block's scale (the rotation's error can move a value over a
        # tie, and the scale by a unit of fp16), then one fp16 rounding
        amax = np.abs(wk).reshape(n, kv, -1, 32).max(-1).repeat(32, -1)
        assert (np.abs(gk - wk) <= amax / 127 * 0.5 * (1 + 2.0 ** -9) + 127 * amax / 127 * 2.0 ** -10 + pair + half(wk)
                + 2.0 ** -17)[kept].all()
        # v is not rotated: the codes and scales are those of the block format's encoder, bit for bit
        blocks = oracle.quantize(Q8_0, np.ascontiguousarray(xv.reshape(n * kv, dim))).reshape(n, kv, dim // 32, 34)
        pool = cache.v.cpu().numpy()
        for i in np.nonzero(kept)[0]:
            pg, cell = divmod(int(slots[i]), page)
            codes = pool[pg, :, cell * dim:(cell + 1) * dim].reshape(kv, dim // 32, 32)
            scales = pool[pg, :, page * dim + cell * dim // 16:page * dim + (cell + 1) * dim // 16].reshape(kv, dim // 32, 2)
            assert np.array_equal(codes, blocks[i, :, :, 2:]) and np.array_equal(scales, blocks[i, :, :, :2])
    assert syn.device_status() == syn.OK


def test_append_nonfinite_and_overflow(syn):
    """F16 overflows to infinity as fp16 does; a Q8_0 block that cannot be stored reads as NaN, and
    its neighbours are right."""
    import torch
    dim = 64
    k = torch.zeros((1, 1, dim), device="cuda")
    k[0, 0, 3], k[0, 0, 40] = 1e6, 2.0
    v = torch.ones((1, 1, dim), device="cuda")
    v[0, 0, 50] = float("nan")
    slots = torch.tensor([5], device="cuda")
    rope = syn.Rope(0)
    c = syn.KVCache.empty(F16, 1, dim, 8, 2)
    syn.kv_append(c, rope, k, v, None, slots)
    rk, rv = syn.kv_read(c, slots)
    assert torch.isinf(rk[0, 0, 3]) and rk[0, 0, 40] == 2 and torch.isnan(rv[0, 0, 50]) and rv[0, 0, 49] == 1
    c = syn.KVCache.empty(Q8_0, 1, dim, 8, 2)
    k[0, 0, 3] = 1e9
    syn.kv_append(c, rope, k, v, None, slots)
    rk, rv = syn.kv_read(c, slots)
    assert torch.isnan(rk[0, 0, :32]).all() and rk[0, 0, 40] == 2 and (rk[0, 0, 41:] == 0).all()
    assert torch.isnan(rv[0, 0, 32:]).all() and (rv[0, 0, :32] == 1).all()


def test_append_bad_slot_is_not_followed(syn):
    import torch
    c = syn.KVCache.empty(F16, 2, 64, 8, 2)
    k = torch.randn((2, 2, 64), device="cuda")
    slots = torch.tensor([16, 3], device="cuda")
    syn.kv_append(c, syn.Rope(0), k, k, None, slots)
    assert syn.device_status(clear=True) == syn.ERR_BOUNDS
    assert torch.equal(c.k[0, :, 3], k[1].half()) and c.k.count_nonzero() == k[1].half().count_nonzero()
    rk, _ = syn.kv_read(c, slots)
    assert syn.device_status(clear=True) == syn.ERR_BOUNDS
    assert (rk[0] == 0).all() and torch.equal(rk[1], k[1].half())


# ---- prefill -------------------------------------------------------------------------------

# p is rounded to fp16 (relative 2^-11 at most), as are the expanded Q8_0 keys and values; a score
# error e changes the output by at most 2 e max|v|.  F16: 2^-11 max|v| for p and 2^-20 (1 + A) max|v|
# for fp32 scores; Q8_0: also 2^-11 A (keys, twice e) and 2^-11 (values).  An fp16 output adds half a
# unit of its last place.
def prefill_bound(t, size, vmax, out, f16):
    b = vmax * 2.0 ** -11 + size * 2.0 ** -20
    if t == Q8_0:
        b = b + vmax * 2.0 ** -11 + 2 * size * 2.0 ** -11
    return b + (np.abs(out) * 2.0 ** -11 + 2.0 ** -24 if f16 else 0)


def run_prefill(syn, t, heads, kv, dim, page, lens, new, seed, scale=None, garbage=np.nan, dts=("float32", "float16"),
                qscale=1.0, **opt):
    import torch
    rng = np.random.default_rng([t, heads, kv, dim, page, seed])
    cache, pages, seqs = make_cache(syn, rng, t, kv, dim, page, lens, garbage=garbage)
    n_tok = sum(new)
    q = (qscale * rng.standard_normal((n_tok, heads, dim))).astype(np.float16)
    kw, rows, first, pre, sl = options(rng, lens, new, heads, **opt)
    sc = dim ** -0.5 if scale is None else scale
    ref, size = reference(q, seqs, rows, first, pre, kw["window"], sc, kw["cap"], sl)
    vmax = np.concatenate([np.full((n, 1, 1), np.abs(v).max() if v.size else 0.0) for n, (_, v) in zip(new, seqs)])
    starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for dt in dts:
        out = torch.full((n_tok, heads, dim), float("nan"), dtype=getattr(torch, dt), device="cuda")
        got = syn.attn_prefill(cache, torch.from_numpy(q).cuda(), starts, pages, ld, out, scale=scale, **kw)
        got = got.double().cpu().numpy()
        err, bound = np.abs(got - ref), prefill_bound(t, size, vmax, ref, dt == "float16")
        assert (err <= bound).all(), (np.nanmax(err / np.maximum(bound, 1e-30)), np.argwhere(~(err <= bound))[:5])
    assert syn.device_status() == syn.OK


@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("heads,kv,dim,page", [(8, 2, 64, 16), (4, 4, 32, 8), (12, 1, 96, 32), (8, 1, 128, 64),
                                               (5, 1, 128, 8), (3, 1, 160, 16), (4, 2, 256, 128), (24, 1, 64, 256)])
def test_prefill_shapes(syn, t, heads, kv, dim, page):
    run_prefill(syn, t, heads, kv, dim, page, [1, 17, 128, 129, 300, 5, 64, 0], [1, 17, 40, 129, 33, 0, 2, 0], 1)


@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("opt", [{"cap": 5.0}, {"window": 37}, {"window": 1}, {"slopes": True}, {"docs": True}, {"prefix": True},
                                 {"window": 140, "prefix": True}, {"cap": 20.0, "window": 100, "prefix": True, "slopes": True,
                                                                   "docs": True}])
def test_prefill_options(syn, t, dim, opt):
    run_prefill(syn, t, 4, 2, dim, 16, [150, 400, 31, 270], [150, 60, 31, 1], 2, scale=0.1, **opt)


@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prefill_split_long(syn, t, dim):
    """A few tokens over a long cache: the item's keys are split between CTAs and joined."""
    run_prefill(syn, t, 4, 2, dim, 64, [9001, 2000], [5, 1], 3)


def test_prefill_growing_maxima(syn):
    """Scores that grow along the row by far more than the maximum's lag."""
    import torch
    rng = np.random.default_rng(12)
    dim, page, n = 64, 16, 700
    k = rng.standard_normal((n, 1, dim)) * (1 + np.arange(n)[:, None, None] / 20.0)
    v = rng.standard_normal((n, 1, dim))
    q = rng.standard_normal((30, 2, dim)).astype(np.float16)
    cache = syn.KVCache.empty(F16, 1, dim, page, 44)
    kp = np.zeros((44 * page, 1, dim), np.float16)
    vp = np.zeros_like(kp)
    kp[:n], vp[:n] = k, v
    cache.k.copy_(torch.from_numpy(kp.reshape(44, page, 1, dim).transpose(0, 2, 1, 3).copy()))
    cache.v.copy_(torch.from_numpy(vp.reshape(44, page, 1, dim).transpose(0, 2, 1, 3).copy()))
    pages = torch.arange(44, dtype=torch.int32, device="cuda").view(1, -1)
    pos = np.arange(n - 30, n)
    ref, size = attn_ref.attention(q, kp[:n], vp[:n], pos, np.zeros(30), 0, 0, 1.0, 0.0, None)
    got = syn.attn_prefill(cache, torch.from_numpy(q).cuda(), torch.tensor([0, 30], dtype=torch.int32, device="cuda"), pages,
                           torch.tensor([n], dtype=torch.int32, device="cuda"), scale=1.0).double().cpu().numpy()
    assert (np.abs(got - ref) <= prefill_bound(F16, size, np.abs(vp).max(), ref, False)).all()


@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_prefill_scales_that_are_not_positive(syn, scale):
    run_prefill(syn, F16, 2, 1, 64, 16, [200], [70], 4, scale=scale)


@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("split", [False, True])
def test_prefill_nonfinite_values_stay_where_they_are_seen(syn, t, split):
    """A NaN or infinity in a cached row reaches the rows that see it and no other, although they
    share tiles."""
    import torch
    rng = np.random.default_rng(14)
    heads, kv, dim, page, n, new = 4, 2, 64, 16, 1500 if split else 300, 40
    cache, pages, seqs = make_cache(syn, rng, t, kv, dim, page, [n])
    q = rng.standard_normal((new, heads, dim)).astype(np.float16)
    bad = n - 20  # seen by the last 20 tokens
    pg, cell = int(pages[0, bad // page]), bad % page
    if t == F16:
        cache.v[pg, :, cell, 5] = float("inf")
        cache.k[pg, 0, cell, 3] = float("nan")
    else:
        for pool, code in ((cache.v, 0x7C00), (cache.k, 0x7E00)):
            at = page * dim + cell * dim // 16
            pool[pg, 0, at:at + 2] = torch.tensor([code & 255, code >> 8], dtype=torch.uint8, device="cuda")
    k, v = seqs[0]
    pos = np.arange(n - new, n)
    ref, size = attn_ref.attention(q, k, v, pos, np.zeros(new), 0, 0, dim ** -0.5, 0.0, None)
    got = syn.attn_prefill(cache, torch.from_numpy(q).cuda(), torch.tensor([0, new], dtype=torch.int32, device="cuda"), pages,
                           torch.tensor([n], dtype=torch.int32, device="cuda")).double().cpu().numpy()
    before = pos < bad
    assert (np.abs(got - ref) <= prefill_bound(t, size, np.abs(v).max(), ref, False))[before].all()
    assert np.isnan(got[~before][:, :heads // kv]).all()  # a NaN key: every value of the heads that see it
    if t == F16:
        assert not np.isfinite(got[~before][:, heads // kv:, 5]).any() and np.isfinite(got[~before][:, heads // kv:, :5]).all()
    assert syn.device_status() == syn.OK


def test_prefill_matches_decode_and_batches(syn):
    """One new token gives what the one-token call gives; in deterministic mode a sequence's rows have
    the same bits alone and in a batch."""
    import torch
    rng = np.random.default_rng(15)
    heads, kv, dim, page = 8, 2, 128, 32
    lens, new = [700, 90, 2000], [200, 90, 1]
    cache, pages, _ = make_cache(syn, rng, F16, kv, dim, page, lens)
    q = torch.from_numpy(rng.standard_normal((sum(new), heads, dim)).astype(np.float16)).cuda()
    st = np.concatenate([[0], np.cumsum(new)])
    starts, ld = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (st, lens))
    old = syn.set_deterministic(True)
    try:
        both = syn.attn_prefill(cache, q, starts, pages, ld)
        for s in range(3):
            one = syn.attn_prefill(cache, q[st[s]:st[s + 1]].contiguous(), torch.tensor([0, new[s]], dtype=torch.int32, device="cuda"),
                                   pages[s:s + 1].contiguous(), ld[s:s + 1].contiguous())
            assert torch.equal(one, both[st[s]:st[s + 1]])
    finally:
        syn.set_deterministic(old)
    last = syn.attn_decode(cache, q[-1:].contiguous(), pages[2:].contiguous(), ld[2:].contiguous())
    assert (last[0] - both[-1]).abs().max().item() < 2.0 ** -11 * 6


def test_prefill_strides_streams_and_bad_pages(syn):
    import torch
    rng = np.random.default_rng(16)
    heads, kv, dim, page = 4, 2, 64, 16
    lens, new = [90, 200], [30, 77]
    cache, pages, seqs = make_cache(syn, rng, F16, kv, dim, page, lens, garbage=np.inf)
    both = torch.stack([cache.k, cache.v], 1)
    mixed = syn.KVCache(F16, kv, dim, page, both[:, 0], both[:, 1])
    wide = torch.randn((107, heads + 4, dim), device="cuda").half()
    wide_out = torch.zeros((107, heads + 8, dim), device="cuda")
    q = wide[:, 2:2 + heads]
    starts = torch.tensor([0, 30, 107], dtype=torch.int32, device="cuda")
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    rows = [np.arange(60, 90), np.arange(123, 200)]
    ref, size = reference(q.cpu().numpy(), seqs, rows, [np.zeros(30), np.zeros(77)], [0, 0], 0, dim ** -0.5, 0.0, None)
    vmax = max(np.abs(v).max() for _, v in seqs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    syn.attn_prefill(mixed, q, starts, pages, ld, wide_out[:, 3:3 + heads], stream=side)
    side.synchronize()
    got = wide_out[:, 3:3 + heads].double().cpu().numpy()
    assert (np.abs(got - ref) <= prefill_bound(F16, size, vmax, ref, False)).all()
    assert (wide_out[:, :3] == 0).all() and (wide_out[:, 3 + heads:] == 0).all()
    p = pages.clone()
    p[0, 2] = 10 ** 6
    got = syn.attn_prefill(mixed, q, starts, p, ld).double().cpu().numpy()
    assert syn.device_status(clear=True) == syn.ERR_BOUNDS
    assert (np.abs(got - ref) <= prefill_bound(F16, size, vmax, ref, False))[30:].all()
