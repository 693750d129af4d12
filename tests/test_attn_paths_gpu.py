"""The paged-cache operators on the GPU where they choose between ways: a Q8_0 cache expanded ahead of
the prefill, many sequences, both forms of the cap, graphs, and pools past 32-bit offsets."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_ref  # noqa: E402
from test_attn_gpu import F16, Q8_0, make_cache, prefill_bound, decode_bound, reference, run_prefill, syn  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def launches(syn, call):
    n = syn.launch_count()
    call()
    return syn.launch_count() - n


# ---- a Q8_0 cache expanded ahead of the kernel ---------------------------------------------
# (from 8 tiles of 256 (token, head) rows a sequence with a cap or slopes and heads up to 128, else 32)

@pytest.mark.parametrize("heads,kv,dim,page,new,opt", [
    (8, 1, 64, 16, [260, 300], {"slopes": True}),
    (16, 2, 128, 8, [260, 257], {"cap": 5.0}),
    (24, 1, 96, 64, [200, 0], {"slopes": True, "docs": True}),
    (8, 1, 128, 256, [270], {"slopes": True, "window": 40}),
    (8, 1, 64, 32, [270], {"cap": 20.0, "window": 150, "prefix": True}),
    (32, 1, 64, 16, [270], {}),
    (32, 1, 256, 16, [270], {"window": 60}),
    (32, 1, 160, 32, [260], {"docs": True}),
])
def test_expanded_cache(syn, heads, kv, dim, page, new, opt):
    lens = [n + 41 * i + 7 for i, n in enumerate(new)]
    run_prefill(syn, Q8_0, heads, kv, dim, page, lens, new, 21, scale=0.1, **opt)


def test_cache_is_expanded_from_the_stated_size_on(syn):
    import torch
    rng = np.random.default_rng(30)
    cache, pages, _ = make_cache(syn, rng, Q8_0, 1, 64, 16, [400])
    ld = torch.tensor([400], dtype=torch.int32, device="cuda")
    for n, opt, want in ((255, {"cap": 9.0}, 1), (256, {"cap": 9.0}, 2), (257, {}, 1)):
        q = torch.zeros((n, 8, 64), dtype=torch.float16, device="cuda")
        call = syn.prepare_attn_prefill(cache, q, torch.tensor([0, n], dtype=torch.int32, device="cuda"), pages, ld, **opt)
        assert launches(syn, call) == want
        old = syn.set_deterministic(True)
        assert launches(syn, call) == 1
        syn.set_deterministic(old)


@pytest.mark.parametrize("ahead", [False, True])
def test_cached_values_past_fp16(syn, ahead):
    """A Q8_0 cache holds values that fp16 does not (a scale above 516): rows that see one are right."""
    import torch
    rng = np.random.default_rng(31)
    heads, dim, page, n, new = 8, 64, 16, 330, 260 if ahead else 60
    cache, pages, seqs = make_cache(syn, rng, Q8_0, 1, dim, page, [n])
    (k, v), j = seqs[0], n - 30
    pg, cell = int(pages[0, j // page]), j % page
    codes = cache.v[pg, 0, :page * dim].view(torch.int8).view(page, dim)[cell, :32].double().cpu().numpy()
    at = page * dim + cell * dim // 16
    cache.v[pg, 0, at:at + 2] = torch.from_numpy(np.array([1500.0], np.float16).view(np.uint8)).cuda()
    v[j, 0, :32] = codes * 1500.0
    q = rng.standard_normal((new, heads, dim)).astype(np.float16)
    slopes = (2.0 ** -np.arange(1, heads + 1)).astype(np.float32)
    call = syn.prepare_attn_prefill(cache, torch.from_numpy(q).cuda(), torch.tensor([0, new], dtype=torch.int32, device="cuda"), pages,
                                    torch.tensor([n], dtype=torch.int32, device="cuda"), slopes=torch.from_numpy(slopes).cuda())
    assert launches(syn, call) == (2 if ahead else 1)
    got = call().double().cpu().numpy()
    pos = np.arange(n - new, n)
    ref, size = attn_ref.attention(q, k, v, pos, np.zeros(new), 0, 0, dim ** -0.5, 0.0, slopes)
    seen = np.where(pos >= j, np.abs(v).max(), np.abs(np.delete(v, j, 0)).max())[:, None, None]
    assert (np.abs(got - ref) <= prefill_bound(Q8_0, size, seen, ref, False)).all()
    one = syn.attn_decode(cache, torch.from_numpy(q[-1:]).cuda(), pages, torch.tensor([n], dtype=torch.int32, device="cuda"),
                          slopes=torch.from_numpy(slopes).cuda()).double().cpu().numpy()
    assert (np.abs(one[0] - ref[-1]) <= decode_bound(size[-1], ref[-1], False)).all()
    assert syn.device_status() == syn.OK


def test_expanded_cache_nonfinite_and_bad_pages(syn):
    """What a row does not see does not reach it: a NaN key seen by the last rows alone, and a page
    outside the pool that only the other sequence has."""
    import torch
    rng = np.random.default_rng(32)
    heads, dim, page, lens, new = 8, 64, 16, [300, 310], [260, 260]
    cache, pages, seqs = make_cache(syn, rng, Q8_0, 1, dim, page, lens)
    j = 290
    pg, cell = int(pages[0, j // page]), j % page
    at = page * dim + cell * dim // 16
    cache.k[pg, 0, at:at + 2] = torch.tensor([0, 0x7E], dtype=torch.uint8, device="cuda")
    q = rng.standard_normal((520, heads, dim)).astype(np.float16)
    qd = torch.from_numpy(q).cuda()
    starts = torch.tensor([0, 260, 520], dtype=torch.int32, device="cuda")
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    rows = [np.arange(n - m, n) for n, m in zip(lens, new)]
    cap = 30.0
    ref, size = reference(q, seqs, rows, [np.zeros(260)] * 2, [0, 0], 0, dim ** -0.5, cap, None)
    vmax = max(np.abs(v).max() for _, v in seqs)
    good = np.concatenate([rows[0] < j, np.ones(260, bool)])
    got = syn.attn_prefill(cache, qd, starts, pages, ld, cap=cap).double().cpu().numpy()
    assert (np.abs(got - ref) <= prefill_bound(Q8_0, size, vmax, ref, False))[good].all() and np.isnan(got[~good]).all()
    assert syn.device_status() == syn.OK
    p = pages.clone()
    p[1, 3] = -7
    got = syn.attn_prefill(cache, qd, starts, p, ld, cap=cap).double().cpu().numpy()
    assert syn.device_status(clear=True) == syn.ERR_BOUNDS
    assert (np.abs(got - ref) <= prefill_bound(Q8_0, size, vmax, ref, False))[:260][good[:260]].all()


# ---- how decode deals its work --------------------------------------------------------------
# (ranges over items of unlike lengths, each with some steps for its ends; blocks of steps for few long ones)

@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("heads,kv,dim,lens,limit", [
    (8, 2, 64, [3, 40, 0, 64, 65, 2, 700, 1, 1, 1, 128, 30, 5000, 17], 1),
    (8, 2, 64, [3, 40, 0, 64, 65, 2, 700, 1, 1, 1, 128, 30, 5000, 17] * 3, 7),
    (4, 4, 128, [40] * 70 + [9000] + [0] * 5 + [33] * 60, 0),
    (24, 1, 128, [20000], 0),
    (16, 2, 96, [12000, 1, 300], 0),
    (8, 1, 256, [5000, 7000], 16),
])
def test_decode_ranges(syn, t, heads, kv, dim, lens, limit):
    import torch
    rng = np.random.default_rng([t, dim, limit])
    cache, pages, seqs = make_cache(syn, rng, t, kv, dim, 32, lens)
    q = rng.standard_normal((len(lens), heads, dim)).astype(np.float16)
    old = syn.set_sm_limit(limit)
    try:
        got = syn.attn_decode(cache, torch.from_numpy(q).cuda(), pages, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    finally:
        syn.set_sm_limit(old)
    got = got.double().cpu().numpy()
    ref, size = reference(q, seqs, [np.array([n - 1]) for n in lens], [np.zeros(1)] * len(lens), [0] * len(lens), 0, dim ** -0.5, 0.0, None)
    assert (np.abs(got - ref) <= decode_bound(size, ref, False)).all()
    assert syn.device_status() == syn.OK


@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("heads,kv,dim,lens,new,dtype", [
    (24, 1, 128, [2000], [9], "float16"), (6, 2, 64, [4096, 1000], [64, 3], "float32"), (5, 1, 256, [3000], [30], "float16"),
    (3, 1, 96, [5000], [7], "float32")])
def test_prefill_parts_and_joins(syn, t, heads, kv, dim, lens, new, dtype):
    run_prefill(syn, t, heads, kv, dim, 16, lens, new, 25, dts=(dtype,))


# ---- many sequences, both forms of the cap, empty rows -------------------------------------

@pytest.mark.parametrize("n_seq", [33, 1030])
def test_prefill_many_sequences(syn, n_seq):
    rng = np.random.default_rng(n_seq)
    new = rng.integers(0, 4, n_seq).tolist()
    lens = [m + int(rng.integers(0, 9)) for m in new]
    new[5], lens[5] = 150, 400
    run_prefill(syn, F16, 2, 1, 64, 8, lens, new, 23, dts=("float32",))


@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("cap,qscale", [(50.0, 1.0), (1.0, 1.0), (2.0, 8.0), (1000.0, 0.01)])
def test_prefill_cap_small_and_large_scores(syn, t, cap, qscale):
    run_prefill(syn, t, 4, 1, 128, 16, [200, 140], [90, 140], 24, qscale=qscale, cap=cap)


@pytest.mark.parametrize("t", [F16, Q8_0])
def test_tokens_before_the_first_position(syn, t):
    """A sequence of fewer rows than new tokens: the tokens ahead of position 0 see nothing and give zeros."""
    import torch
    rng = np.random.default_rng(33)
    lens, new = [3, 0, 40], [5, 4, 2]
    cache, pages, seqs = make_cache(syn, rng, t, 2, 64, 8, lens)
    q = rng.standard_normal((11, 4, 64)).astype(np.float16)
    starts = torch.tensor([0, 5, 9, 11], dtype=torch.int32, device="cuda")
    got = syn.attn_prefill(cache, torch.from_numpy(q).cuda(), starts, pages, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    got = got.double().cpu().numpy()
    ref, size = reference(q, seqs, [np.arange(n - m, n) for n, m in zip(lens, new)], [np.zeros(m) for m in new], [0] * 3, 0, 0.125, 0.0, None)
    assert (ref[:2] == 0).all() and (got[:2] == 0).all() and (got[5:9] == 0).all()
    vmax = max(np.abs(v).max() for _, v in seqs if v.size)
    assert (np.abs(got - ref) <= prefill_bound(t, size, vmax, ref, False)).all()


# ---- graphs --------------------------------------------------------------------------------

@pytest.mark.parametrize("t,slopes", [(F16, False), (Q8_0, False), (Q8_0, True)])
def test_append_and_prefill_in_a_graph(syn, t, slopes):
    """A graph captured at short lengths, replayed on longer ones and other slots, also after a call
    that needed a larger workspace."""
    import torch
    rng = np.random.default_rng(34)
    heads, kv, dim, page, n = 8, 1, 64, 16, 260
    cache = syn.KVCache.empty(t, kv, dim, page, 40)
    x = torch.from_numpy(rng.standard_normal((n, heads + 2 * kv, dim)).astype(np.float32)).cuda()
    rope = syn.Rope(dim)
    pages = torch.randperm(40, device="cuda").to(torch.int32).view(1, 40)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    q_rot = torch.zeros((n, heads, dim), dtype=torch.float16, device="cuda")
    out = torch.zeros((n, heads, dim), device="cuda")
    opt = {"slopes": torch.full((heads,), 0.02, device="cuda")} if slopes else {}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = syn.prepare_kv_append(cache, rope, x[:, heads:heads + kv], x[:, heads + kv:], pos, slots, q=x[:, :heads], q_out=q_rot, stream=side)
    p = syn.prepare_attn_prefill(cache, q_rot, starts, pages, lens, out, stream=side, **opt)
    a()
    p()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        a()
        p()
    big = syn.KVCache.empty(t, kv, dim, page, 4000)
    more = syn.prepare_attn_prefill(big, torch.zeros((n, heads, dim), dtype=torch.float16, device="cuda"), starts,
                                    torch.arange(4000, dtype=torch.int32, device="cuda").view(1, -1),
                                    torch.tensor([50000], dtype=torch.int32, device="cuda"), stream=side, **opt)
    torch.cuda.synchronize()
    more()
    torch.cuda.synchronize()
    row = torch.arange(n, device="cuda") + 101
    cache.k.random_(0, 100) if t == Q8_0 else cache.k.normal_()
    cache.v.random_(0, 100) if t == Q8_0 else cache.v.normal_()
    if t == Q8_0:  # (the scales: 2^-4)
        for pool in (cache.k, cache.v):
            pool[:, :, page * dim:].view(torch.float16).fill_(0.0625)
    slots.copy_(pages[0, row // page].long() * page + row % page)
    lens.fill_(101 + n)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    got = out.clone()
    want_q = syn.kv_append(cache, rope, x[:, heads:heads + kv].contiguous(), x[:, heads + kv:].contiguous(), pos, slots,
                           q=x[:, :heads].contiguous())
    assert torch.equal(want_q, q_rot)
    every = torch.arange(101 + n, device="cuda")
    k, v = syn.kv_read(cache, pages[0, every // page].long() * page + every % page)
    k, v = k.double().cpu().numpy(), v.double().cpu().numpy()
    sl = np.full(heads, np.float32(0.02)) if slopes else None
    ref, size = attn_ref.attention(want_q.cpu().numpy(), k, v, np.arange(101, 101 + n), np.zeros(n), 0, 0, dim ** -0.5, 0.0, sl)
    assert (np.abs(got.double().cpu().numpy() - ref) <= prefill_bound(t, size, np.abs(v).max(), ref, False)).all()
    assert syn.device_status() == syn.OK


# ---- pools past 32-bit offsets -------------------------------------------------------------

@pytest.mark.parametrize("t", [F16, Q8_0])
def test_pools_past_32_bit_offsets(syn, t):
    """The last pages of pools of more than 2^32 bytes give the bits that the first pages of small ones give."""
    import torch
    kv, heads, dim, page, n = 8, 16, 128, 64, 700
    n_pages = 36000 if t == F16 else 66000
    big, small = syn.KVCache.empty(t, kv, dim, page, n_pages), syn.KVCache.empty(t, kv, dim, page, 11)
    assert n_pages * big.n_kv_heads * syn.syn_kv_tile_bytes(t, dim, page) > 2 ** 32
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((n, heads + 2 * kv, dim), device="cuda", generator=gen)
    rope, pos = syn.Rope(dim), torch.arange(n, dtype=torch.int32, device="cuda")
    results = []
    for c, at in ((small, 0), (big, n_pages - 11)):
        slots = torch.arange(n, device="cuda") + at * page
        q = syn.kv_append(c, rope, x[:, heads:heads + kv], x[:, heads + kv:], pos, slots, q=x[:, :heads])
        k, v = syn.kv_read(c, slots)
        pages = (torch.arange(11, device="cuda") + at).to(torch.int32).view(1, 11)
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        one = syn.attn_decode(c, q[-1:], pages, lens)
        many = syn.attn_prefill(c, q[-300:], torch.tensor([0, 300], dtype=torch.int32, device="cuda"), pages, lens)
        results.append((q, k, v, one, many))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert results[0][1].abs().max() > 0 and syn.device_status() == syn.OK
