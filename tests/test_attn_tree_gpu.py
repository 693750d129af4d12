"""syn_attn_tree on the GPU against its definition in 64 bits.  Tolerances as for the prefill form (p rounded
to fp16 once, Q8_0 keys and values as well, scores and sums in fp32): test_attn_gpu.prefill_bound."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_attn_gpu import F16, Q8_0, make_cache, prefill_bound  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def syn():
    import torch
    assert torch.cuda.is_available()
    from gguf_block_quantized_gb300 import syn
    yield syn
    torch.cuda.synchronize()
    assert syn.device_status() == syn.OK


def parents_of(rng, n, kind):
    i = np.arange(n)
    if kind == "chain":
        return i - 1
    if kind == "flat":
        return np.full(n, -1)
    if kind == "star":
        return np.where(i == 0, -1, 0)
    return np.array([rng.integers(-1, j) if j and rng.random() < 0.9 else -1 for j in i], np.int64).reshape(n)


def tree_attention(q, k, v, parents, first, prefix, window, scale, cap, slopes):
    """One sequence: (out, size), size the largest |v| times (1 + the largest sum |q_i k_i| scale + bias), per row."""
    n, H, D = q.shape
    ln, K = k.shape[:2]
    c = ln - n
    out, size = np.zeros((n, H, D)), np.zeros((n, H, 1))
    depth, chains = np.zeros(n, np.int64), []
    for i in range(n):
        a = int(parents[i])
        chains.append([i] if a < 0 else [i] + chains[a])
        depth[i] = len(chains[i]) - 1
    where = np.concatenate([np.arange(max(c, 0)), c + depth[max(-c, 0):]])
    for t in range(n):
        p = c + depth[t]
        seen = np.zeros(ln, bool)
        j = np.arange(max(c, 0))
        seen[:len(j)] = (j >= first[t]) & ((j < prefix) | (window == 0) | (p - j < window))
        for a in chains[t]:
            if c + a >= max(first[t], 0) and (window == 0 or depth[t] - depth[a] < window):
                seen[c + a] = True
        idx = np.nonzero(seen)[0]
        if idx.size == 0:
            continue
        far = np.abs(p - where[idx])
        for h in range(H):
            kk, vv = k[idx, h // (H // K)].astype(np.float64), v[idx, h // (H // K)].astype(np.float64)
            qq = q[t, h].astype(np.float64)
            s = kk @ qq * scale
            if cap > 0:
                s = cap * np.tanh(s / cap)
            if slopes is not None:
                s = s - float(slopes[h]) * far
            w = np.exp(s - s.max())
            out[t, h] = w @ vv / w.sum()
            size[t, h] = np.abs(vv).max() * (1 + (np.abs(kk) @ np.abs(qq)).max() * abs(scale)
                                             + (0 if slopes is None else float(slopes[h]) * far.max()))
    return out, size


def run(syn, t, heads, kv, dim, page, lens, new, seed, kind="any", cap=0.0, window=0, prefix=False, slopes=False, docs=False,
        scale=None, garbage=np.nan, dts=("float32", "float16"), check=True):
    import torch
    rng = np.random.default_rng(seed)
    cache, pages, seqs = make_cache(syn, rng, t, kv, dim, page, lens, garbage)
    q = rng.standard_normal((sum(new), heads, dim)).astype(np.float16)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    parents = [parents_of(rng, n, kind) for n in new]
    pre = np.array([rng.integers(0, n + 3) if prefix else 0 for n in lens], np.int32)
    first = [np.array([rng.integers(-1, max(1, ln - n) + (3 if i % 5 == 0 else 0)) if docs else 0 for i in range(n)], np.int32)
             for ln, n in zip(lens, new)]
    sl = (2.0 ** (-8.0 * (np.arange(heads) + 1) / heads)).astype(np.float32) if slopes else None
    scale = dim ** -0.5 if scale is None else scale
    outs, sizes, vmax = [], [], 0.0
    for s, (k, v) in enumerate(seqs):
        o, z = tree_attention(q[starts[s]:starts[s + 1]], k, v, parents[s], first[s], int(pre[s]), window, scale, cap, sl)
        outs.append(o)
        sizes.append(z)
        vmax = max(vmax, float(np.abs(v).max()) if len(v) else 0.0)
    ref, size = np.concatenate(outs), np.concatenate(sizes)
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    kw = {"cap": cap, "window": window, "scale": scale, "prefix": i32(pre) if prefix else None,
          "first": i32(np.concatenate(first)) if docs else None, "slopes": torch.from_numpy(sl).cuda() if slopes else None}
    args = cache, torch.from_numpy(q).cuda(), i32(starts), i32(np.concatenate(parents)), pages, i32(lens)
    for dt in dts:
        out = torch.full(q.shape, torch.nan, dtype=getattr(torch, dt), device="cuda")
        got = syn.attn_tree(*args, out, **kw).double().cpu().numpy()
        if check:
            err, bound = np.abs(got - ref), prefill_bound(t, size, vmax, ref, dt == "float16")
            assert (err <= bound).all(), (np.nanmax(err / np.maximum(bound, 1e-30)), np.argwhere(~(err <= bound))[:5])
    return args, kw, got, ref


LENS, NEW = [1, 9, 64, 128, 129, 200, 777, 0, 2000, 50], [1, 9, 1, 17, 30, 64, 5, 0, 26, 0]


@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("heads,kv,dim,page", [(8, 2, 64, 16), (4, 4, 32, 8), (12, 1, 96, 32), (8, 1, 128, 64), (20, 2, 128, 8),
                                               (3, 1, 160, 16), (16, 2, 256, 128), (24, 1, 64, 256), (40, 1, 256, 8)])
def test_shapes(syn, t, heads, kv, dim, page):
    run(syn, t, heads, kv, dim, page, LENS, NEW, [t, heads, dim])


OPTIONS = [dict(cap=5.0), dict(window=1), dict(window=4), dict(window=40), dict(prefix=True), dict(prefix=True, window=20), dict(slopes=True),
           dict(slopes=True, prefix=True, window=30), dict(docs=True), dict(docs=True, prefix=True), dict(docs=True, window=9, cap=2.0),
           dict(docs=True, prefix=True, window=50, slopes=True, cap=20.0), dict(scale=-0.1), dict(scale=0.0, slopes=True)]


@pytest.mark.parametrize("t,dim,page", [(F16, 64, 16), (F16, 128, 64), (Q8_0, 128, 32), (F16, 256, 8), (Q8_0, 256, 64), (Q8_0, 32, 8)])
@pytest.mark.parametrize("opt", OPTIONS, ids=lambda o: "-".join(o))
def test_options(syn, t, dim, page, opt):
    run(syn, t, 8, 2, dim, page, LENS, NEW, [t, dim, len(opt)], dts=("float32",), **opt)


@pytest.mark.parametrize("kind", ["chain", "flat", "star"])
@pytest.mark.parametrize("t,dim", [(F16, 128), (Q8_0, 64), (F16, 256)])
def test_kinds_of_trees(syn, kind, t, dim):
    run(syn, t, 4, 1, dim, 16, [300, 41, 130, 64], [200, 41, 129, 1], [7, dim], kind, dts=("float32",))
    run(syn, t, 4, 1, dim, 16, [300, 41, 130, 64], [200, 41, 129, 1], [8, dim], kind, dts=("float32",), slopes=True, window=7)


@pytest.mark.parametrize("t,dim", [(F16, 64), (F16, 128), (Q8_0, 128), (F16, 256), (Q8_0, 256)])
@pytest.mark.parametrize("heads,kv", [(8, 2), (4, 1), (24, 1)])
def test_long_contexts_are_split(syn, t, dim, heads, kv):
    run(syn, t, heads, kv, dim, 64, [9000, 30, 700], [14, 30, 1], [9, dim, heads], dts=("float32",))
    run(syn, t, heads, kv, dim, 64, [7003], [70], [10, dim, heads], dts=("float16",), slopes=True, cap=9.0, window=6000)


def test_many_sequences(syn):
    rng = np.random.default_rng(1)
    for n in (33, 300):
        lens = rng.integers(0, 150, n).tolist()
        new = [int(rng.integers(0, min(m, 12) + 1)) for m in lens]
        run(syn, F16, 4, 2, 64, 8, lens, new, [11, n], dts=("float32",))
        run(syn, Q8_0, 4, 2, 64, 8, lens, new, [12, n], dts=("float32",), docs=True, window=30)


def test_more_sequences_than_a_launch_takes(syn):
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 40, 1100).tolist()
    run(syn, F16, 2, 1, 32, 8, lens, [min(m, 3) for m in lens], 13, dts=("float32",))


@pytest.mark.parametrize("t", [F16, Q8_0])
def test_chains_are_the_prefill_form(syn, t):
    import torch
    lens, new = [700, 90, 33], [40, 90, 1]
    for opt in ({}, {"window": 25}, {"slopes": True}, {"cap": 4.0}):
        args, kw, got, _ = run(syn, t, 8, 2, 64, 16, lens, new, 14, "chain", dts=("float32",), **opt)
        cache, q, starts, _, pages, ln = args
        want = syn.attn_prefill(cache, q, starts, pages, ln, **kw).double().cpu().numpy()
        # (two results, each within a few roundings of p: 2^-11 of the largest value)
        assert np.abs(got - want).max() <= 2.0 ** -10 * 8 + 0
        torch.cuda.synchronize()


@pytest.mark.parametrize("t,dim", [(F16, 64), (Q8_0, 128), (F16, 256)])
def test_rows_beside_infinite_values(syn, t, dim):
    """What a node does not see does not reach it: siblings' and their descendants' rows hold infinities and NaN."""
    import torch
    rng = np.random.default_rng(15)
    lens, new, page = [150, 700], [24, 24], 16
    cache, pages, seqs = make_cache(syn, rng, t, 1, dim, page, lens)
    parents = np.concatenate([parents_of(rng, 24, "any")] * 2)
    q = rng.standard_normal((48, 4, dim)).astype(np.float16)
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    args = (i32([0, 24, 48]), i32(parents), pages, i32(lens))
    clean = syn.attn_tree(cache, torch.from_numpy(q).cuda(), *args).double().cpu().numpy()
    for bad in (0, 5, 23):
        k, v = cache.k.clone(), cache.v.clone()
        for s in (0, 1):
            row = lens[s] - 24 + bad
            pg, cell = int(pages[s, row // page]), row % page
            for pool, x in ((k, torch.inf), (v, torch.nan)):
                if t == F16:
                    pool[pg, 0, cell] = x
                else:
                    at = page * dim + cell * (dim // 16)
                    pool[pg, 0, at:at + dim // 16] = torch.tensor([0x00, 0x7E] * (dim // 32), dtype=torch.uint8, device="cuda")
        hurt = syn.KVCache(t, 1, dim, page, k, v)
        got = syn.attn_tree(hurt, torch.from_numpy(q).cuda(), *args).double().cpu().numpy()
        sees = np.zeros(48, bool)
        for s in (0, 1):
            for i in range(24):
                a = i
                while a >= 0:
                    sees[24 * s + i] |= a == bad
                    a = parents[24 * s + a]
        assert np.isfinite(got[~sees]).all() and not np.isfinite(got[sees]).all(axis=(1, 2)).any()
        assert np.abs(got - clean)[~sees].max() <= 2.0 ** -9 * np.abs(clean).max() * (4 if t == Q8_0 else 1)


def test_lengths_that_do_not_hold_the_drafts(syn):
    """lens below the number of new tokens: the tokens whose rows are before 0 are not there to be seen."""
    import torch
    rng = np.random.default_rng(16)
    for ln, n in ((0, 4), (3, 8), (1, 2)):
        cache, pages, seqs = make_cache(syn, rng, F16, 2, 64, 16, [max(ln, 1)])
        k, v = (x[:ln] for x in seqs[0])
        parents = parents_of(rng, n, "any")
        q = rng.standard_normal((n, 4, 64)).astype(np.float16)
        ref, size = tree_attention(q, k, v, parents, np.zeros(n), 0, 0, 0.125, 0.0, None)
        i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
        got = syn.attn_tree(cache, torch.from_numpy(q).cuda(), i32([0, n]), i32(parents), pages, i32([ln])).double().cpu().numpy()
        assert (np.abs(got - ref) <= prefill_bound(F16, size, 6.0, ref, False)).all()


def test_parents_that_do_not_go_down(syn):
    """A parent at or past its token is none, and reported; any negative number is none."""
    import torch
    args, kw, _, _ = run(syn, F16, 4, 2, 64, 16, [100, 60], [12, 9], 17, dts=("float32",))
    parents = args[3]
    for at, value, bad in ((3, 3, True), (5, 2 ** 31 - 1, True), (20, 8, True), (0, -(2 ** 31), False), (15, -9, False)):
        p = parents.clone()
        p[at] = value
        got = syn.attn_tree(*args[:3], p, *args[4:], **kw)
        assert syn.device_status() == (syn.ERR_BOUNDS if bad else syn.OK), (at, value)
        p[at] = -1
        assert torch.equal(got, syn.attn_tree(*args[:3], p, *args[4:], **kw))


def test_pages_that_nothing_sees(syn):
    """Ids of pages ahead of every window or past the length may be anything; a page that is seen may not."""
    import torch
    args, kw, got, _ = run(syn, F16, 4, 2, 64, 16, [500, 300], [10, 6], 18, dts=("float32",), window=40)
    pages = args[4].clone()
    pages[0, :27] = 10 ** 9  # rows 0 .. 431; node depths put windows at 490 + depth - 39 and up
    pages[1, 19:] = -3
    again = syn.attn_tree(*args[:4], pages, *args[5:], **kw).double().cpu().numpy()
    assert syn.device_status() == syn.OK and np.array_equal(got, again)
    pages[0, 30] = 10 ** 9
    syn.attn_tree(*args[:4], pages, *args[5:], **kw)
    assert syn.device_status() == syn.ERR_BOUNDS


@pytest.mark.parametrize("t,dim", [(F16, 128), (Q8_0, 64), (F16, 256)])
def test_deterministic(syn, t, dim):
    """A sequence's bits do not depend on the others, nor on the SMs."""
    import torch
    old = syn.set_deterministic(True)
    try:
        args, kw, _, _ = run(syn, t, 8, 2, dim, 16, [3000, 70, 400], [20, 70, 33], 19, dts=("float32",))
        cache, q, starts, parents, pages, lens = args
        want = syn.attn_tree(*args, **kw).clone()
        for s, (a, b) in enumerate(((0, 20), (20, 90), (90, 123))):
            one = syn.attn_tree(cache, q[a:b], torch.tensor([0, b - a], dtype=torch.int32, device="cuda"), parents[a:b].contiguous(),
                                pages[s:s + 1], lens[s:s + 1], **kw)
            assert torch.equal(one, want[a:b])
        lim = syn.set_sm_limit(3)
        try:
            assert torch.equal(syn.attn_tree(*args, **kw), want)
        finally:
            syn.set_sm_limit(lim)
    finally:
        syn.set_deterministic(old)


@pytest.mark.parametrize("limit", [1, 3, 17])
def test_sm_limit(syn, limit):
    old = syn.set_sm_limit(limit)
    try:
        for t, dim in ((F16, 128), (Q8_0, 128), (F16, 256)):
            run(syn, t, 8, 2, dim, 64, [4000, 200, 31, 900], [26, 130, 7, 1], 20, dts=("float32",))
    finally:
        syn.set_sm_limit(old)


def test_strided_rows_and_repeats(syn):
    """q and out in a fused buffer; the rows behind the last token stay; the same bits again."""
    import torch
    args, kw, got, _ = run(syn, F16, 4, 2, 64, 16, [900, 60], [13, 60], 21, dts=("float32",))
    cache, q, starts, parents, pages, lens = args
    wide = torch.full((80, 7, 64), 3.0, dtype=torch.float16, device="cuda")
    wide[:73, 1:5] = q
    out = torch.full((80, 6, 64), 7.0, device="cuda")
    for _ in range(3):
        syn.attn_tree(cache, wide[:73, 1:5], starts, parents, pages, lens, out[:73, 2:], **kw)
        assert np.array_equal(out[:73, 2:].double().cpu().numpy(), got)
    assert (out[73:] == 7).all() and (out[:, :2] == 7).all()


def test_captured(syn):
    """One graph, replayed as lengths, trees and tables change."""
    import torch
    rng = np.random.default_rng(22)
    lens, new = [3000, 80, 500], [20, 20, 20]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        args, kw, _, _ = run(syn, F16, 8, 2, 128, 16, lens, new, 22, dts=("float32",))
        cache, q, starts, parents, pages, ln = args
        out = torch.empty(q.shape, device="cuda")
        step = syn.prepare_attn_tree(*args, out, **kw)
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for cut in (0, 100, 2900):
            ln.copy_(torch.tensor([3000 - cut, 80 - cut // 50, 500 - cut // 10], dtype=torch.int32, device="cuda"))
            parents.copy_(torch.from_numpy(np.concatenate([parents_of(rng, 20, "any") for _ in new]).astype(np.int32)))
            graph.replay()
            got = out.clone()
            want = syn.attn_tree(*args, **kw)
            side.synchronize()
            assert torch.equal(got, want)


def test_calls_of_nothing(syn):
    import torch
    cache = syn.KVCache.empty(F16, 2, 64, 16, 4)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.zeros((0, 4, 64), dtype=torch.float16, device="cuda")
    assert syn.attn_tree(cache, q, i32(1), i32(0), i32(0, 3), i32(0)).shape == q.shape
    assert syn.attn_tree(cache, q, i32(3), i32(0), i32(2, 3), i32(2)).shape == q.shape
