"""The pages of a cache (syn_kv_fork, _extend, _compact, _trim, _copy) on the GPU against plain forms: every
result is a whole number or a copied row, so all have to be equal."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import pages_ref  # noqa: E402

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


def dev(x, dtype=None):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype or np.int32)).cuda()


def make_cache(syn, t, kv, dim, page, n_pages, seed=0, strided=False):
    """A cache of random bits; strided: both pools in one allocation."""
    import torch
    shape = (kv, page, dim) if t == F16 else (kv, page * dim // 16 * 17)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    raw = torch.randint(0, 256, (n_pages, 2, *shape[:-1], shape[-1] * (2 if t == F16 else 1)), dtype=torch.uint8, device="cuda",
                        generator=gen)
    both = raw.view(torch.float16) if t == F16 else raw
    k, v = (both[:, 0], both[:, 1]) if strided else (both[:, 0].contiguous(), both[:, 1].contiguous())
    return syn.KVCache(t, kv, dim, page, k, v)


def planes(cache, dim, page):
    """The pools' bits as numpy [plane][pages][kv][page][bytes of a row]."""
    import torch
    out = []
    for pool in (cache.k, cache.v):
        if cache.type == F16:
            out.append(pool.contiguous().view(torch.uint8).cpu().numpy())
        else:
            x = pool.cpu().numpy()
            out.append(x[..., :page * dim].reshape(*x.shape[:2], page, dim))
            out.append(x[..., page * dim:].reshape(*x.shape[:2], page, dim // 16))
    return [p.copy() for p in out]


def counts(n_pages, *tables):
    return np.bincount(np.concatenate([t[t >= 0].ravel() for t in tables] + [np.zeros(0, np.int64)]).astype(np.int64), minlength=n_pages)


def same(got, want, what):
    assert np.array_equal(got.cpu().numpy(), want), what


@pytest.mark.parametrize("page", [8, 64])
@pytest.mark.parametrize("seqs,width,n_pages", [(1, 1, 3), (7, 5, 20), (64, 12, 300), (1100, 4, 2500)])
def test_a_run_of_calls(syn, page, seqs, width, n_pages):
    """Sequences grown, forked and cut at random, pages short at times: tables, counts, lengths, slots
    and the rows of copied pages after every call."""
    import torch
    rng = np.random.default_rng([page, seqs])
    cache = make_cache(syn, F16, 2, 32, page, n_pages)
    refs, pages, lens = np.zeros(n_pages, np.int32), np.full((seqs, width), -1, np.int32), np.zeros(seqs, np.int32)
    d_refs, d_pages, d_lens = dev(refs), dev(pages), dev(lens)
    for step in range(14):
        most = rng.choice([1, 3, page + 2, 2 * page])
        new = rng.integers(0, most + 1, seqs) if step % 3 else np.ones(seqs, np.int64)
        starts = np.concatenate([[0], np.cumsum(new)])
        bits = planes(cache, 32, page)
        free = (refs == 0).sum()
        refs, pages, lens, slots, moves = pages_ref.extend(refs, pages, lens, new, page)
        for to in bits:
            for a, b, n in moves.values():
                to[b, :, :n] = to[a, :, :n]
        if step % 3 == 0:
            got_lens, got_slots = syn.kv_extend(cache, d_refs, d_pages, d_lens)
        else:
            got_lens, got_slots = syn.kv_extend(cache, d_refs, d_pages, d_lens, starts=dev(starts), n_tok=int(starts[-1]))
        assert got_lens is d_lens
        same(d_pages, pages, (step, free))
        same(d_refs, refs, step)
        same(d_lens, lens, step)
        same(got_slots, slots, step)
        for x, y in zip(planes(cache, 32, page), bits):
            assert np.array_equal(x, y), step
        assert np.array_equal(refs, counts(n_pages, pages))
        if step % 4 == 3:  # cut some, drop some
            lens = np.where(rng.random(seqs) < 0.5, rng.integers(0, lens + 1), lens).astype(np.int32)
            lens[rng.random(seqs) < 0.2] = 0
            d_lens.copy_(dev(lens))
            refs, pages = pages_ref.trim(refs, pages, lens, page)
            syn.kv_trim(cache, d_refs, d_pages, d_lens)
        else:
            source = rng.integers(-1, seqs, seqs).astype(np.int32)
            if step % 2:
                source = np.where(rng.random(seqs) < 0.7, np.arange(seqs), source).astype(np.int32)
            refs, new_pages, new_lens = pages_ref.fork(refs, pages, lens, page, source)
            got_pages, got_lens = syn.kv_fork(cache, d_refs, dev(source), d_pages, d_lens)
            same(d_refs, refs, step)
            refs, pages = pages_ref.trim(refs, pages, np.zeros(seqs), page)
            syn.kv_trim(cache, d_refs, d_pages, torch.zeros_like(d_lens))
            assert (pages == -1).all()
            same(d_pages, pages, step)
            pages, lens, d_pages, d_lens = new_pages, new_lens, got_pages, got_lens.clone()
        same(d_pages, pages, step)
        same(d_refs, refs, step)
        same(d_lens, lens, step)
        assert np.array_equal(refs, counts(n_pages, pages))


@pytest.mark.parametrize("t,kv,dim,strided", [(F16, 3, 96, False), (F16, 1, 256, True), (Q8_0, 2, 32, False), (Q8_0, 5, 96, True),
                                              (Q8_0, 1, 256, False)])
def test_a_shared_page_is_copied(syn, t, kv, dim, strided):
    """Rows of every tile, codes and scales; the rest of the new page stays as it was."""
    page, n_pages = 32, 9
    cache = make_cache(syn, t, kv, dim, page, n_pages, 1, strided)
    pages = np.array([[4, 2], [4, 2], [4, 7], [-1, -1]], np.int32)
    refs = counts(n_pages, pages).astype(np.int32)
    lens = np.array([45, 33, 64, 0], np.int32)
    new = [3, 1, 0, 2]
    bits = planes(cache, dim, page)
    want = pages_ref.extend(refs, pages, lens, new, page)
    for to in bits:
        for a, b, n in want[4].values():
            to[b, :, :n] = to[a, :, :n]
    d = dev(refs), dev(pages), dev(lens)
    got = syn.kv_extend(cache, *d, starts=dev([0, 3, 4, 4, 6]), n_tok=6)
    for x, y, what in ((d[0], want[0], "refs"), (d[1], want[1], "pages"), (got[0], want[2], "lens"), (got[1], want[3], "slots")):
        same(x, y, what)
    # both holders of page 2 write: the first moves, the second keeps it
    assert want[1][1, 1] == 2 and want[1][0, 1] != 2
    for x, y in zip(planes(cache, dim, page), bits):
        assert np.array_equal(x, y)


def test_many_pages_and_columns(syn):
    """Free pages far up a large pool, one sequence's new rows over many columns."""
    import torch
    page, n_pages, width = 8, 70001, 3000
    pools = [torch.zeros((n_pages, 1, page, 32), dtype=torch.float16, device="cuda") for _ in range(2)]
    cache = syn.KVCache(F16, 1, 32, page, *pools)
    rng = np.random.default_rng(2)
    refs = (rng.random(n_pages) < 0.95).astype(np.int32)
    refs[:60000] = 1
    pages = np.full((2, width), -1, np.int32)
    new = [8 * 200 + 3, 5]
    want = pages_ref.extend(refs, pages, np.zeros(2, np.int32), new, page)
    d = dev(refs), dev(pages), dev(np.zeros(2))
    got = syn.kv_extend(cache, *d, starts=dev([0, new[0], sum(new)]), n_tok=sum(new))
    for x, y, what in ((d[0], want[0], "refs"), (d[1], want[1], "pages"), (got[0], want[2], "lens"), (got[1], want[3], "slots")):
        same(x, y, what)
    # a pool that is full: nothing changes
    d[0].clamp_(min=1)
    before = [x.clone() for x in d]
    got = syn.kv_extend(cache, *d, starts=dev([0, 5, 5000]), n_tok=5000)
    assert all(torch.equal(x, y) for x, y in zip(d[:2], before[:2])) and (got[1] == -1)[5:].all()


@pytest.mark.parametrize("t,kv,dim,page,strided", [(F16, 2, 32, 8, False), (F16, 8, 128, 64, True), (Q8_0, 2, 96, 16, False),
                                                   (Q8_0, 1, 256, 128, True), (F16, 1, 160, 256, False), (Q8_0, 4, 32, 8, False)])
def test_compact(syn, t, kv, dim, page, strided):
    rng = np.random.default_rng([t, dim])
    lens = [0, 1, 7, 40, 300, 2500, 6 * page]
    need = [-(-n // page) for n in lens]
    n_pages, width = sum(need) + 2, max(need) + 1
    cache = make_cache(syn, t, kv, dim, page, n_pages, 3, strided)
    order = rng.permutation(n_pages)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = order[at:at + m]
        at += m
    for share, based in ((0.5, True), (0.02, False), (1.0, False), (0.97, True), (0.0, True)):
        base = np.array([rng.integers(0, n + 1) if based else 0 for n in lens], np.int32)
        rows = [np.sort(rng.permutation(n - b)[:int(round(share * (n - b)))]) for n, b in zip(lens, base)]
        starts = np.concatenate([[0], np.cumsum([len(r) for r in rows])])
        want = planes(cache, dim, page)
        for x in want:
            for s, r in enumerate(rows):
                to, come = base[s] + np.arange(len(r)), base[s] + r
                x[table[s, to // page], :, to % page] = x[table[s, come // page], :, come % page]
        got = syn.kv_compact(cache, dev(counts(n_pages, table)), dev(table), dev(base), dev(starts), dev(np.concatenate(rows)))
        same(got, base + np.diff(starts), "lengths")
        for x, y in zip(planes(cache, dim, page), want):
            assert np.array_equal(x, y), (share, based)


def test_compact_of_one_long_sequence(syn):
    import torch
    page, n_pages = 16, 2500
    for t in (F16, Q8_0):
        cache = make_cache(syn, t, 1, 64, page, n_pages, 4)
        rng = np.random.default_rng(6)
        table = rng.permutation(n_pages)[None].astype(np.int32)
        rows = np.sort(rng.permutation(page * n_pages)[:30011])
        want = planes(cache, 64, page)
        to = np.arange(len(rows))
        for x in want:
            x[table[0, to // page], :, to % page] = x[table[0, rows // page], :, rows % page]
        for limit in (0,):
            old = syn.set_sm_limit(limit)
            try:
                syn.kv_compact(cache, None, dev(table), dev([0]), dev([0, len(rows)]), dev(rows))
            finally:
                syn.set_sm_limit(old)
        for x, y in zip(planes(cache, 64, page), want):
            assert np.array_equal(x, y)


def test_compact_leaves_shared_pages_alone(syn):
    page, n_pages = 8, 6
    cache = make_cache(syn, F16, 1, 32, page, n_pages, 5)
    table = np.array([[1, 3], [1, 4]], np.int32)
    before = planes(cache, 32, page)
    syn.kv_compact(cache, dev(counts(n_pages, table)), dev(table), dev([0, 0]), dev([0, 2, 2]), dev([0, 9]))
    assert syn.device_status() == syn.ERR_BOUNDS
    for x, y in zip(planes(cache, 32, page), before):
        assert np.array_equal(x, y)
    # rows out of order or outside the table are skipped
    for rows, base in (([3, 2], 0), ([0, 16], 0), ([-1, 2], 0), ([1, 2], 30)):
        syn.kv_compact(cache, None, dev(table[:1]), dev([base]), dev([0, 2]), dev(rows))
        assert syn.device_status() == syn.ERR_BOUNDS, rows


@pytest.mark.parametrize("t,kv,dim,page", [(F16, 2, 32, 8), (F16, 8, 128, 64), (Q8_0, 3, 96, 8), (Q8_0, 1, 256, 256)])
def test_copy(syn, t, kv, dim, page):
    import torch
    a, b = make_cache(syn, t, kv, dim, page, 11, 6, True), make_cache(syn, t, kv, dim, page, 7, 7)
    want = planes(b, dim, page)
    src, dst = [3, 10, 0, 3], [6, 0, 2, 5]
    for x, y in zip(planes(a, dim, page), want):
        y[dst] = x[src]
    syn.kv_copy(a, b, dev(src), dev(dst))
    for x, y in zip(planes(b, dim, page), want):
        assert np.array_equal(x, y)
    for x, y in zip(planes(a, dim, page), want):
        y[[1, 4]] = x[[8, 9]]
    syn.kv_copy(a, b, dev([8, 11, 9, -1, 2]), dev([1, 3, 4, 3, 7]))  # two ids of one pool, one of the other: skipped
    assert syn.device_status() == syn.ERR_BOUNDS
    for x, y in zip(planes(b, dim, page), want):
        assert np.array_equal(x, y)


def test_bad_tables(syn):
    """Ids outside the pool count as no page, pages given back twice stay free; all are reported."""
    import torch
    cache = make_cache(syn, F16, 1, 32, 8, 6, 8)
    refs, pages, lens = dev([1, 1, 0, 0, 0, 0]), dev([[0, 99], [1, -7]]), dev([16, 8])
    got, got_lens = syn.kv_fork(cache, refs, dev([0, 1, 2]), pages, lens)
    assert syn.device_status() == syn.ERR_BOUNDS
    assert got.tolist() == [[0, -1], [1, -1], [-1, -1]] and got_lens.tolist() == [16, 8, 0] and refs.tolist() == [2, 2, 0, 0, 0, 0]
    lens = dev([8, 8])
    _, slots = syn.kv_extend(cache, refs, pages, lens)
    assert syn.device_status() == syn.ERR_BOUNDS
    assert pages.tolist() == [[0, 2], [1, 3]] and slots.tolist() == [16, 24] and lens.tolist() == [9, 9]
    table = dev([[5, 77], [4, -1]])
    syn.kv_trim(cache, refs, table, dev([0, -3]))
    assert syn.device_status() == syn.ERR_BOUNDS
    assert refs.tolist() == [2, 2, 1, 1, 0, 0] and (table == -1).all()
    # starts that run backwards, or past the call's rows, are no rows
    lens = dev([9, 9])
    _, slots = syn.kv_extend(cache, refs, pages, lens, starts=dev([2, 0, 9]), n_tok=3)
    assert lens.tolist() == [9, 9] and (slots == -1).all()
    assert syn.device_status() == syn.OK
    # a table without room, a length past it
    lens = dev([9, 100])
    syn.kv_extend(cache, refs, pages, lens, starts=dev([0, 8, 9]), n_tok=9)
    assert lens.tolist() == [9, 16] and refs.tolist() == [2, 2, 1, 1, 0, 0]


def test_captured(syn):
    """A step's calls in one graph, replayed as lengths and tables change."""
    import torch
    page, n_pages, seqs = 8, 40, 3
    cache = make_cache(syn, F16, 2, 32, page, n_pages, 9)
    refs, pages, lens = np.zeros(n_pages, np.int32), np.full((seqs, 6), -1, np.int32), np.zeros(seqs, np.int32)
    d_refs, d_pages, d_lens, d_base = dev(refs), dev(pages), dev(lens), dev(lens)
    starts, keep = dev([0, 4, 8, 12]), dev([0, 2, 4, 6])
    rows, long = dev([0, 2, 0, 3, 0, 1]), torch.empty_like(d_lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        steps = [syn.prepare_kv_extend(cache, d_refs, d_pages, d_base, long, starts=starts, n_tok=12),
                 syn.prepare_kv_compact(cache, d_refs, d_pages, d_base, keep, rows, d_lens),
                 syn.prepare_kv_trim(cache, d_refs, d_pages, d_lens)]
        syn.kv_extend(cache, d_refs.clone(), d_pages.clone(), d_base.clone(), starts=starts, n_tok=12)  # the workspace
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for step in steps:
                step()
            d_base.copy_(d_lens)
        for i in range(9):
            graph.replay()
            refs, pages, lens, _, _ = pages_ref.extend(refs, pages, lens, [4] * seqs, page)
            lens = lens - 2
            refs, pages = pages_ref.trim(refs, pages, lens, page)
            side.synchronize()
            same(d_pages, pages, i)
            same(d_refs, refs, i)
            same(d_lens, lens, i)


@pytest.mark.parametrize("t,kv,dim,page", [(F16, 1, 64, 8), (F16, 2, 160, 64), (Q8_0, 3, 96, 16), (Q8_0, 2, 128, 32), (Q8_0, 1, 64, 8),
                                           (F16, 9, 256, 16)])
def test_compact_of_long_lists(syn, t, kv, dim, page):
    """Lists that many CTAs share: nearly all rows kept, few, runs that stay, sequences of one row between long ones."""
    rng = np.random.default_rng([t, kv, dim])
    lens = [1, 9000, 3, 0, 4100, 1, 300, 5000]
    need = [-(-n // page) for n in lens]
    n_pages, width = sum(need), max(need)
    cache = make_cache(syn, t, kv, dim, page, n_pages, 11)
    table = np.full((len(lens), width), -1, np.int32)
    order, at = rng.permutation(n_pages), 0
    for s, m in enumerate(need):
        table[s, :m] = order[at:at + m]
        at += m
    refs = counts(n_pages, table)
    for kind in ("most", "half", "gap", "late"):
        rows = []
        for n in lens:
            if kind == "most":
                keep = rng.random(n) < 0.999
            elif kind == "half":
                keep = rng.random(n) < 0.5
            elif kind == "gap":  # all but the first: every row moves down by one
                keep = np.arange(n) != 0
            else:  # the first stay where they are
                keep = (np.arange(n) < n // 2) | (rng.random(n) < 0.3)
            rows.append(np.nonzero(keep)[0])
        starts = np.concatenate([[0], np.cumsum([len(r) for r in rows])])
        assert starts[-1] > 4096
        want = planes(cache, dim, page)
        for x in want:
            for s, r in enumerate(rows):
                to = np.arange(len(r))
                x[table[s, to // page], :, to % page] = x[table[s, r // page], :, r % page]
        got = syn.kv_compact(cache, dev(refs), dev(table), dev(np.zeros(len(lens))), dev(starts), dev(np.concatenate(rows)))
        same(got, np.diff(starts), kind)
        for x, y in zip(planes(cache, dim, page), want):
            assert np.array_equal(x, y), kind
    # again with few SMs, and bad rows in the middle
    old = syn.set_sm_limit(1)
    try:
        want = planes(cache, dim, page)
        rows = np.arange(1, 5000)
        rows[3000] = 1
        bad = rows.copy()
        ok = np.ones(len(rows), bool)
        ok[3000] = False
        for x in want:
            to = np.arange(len(rows))[ok]
            x[table[1, to // page], :, to % page] = x[table[1, rows[ok] // page], :, rows[ok] % page]
        syn.kv_compact(cache, dev(refs), dev(table[1:2]), dev([0]), dev([0, len(rows)]), dev(bad))
        assert syn.device_status() == syn.ERR_BOUNDS
        for x, y in zip(planes(cache, dim, page), want):
            assert np.array_equal(x, y)
    finally:
        syn.set_sm_limit(old)


@pytest.mark.parametrize("t,kv,dim,page", [(F16, 8, 128, 16), (Q8_0, 8, 128, 16), (F16, 5, 96, 8), (Q8_0, 3, 160, 64), (Q8_0, 1, 64, 8)])
@pytest.mark.parametrize("n_seq", [9, 61, 190])
def test_compact_of_many_sequences(syn, t, kv, dim, page, n_seq):
    """Several tiles to a CTA, batches that end inside a tile; no rows, one row and some hundred of a sequence."""
    rng = np.random.default_rng([t, kv, dim, n_seq])
    lens = rng.integers(0, 40, n_seq)
    lens[rng.integers(0, n_seq, 3)] = [0, 1, 700]
    base = rng.integers(0, 30, n_seq)
    need = -(-(base + lens) // page)
    n_pages, width = int(need.sum()), int(need.max())
    cache = make_cache(syn, t, kv, dim, page, n_pages, 12)
    table = np.full((n_seq, width), -1, np.int32)
    order, at = rng.permutation(n_pages), 0
    for s, m in enumerate(need):
        table[s, :m] = order[at:at + m]
        at += m
    rows = [np.nonzero(rng.random(n) < 0.5)[0] for n in lens]
    starts = np.concatenate([[0], np.cumsum([len(r) for r in rows])])
    want = planes(cache, dim, page)
    for x in want:
        for s, r in enumerate(rows):
            to, r = base[s] + np.arange(len(r)), base[s] + r
            x[table[s, to // page], :, to % page] = x[table[s, r // page], :, r % page]
    got = syn.kv_compact(cache, dev(counts(n_pages, table)), dev(table), dev(base), dev(starts), dev(np.concatenate(rows)))
    same(got, base + np.diff(starts), "lengths")
    for x, y in zip(planes(cache, dim, page), want):
        assert np.array_equal(x, y)
    assert syn.device_status() == syn.OK
