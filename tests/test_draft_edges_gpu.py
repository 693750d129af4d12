"""The operators of drafted tokens where several of their parts meet: many candidates over several turns, long lists one
after the other, few SMs, values at the ends of their types."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

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


def most_likely(x, n_top):
    """The tokens of the n_top largest, ties to the lower one."""
    import torch
    bits = (x.float() + 0.0).view(torch.int32)
    key = ((bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32) - torch.arange(x.shape[1], device="cuda")
    return torch.topk(key, n_top, 1).indices.to(torch.int32)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("rows,n_top", [(600, 40), (600, 50), (600, 64), (310, 57)])
def test_candidates_over_several_turns(syn, rows, n_top, half):
    """A CTA to a row of 128256 logits: 16 or 32 units a turn are read again, and more than 64 logits found, so that the list
    is cut between two turns."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(rows + n_top)
    for _ in range(4):
        x = torch.randn((rows, 128256), device="cuda", generator=gen)
        if half:
            x = x.half()  # (ties among the largest)
        want = most_likely(x, n_top)
        for _ in range(3):
            got = syn.logprobs(x, n_top=n_top)
            assert torch.equal(got.top, want)
            z = x.gather(1, want.long()).double() - torch.logsumexp(x.double(), 1, keepdim=True)
            # 2^-17 for ln S, 2^-22 of the log probability
            assert ((got.top_logprob - z).abs() <= 2.0 ** -17 + 2.0 ** -22 * z.abs()).all()


def packed_case(syn, rng, t, kv, dim, page, n):
    """A cache of random bits that one sequence of n rows fills, its table, and the pools' planes [pages, kv, page, bytes]."""
    import torch
    n_pages = -(-n // page)
    shape = (kv, page, dim * 2) if t == F16 else (kv, page * dim // 16 * 17)
    pools = [torch.randint(0, 256, (n_pages, *shape), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = syn.KVCache(t, kv, dim, page, *(p.view(torch.float16) if t == F16 else p for p in pools))
    planes = pools if t == F16 else [x for p in pools for x in (p[..., :page * dim].unflatten(-1, (page, dim)),
                                                                p[..., page * dim:].unflatten(-1, (page, dim // 16)))]
    return cache, torch.from_numpy(rng.permutation(n_pages)).cuda(), planes


def pack(planes, table, rows, page):
    """The planes as the rows (numpy, ascending) leave them."""
    import torch
    to, come = torch.arange(len(rows), device="cuda"), torch.from_numpy(rows).cuda()
    out = []
    for x in planes:
        y = x.clone()
        y[table[to // page], :, to % page] = x[table[come // page], :, come % page]
        out.append(y)
    return out


@pytest.mark.parametrize("t,kv,dim", [(F16, 2, 64), (Q8_0, 4, 128), (Q8_0, 1, 32)])
def test_long_lists_one_after_the_other(syn, t, kv, dim):
    """Calls that follow each other on a stream use the same counters and flags: each leaves them at zero."""
    import torch
    rng, page, n = np.random.default_rng(dim), 16, 9000
    cases = [packed_case(syn, rng, t, kv, dim, page, n) for _ in range(6)]
    for turn in range(10):
        keep = [np.nonzero(rng.random(n) < share)[0] for share in (0.5, 0.999, 0.3, 0.97, 0.6, 0.9)]
        want = [pack(planes, table, r, page) for (_, table, planes), r in zip(cases, keep)]
        steps = [syn.prepare_kv_compact(cache, None, table[None].int(), torch.zeros(1, dtype=torch.int32, device="cuda"),
                                        torch.tensor([0, len(r)], dtype=torch.int32, device="cuda"),
                                        torch.from_numpy(r.astype(np.int32)).cuda()) for (cache, table, _), r in zip(cases, keep)]
        torch.cuda.synchronize()
        lens = [step() for step in steps]
        assert [x.item() for x in lens] == [len(r) for r in keep]
        for (_, _, planes), w in zip(cases, want):
            assert all(torch.equal(x, y) for x, y in zip(planes, w)), turn


def reference(x, scale=1.0, cap=0.0):
    """Log probabilities and entropy of rows without NaN, in 64 bits."""
    import torch
    x = x.double()
    z = cap * torch.tanh(x / cap) if cap else x
    z = torch.where(x == -torch.inf, x, z) * scale
    z = z - z.amax(1, keepdim=True)
    logp = z - torch.log(torch.exp(z).sum(1, keepdim=True))
    p = torch.exp(logp)
    return logp, -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)


@pytest.mark.parametrize("v", [40, 20001, 128256])
def test_logits_of_the_types_lowest_value(syn, v):
    """A mask of finfo.min instead of -inf: such a token's log probability is a number as long as fp32 holds it."""
    import torch
    for t in (torch.float32, torch.float16):
        low = torch.finfo(t).min
        x = torch.randn((6, v), device="cuda").to(t)
        x[0, 1:] = low
        x[1, ::2] = low
        x[2, v // 2:] = low
        x[3] = low  # (all alike)
        x[4] = low
        x[4, 3] = -low
        ids = torch.tensor([[v - 1, 0], [0, 1], [v - 1, 0], [0, v - 1], [3, 0], [0, v - 1]], dtype=torch.int32, device="cuda")
        for scale in (1.0, 0.25, 3.0, 1e-30):
            want, entropy = reference(x, scale)
            got = syn.logprobs(x, ids, 3, scale=scale)
            for value, want in ((got.logprob, want.gather(1, ids.long())), (got.top_logprob, want.gather(1, most_likely(x, 3).long())),
                                (got.entropy, entropy)):
                limit = torch.finfo(torch.float32).max
                over = want < -limit * (1 + 2.0 ** -24)  # (what fp32 does not hold is -inf)
                assert (value[over] == -torch.inf).all()
                off = (value.double() - want)[~over].abs()
                assert (off <= 2.0 ** -17 + 2.0 ** -22 * want[~over].abs()).all(), (t, scale)
            assert torch.equal(got.top, most_likely(x, 3))


def test_scales_at_the_ends_of_the_float_range(syn):
    """The largest logits alone count under the largest scales, all alike under the smallest."""
    import torch
    x = torch.randn((3, 5000), device="cuda")
    x[1, 7:9] = 20.0
    x[2, 9] = 30.0
    for scale in (3e38, 1e30):
        got = syn.logprobs(x, x.argmax(1, keepdim=True).int(), 2, scale=scale)
        want = torch.tensor([0.0, float(np.log(2.0)), 0.0], dtype=torch.float32, device="cuda")
        assert torch.allclose(got.entropy, want, rtol=0, atol=1e-6) and torch.allclose(got.logprob[:, 0], -want, rtol=0, atol=1e-6)
        assert got.top_logprob[0, 1] < -1e25 and got.top_logprob[2, 1] < -1e25
    got = syn.logprobs(x, n_top=1, scale=1e-38)
    assert torch.allclose(got.entropy, torch.full((3,), float(np.log(5000.0)), device="cuda"), rtol=1e-6, atol=0)


def test_starts_that_overlap_are_refused(syn):
    """More new rows in all than the call has: nothing changes, and it is reported.  (Sums of columns stop at 2^30, so that
    none comes out small.)"""
    import torch
    cache = syn.KVCache.empty(F16, 1, 32, 8, 200)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    refs, pages, lens = i32([0] * 200), torch.full((9, 8), -1, dtype=torch.int32, device="cuda"), i32([3] * 9)
    _, slots = syn.kv_extend(cache, refs, pages, lens, starts=i32([0, 40] * 5), n_tok=40)
    assert syn.device_status() == syn.ERR_BOUNDS
    assert lens.tolist() == [3] * 9 and (refs == 0).all() and (pages == -1).all() and (slots == -1).all()


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.0 ** 90])
@pytest.mark.parametrize("slopes", [False, True])
def test_large_products_under_large_scales(syn, scale, slopes):
    """The key of the largest product takes all the weight, in every form of the attention, where products are past 2^28 and
    the scale is the float range's end; queries of zeros see every key alike (without slopes)."""
    import torch
    rng = np.random.default_rng(51)
    n, new, heads, dim = 120, 20, 4, 64
    k = np.zeros((128, 1, dim), np.float16)
    k[:n, 0, 0] = 512.0 * (rng.permutation(n) - n // 2)  # (7 bits: exact; 2^15 at most)
    v = rng.integers(-100, 100, (128, dim)).astype(np.float16)
    q = np.zeros((new, heads, dim), np.float16)
    q[:, 1::2, 0] = 2.0 ** 15  # products up to 2^30
    pool = lambda x: torch.from_numpy(x.reshape(8, 1, 16, dim)).cuda()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache, pages, on = syn.KVCache(F16, 1, dim, 16, pool(k), pool(v)), i32([list(range(8))]), torch.from_numpy(q).cuda()
    opt = {"scale": scale, "slopes": torch.full((heads,), 0.125, device="cuda") if slopes else None}
    tree = syn.attn_tree(cache, on, i32([0, new]), i32(range(-1, new - 1)), pages, i32([n]), **opt).double().cpu().numpy()
    prefill = syn.attn_prefill(cache, on, i32([0, new]), pages, i32([n]), **opt).double().cpu().numpy()
    one = syn.attn_decode(cache, on[-1:], pages, i32([n]), **opt).double().cpu().numpy()
    for i in range(new):
        seen = k[:n - new + i + 1, 0, 0].astype(np.float64) * np.sign(scale)
        top, mean = v[seen.argmax()].astype(np.float64), v[:len(seen)].astype(np.float64).mean(0)
        for got in (tree[i], prefill[i]) + ((one[0],) if i == new - 1 else ()):
            assert (got[1::2] == top).all(), i
            assert slopes or (np.abs(got[::2] - mean) <= 100 * 2.0 ** -11).all()
    assert syn.device_status() == syn.OK


def test_drafts_of_more_sequences_than_alternatives(syn):
    """logprobs gives at most 64 first tokens: more sequences share them."""
    from gguf_block_quantized_gb300 import attn_block
    r = attn_block.run_drafts(F16, 20, 3, 70, 4, vocab=1000, page=16)
    # (as tests/test_draft_block_gpu.py derives.  The tokens need not be the same: the best two lie closer together than the forms
    # differ in some of 280 draws of 1000 logits, by 0.0009 to 0.0053 where the forms differ by up to 0.013.)
    assert r["held"] == 0 and r["difference"] <= 16 * 8 * 2.0 ** -11 and r["per_step"] >= 1.0


def held_to(got, want, more=0.0):
    """The public bound (include/syn.h): 1e-6 of the larger of 1 and the result's size, and what a cap adds.  (Of a
    result: d and its product 2^-23 of themselves; ln S 2^-22 by its powers, their exponents' roundings 2^-22 of T/S,
    which is below the entropy, its additions some 2^-24 each way; together below 2^-20 of the larger of 1 and the result.)"""
    off = (got.double() - want).abs()
    bound = 1e-6 * want.abs().clamp(min=1) + more
    assert (off <= bound).all(), float((off / bound).max())


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("n,v", [(3, 1), (40, 33), (64, 5003), (2, 50257), (300, 50257), (1, 128256), (320, 128256), (700, 20011)])
@pytest.mark.parametrize("spread", [0.0, 0.3, 2.5, 12.0])
def test_log_probabilities_are_as_exact_as_stated(syn, n, v, half, spread):
    """Rows nearly alike, ordinary and peaked, up to a vocabulary that one CTA sums alone."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(v + n)
    x = (torch.randn((n, v), device="cuda", generator=gen) * spread).to(torch.float16 if half else torch.float32)
    ids = torch.randint(0, v, (n, 8), dtype=torch.int32, device="cuda", generator=gen)
    k = min(v, 20)
    for scale, cap in ((1.0, 0.0), (0.7, 0.0), (1.0, 30.0), (1.25, 5.0)):
        want, entropy = reference(x, float(np.float32(scale)), cap)
        got = syn.logprobs(x, ids, k, scale=scale, cap=cap)
        lax = 5e-7 * cap * scale
        held_to(got.logprob, want.gather(1, ids.long()), lax)
        held_to(got.top_logprob, want.gather(1, most_likely(x, k).long()), lax)
        held_to(got.entropy, entropy, lax * entropy.clamp(min=1))


@pytest.mark.parametrize("limit", [1, 3, 20])
@pytest.mark.parametrize("t,kv,dim", [(F16, 1, 64), (Q8_0, 2, 128), (F16, 3, 256), (Q8_0, 1, 96)])
def test_long_lists_on_few_sms(syn, t, kv, dim, limit):
    """A CTA takes many chunks one after the other, and waits for those of the few others."""
    import torch
    rng, page, n = np.random.default_rng([dim, limit]), 16, 12000
    old = syn.set_sm_limit(limit)
    try:
        for share in (0.5, 0.9995, 0.05):
            cache, table, planes = packed_case(syn, rng, t, kv, dim, page, n)
            rows = np.nonzero(rng.random(n) < share)[0]
            rows = rows if len(rows) >= 1024 else np.sort(rng.permutation(n)[:1024])
            want = pack(planes, table, rows, page)
            got = syn.kv_compact(cache, None, table[None].int(), torch.zeros(1, dtype=torch.int32, device="cuda"),
                                 torch.tensor([0, len(rows)], dtype=torch.int32, device="cuda"), torch.from_numpy(rows.astype(np.int32)).cuda())
            assert got.item() == len(rows)
            assert all(torch.equal(x, y) for x, y in zip(planes, want)), share
    finally:
        syn.set_sm_limit(old)


def test_a_list_that_does_not_ascend_leaves_the_others_alone(syn):
    """What its own sequence's packed rows hold is not defined; the other sequences, the rows behind, the lengths and the report are."""
    import torch
    rng, page, n = np.random.default_rng(77), 16, 4000
    for small in (False, True):
        m = 60 if small else n
        cache, table, planes = packed_case(syn, rng, F16, 2, 64, page, 3 * m)
        pages = table[:3 * m // page].view(3, -1) if 3 * m % (3 * page) == 0 else table[:3 * (m // page)].view(3, -1)
        held = pages.shape[1] * page
        good = np.nonzero(rng.random(held) < 0.6)[0]
        bad = np.arange(1, held // 2)
        bad[len(bad) // 3] = 0
        rows = [good, bad, good]
        want = [x.clone() for x in planes]
        for s in (0, 2):
            for i, y in enumerate(pack(planes, pages[s], good, page)):
                own = pages[s]
                want[i][own] = y[own]
        starts = np.concatenate([[0], np.cumsum([len(r) for r in rows])]).astype(np.int32)
        got = syn.kv_compact(cache, None, pages.int().contiguous(), torch.zeros(3, dtype=torch.int32, device="cuda"), torch.from_numpy(starts).cuda(),
                             torch.from_numpy(np.concatenate(rows).astype(np.int32)).cuda())
        assert syn.device_status() == syn.ERR_BOUNDS
        assert got.tolist() == [len(r) for r in rows]
        row = torch.arange(len(bad), device="cuda")
        for x, w in zip(planes, want):  # (the second sequence's packed rows aside)
            w[pages[1][row // page], :, row % page] = x[pages[1][row // page], :, row % page]
            assert torch.equal(x, w)


@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("heads,kv,dim", [(256, 1, 32), (1024, 1, 32), (600, 2, 64), (300, 1, 256), (1024, 1024, 32)])
def test_trees_of_many_heads(syn, t, heads, kv, dim):
    """A token's heads over one item or several, in numbers that divide 128 or do not."""
    from test_attn_tree_gpu import run
    run(syn, t, heads, kv, dim, 16, [60, 33], [4, 3], [heads, dim], dts=("float32",))
    run(syn, t, heads, kv, dim, 16, [60, 33], [4, 3], [heads, dim], dts=("float32",), window=3, slopes=True)


def test_as_many_sequences_as_extend_takes(syn):
    import pages_ref
    import torch
    rng, n, width, page, n_pages = np.random.default_rng(8), 4096, 5, 8, 15000
    cache = syn.KVCache.empty(F16, 1, 32, page, n_pages)
    refs, pages, lens = np.zeros(n_pages, np.int32), np.full((n, width), -1, np.int32), np.zeros(n, np.int32)
    on = [torch.from_numpy(x.copy()).cuda() for x in (refs, pages, lens)]
    for new in (rng.integers(0, 12, n), rng.integers(0, 20, n), np.ones(n, np.int64), rng.integers(0, 30, n)):  # (the last: pages are short)
        refs, pages, lens, slots, _ = pages_ref.extend(refs, pages, lens, new, page)
        starts = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
        _, got = syn.kv_extend(cache, *on, starts=starts, n_tok=int(new.sum()))
        for x, y in zip((*on, got), (refs, pages, lens, slots)):
            assert np.array_equal(x.cpu().numpy(), y)


@pytest.mark.parametrize("t", [F16, Q8_0])
def test_pools_past_32_bit_offsets(syn, t):
    """Rows and pages at the end of pools of 5 GB: extended, copied, packed and read by trees as in a small pool."""
    import torch
    dim, kv, page = 128, 8, 64
    tile = page * dim * 2 if t == F16 else page * dim // 16 * 17
    n_pages, few = 5 * 10 ** 9 // (tile * kv), 80
    shape = (kv, page, dim) if t == F16 else (kv, page * dim // 16 * 17)
    kind = torch.float16 if t == F16 else torch.uint8
    gen = torch.Generator(device="cuda").manual_seed(3)
    rows = [torch.randn((few, *shape), device="cuda", generator=gen).half() if t == F16 else
            torch.randint(0, 40, (few, *shape), dtype=torch.uint8, device="cuda", generator=gen) for _ in range(2)]
    results = []
    for n in (n_pages, few):
        pools = [torch.empty((n, *shape), dtype=kind, device="cuda") for _ in range(2)]
        for p, r in zip(pools, rows):
            p[-few:] = r
        cache, at = syn.KVCache(t, kv, dim, page, *pools), n - few
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        refs = torch.ones(n, dtype=torch.int32, device="cuda")
        refs[at + 40:] = 0  # (two sequences of 20 pages share the first 20 once, then pages are free)
        pages = torch.full((2, 24), -1, dtype=torch.int32, device="cuda")
        pages[0, :20] = torch.arange(at, at + 20, device="cuda")
        pages[1, :20] = torch.arange(at, at + 20, device="cuda")
        refs[at:at + 20] = 2
        lens, starts = i32([19 * 64 + 5] * 2), i32([0, 70, 140])
        long, slots = syn.kv_extend(cache, refs, pages, lens, torch.empty_like(lens), starts=starts, n_tok=140)
        syn.kv_copy(cache, cache, i32([at + 21, at + 22]), i32([at + 70, at + 71]))
        q = torch.randn((140, 32, dim), device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).half()
        parents = i32([(i - 1) // 2 if i else -1 for i in range(70)] * 2)
        out = syn.attn_tree(cache, q, starts, parents, pages, long)
        own = pages.clone()
        own[:, :19] = torch.arange(at + 41, at + 79, device="cuda").view(2, 19)  # (pages of their own, to be written to)
        keep = torch.arange(0, 19 * 64, 2, dtype=torch.int32, device="cuda")
        for much in (keep, keep[:100]):
            got = syn.kv_compact(cache, None, own, i32([0, 0]), i32([0, much.numel(), 2 * much.numel()]), much.repeat(2))
        results.append([pages - at * (pages >= 0), slots - at * page, refs[at:], long, out, got, *(p[-few:].clone() for p in pools)])
        del pools, cache
    assert syn.device_status() == syn.OK
    for a, b in zip(*results):
        assert torch.equal(a, b)
