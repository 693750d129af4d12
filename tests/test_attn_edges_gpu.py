"""The paged-cache operators on the GPU at the edges of what they accept: signs, sizes and value ranges
of the options, tables and lengths that do not agree, and what a query must not notice."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_ref  # noqa: E402
from test_attn_gpu import F16, Q8_0, make_cache, options, prefill_bound, decode_bound, reference, syn  # noqa: E402,F401
from test_attn_paths_gpu import launches  # noqa: E402

pytestmark = pytest.mark.gpu

# Prefill's ways: an F16 cache, a Q8_0 cache expanded in the kernel (few rows), one expanded ahead of it
# (8 heads on a kv head, from 256 new tokens with a cap or slopes on).
WAYS = [(F16, 60), (Q8_0, 60), (Q8_0, 270)]


def on(x, dtype=None):
    import torch
    y = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return y if dtype is None else y.to(dtype)


def int32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- a cap and a scale below zero ----------------------------------------------------------
# (q with the scale -s is -q with the scale s, exactly; the tolerances are those of the positive scale)

@pytest.mark.parametrize("t,new", WAYS)
@pytest.mark.parametrize("cap,qscale", [(5.0, 1.0), (1.0, 2.0), (50.0, 0.1)])
def test_cap_with_a_negative_scale(syn, t, new, cap, qscale):
    rng = np.random.default_rng([t, new, 41])
    heads, n = 8, new + 50
    cache, pages, seqs = make_cache(syn, rng, t, 1, 64, 16, [n])
    q = (qscale * rng.standard_normal((new, heads, 64))).astype(np.float16)
    ref, size = attn_ref.attention(-q, *seqs[0], np.arange(n - new, n), np.zeros(new), 0, 0, 0.2, cap, None)
    call = syn.prepare_attn_prefill(cache, on(q), int32([0, new]), pages, int32([n]), scale=-0.2, cap=cap)
    assert launches(syn, call) == (2 if new > 256 else 1)
    got = call().double().cpu().numpy()
    assert (np.abs(got - ref) <= prefill_bound(t, size, np.abs(seqs[0][1]).max(), ref, False)).all()
    one = syn.attn_decode(cache, on(q[-1:]), pages, int32([n]), scale=-0.2, cap=cap).double().cpu().numpy()
    assert (np.abs(one - ref[-1:]) <= decode_bound(size[-1:], ref[-1:], False)).all()
    assert syn.device_status() == syn.OK


# ---- a length past what the page table holds -----------------------------------------------

@pytest.mark.parametrize("t,new", WAYS)
@pytest.mark.parametrize("window", [0, 40])
def test_length_past_the_page_table(syn, t, new, window):
    """Such a length is cut to the table: the bits of the call with the cut length, whatever the
    workspace held before."""
    rng = np.random.default_rng([t, new, 42])
    heads, held = 8, 512
    cache, pages, _ = make_cache(syn, rng, t, 1, 64, 16, [held])
    other, _, _ = make_cache(syn, rng, t, 1, 64, 16, [held])
    q = on(rng.standard_normal((new, heads, 64)).astype(np.float16))
    slopes = on(2.0 ** -np.arange(1, heads + 1).astype(np.float32))
    opt = {"window": window, "slopes": slopes}
    starts = int32([0, new])
    syn.attn_prefill(other, q, starts, pages, int32([held]), slopes=slopes)
    got = syn.attn_prefill(cache, q, starts, pages, int32([1000]), **opt)
    one = syn.attn_decode(cache, q[:1], pages, int32([1000]), **opt)
    want = syn.attn_prefill(cache, q, starts, pages, int32([held]), **opt)
    import torch
    assert torch.equal(got, want)
    assert torch.equal(one, syn.attn_decode(cache, q[:1], pages, int32([held]), **opt))
    assert syn.device_status() == syn.OK


# ---- what a query does not see, and the bits of a capped score ------------------------------

@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_deterministic_capped_prefill_alone_and_in_a_batch(syn, t, dim):
    """In deterministic mode a sequence has the same bits alone and with others whose scores are far
    larger (rows of theirs share its tiles)."""
    import torch
    rng = np.random.default_rng([t, dim, 43])
    heads, lens, new = 4, [50, 300, 40], [10, 70, 33]
    cache, pages, _ = make_cache(syn, rng, t, 1, dim, 16, lens)
    st = np.concatenate([[0], np.cumsum(new)])
    q = rng.standard_normal((st[-1], heads, dim)) * np.repeat([0.3, 30.0, 1.0], new)[:, None, None]
    q, ld = on(q.astype(np.float16)), int32(lens)
    old = syn.set_deterministic(True)
    try:
        both = syn.attn_prefill(cache, q, int32(st), pages, ld, cap=8.0)
        for s in range(3):
            one = syn.attn_prefill(cache, q[st[s]:st[s + 1]].contiguous(), int32([0, new[s]]), pages[s:s + 1].contiguous(),
                                   ld[s:s + 1].contiguous(), cap=8.0)
            assert torch.equal(one, both[st[s]:st[s + 1]]), s
    finally:
        syn.set_deterministic(old)


@pytest.mark.parametrize("t,new", WAYS)
@pytest.mark.parametrize("opt", [{"cap": 8.0}, {"cap": 8.0, "slopes": True}, {"cap": 8.0, "window": 20}, {}])
def test_unseen_keys_do_not_change_bits(syn, t, new, opt):
    """Tokens give the same bits whatever the keys after them (and past the sequence's end) hold."""
    import torch
    rng = np.random.default_rng([t, new, 44])
    heads, dim, page, n = 8, 64, 16, new + 21
    cache, pages, _ = make_cache(syn, rng, t, 1, dim, page, [n], garbage=0.25)
    q = on((0.3 * rng.standard_normal((new, heads, dim))).astype(np.float16))
    kw = dict(opt)
    if kw.pop("slopes", False):
        kw["slopes"] = on(2.0 ** -np.arange(1, heads + 1).astype(np.float32))
    call = syn.prepare_attn_prefill(cache, q, int32([0, new]), pages, int32([n]), **kw)
    want = call().clone()
    j = n - 9  # the keys from here on grow a hundredfold, those past the end too
    for row in range(j, -(-n // page) * page):
        pg, cell = int(pages[0, row // page]), row % page
        if t == F16:
            cache.k[pg, :, cell] *= 100
        else:
            at = page * dim + cell * dim // 16
            s = cache.k[pg, 0, at:at + dim // 16].view(torch.float16)
            s.copy_(s * 100)
    got = call()
    assert torch.equal(got[:new - 9], want[:new - 9])
    assert not torch.equal(got[new - 9:], want[new - 9:])


# ---- decode over Q8_0: values and keys of unlike sizes in a row ---------------------------

def q8_pool(codes, scales, page):
    """(rows, dim) codes and (rows, dim / 32) scales as a pool of one kv head, pages in order."""
    rows, dim = codes.shape
    n = -(-rows // page)
    c = np.zeros((n * page, dim), np.int8)
    d = np.zeros((n * page, dim // 32), np.float16)
    c[:rows], d[:rows] = codes, scales
    raw = np.concatenate([c.reshape(n, 1, -1).view(np.uint8), d.reshape(n, 1, -1).view(np.uint8)], -1)
    return on(raw)


def q8_rows(x):
    """Rows as codes and scales, and the values that they stand for."""
    b = x.reshape(len(x), -1, 32)
    d = (np.abs(b).max(-1) / 127).astype(np.float16)
    c = np.clip(np.rint(b / np.where(d == 0, 1, d).astype(np.float64)[..., None]), -127, 127).astype(np.int8)
    return c.reshape(x.shape), d, (c * d.astype(np.float64)[..., None]).reshape(x.shape)


# A row of large values that a head gives next to no weight (its score is 60 below the others': weight
# e^-60) does not limit how exactly that head's output is held: the bound is decode_bound's with the
# largest |v| and A of the other rows.  2^-30 max|v| e^-30 and less is what the row itself may add.
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("large,small", [(1e4, 0.1), (6e4, 0.1), (6e4, 0.01)])
@pytest.mark.parametrize("at", [0, 300, 699])
def test_decode_large_value_row_without_weight(syn, dim, large, small, at):
    rng = np.random.default_rng([dim, int(large), at])
    n, heads, page = 700, 4, 16
    u = rng.choice([-1.0, 1.0], dim)
    k = 0.3 * rng.standard_normal((n, dim))
    k[at] = -u * 60 / np.sqrt(dim)
    v = small * rng.standard_normal((n, dim))
    v[at] *= large / small
    kc, kd, kx = q8_rows(k)
    vc, vd, vx = q8_rows(v)
    cache = syn.KVCache(Q8_0, 1, dim, page, q8_pool(kc, kd, page), q8_pool(vc, vd, page))
    q = (u + 0.3 * rng.standard_normal((heads, dim))).astype(np.float16)[None]
    q[0, 2] = -u  # (one head gives that row all its weight)
    pages = int32(np.arange(-(-n // page))[None])
    ref, size = attn_ref.attention(q, kx[:, None], vx[:, None], np.array([n - 1]), np.zeros(1), 0, 0, dim ** -0.5, 0.0, None)
    others = np.arange(n) != at
    _, mine = attn_ref.attention(q, kx[others, None], vx[others, None], np.array([n - 2]), np.zeros(1), 0, 0, dim ** -0.5, 0.0, None)
    mine[:, 2] = size[:, 2]
    got = syn.attn_decode(cache, on(q), pages, int32([n])).double().cpu().numpy()
    err = np.abs(got - ref)
    assert (err <= decode_bound(mine, ref, False)).all(), (err / mine).max((0, 2)) * 2.0 ** 20


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("n", [3, 40])
def test_decode_key_blocks_with_an_outlier_channel(syn, dim, n):
    """Keys with one channel a hundred times the others, which the query does not look at: what is left
    of the score is held as exactly as if that channel were not there."""
    rng = np.random.default_rng([dim, n, 46])
    heads, page = 8, 16
    codes = np.zeros((n, dim), np.int8)
    for b in range(0, dim, 32):
        codes[np.arange(n), b + rng.integers(1, 32, n)] = rng.choice([-1, 1], n)
    codes[:, ::32] = 127
    kd = np.full((n, dim // 32), 8.0, np.float16)
    kx = (codes.reshape(n, -1, 32) * kd.astype(np.float64)[..., None]).reshape(n, dim)
    vc, vd, vx = q8_rows(rng.standard_normal((n, dim)))
    cache = syn.KVCache(Q8_0, 1, dim, page, q8_pool(codes, kd, page), q8_pool(vc, vd, page))
    q = np.abs(rng.standard_normal((20, heads, dim))).astype(np.float16)
    q[:, :, ::32] = 0
    pages = int32(np.arange(-(-n // page))[None].repeat(20, 0))
    for scale in (dim ** -0.5, 0.02):
        ref, size = attn_ref.attention(q, kx[:, None], vx[:, None], np.full(20, n - 1), np.zeros(20), 0, 0, scale, 0.0, None)
        got = syn.attn_decode(cache, on(q), pages, int32([n] * 20), scale=scale).double().cpu().numpy()
        err = np.abs(got - ref)
        assert (err <= decode_bound(size, ref, False)).all(), (scale, (err / size).max() * 2.0 ** 20)


# ---- rows computed again -------------------------------------------------------------------

@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("opt", [{}, {"cap": 6.0, "slopes": True}, {"window": 300, "prefix": 40}])
def test_rows_beside_infinite_values(syn, t, dim, opt):
    """Infinite values (F16) or scales (Q8_0) that the last tokens see: the tokens before them are right,
    and where they are seen the columns that do not hold them."""
    import torch
    rng = np.random.default_rng([t, dim, 52])
    heads, page, n, new = 4, 16, 1100, 90
    cache, pages, seqs = make_cache(syn, rng, t, 1, dim, page, [n])
    k, v = seqs[0]
    bad = n - 33
    pg, cell = int(pages[0, bad // page]), bad % page
    if t == F16:
        cache.v[pg, 0, cell, 3] = float("inf")
    else:
        at = page * dim + cell * dim // 16
        cache.v[pg, 0, at:at + 2] = torch.tensor([0, 0x7C], dtype=torch.uint8, device="cuda")
    q = rng.standard_normal((new, heads, dim)).astype(np.float16)
    sl = (2.0 ** -np.arange(1.0, heads + 1)).astype(np.float32) if opt.get("slopes") else None
    prefix, window, cap = opt.get("prefix", 0), opt.get("window", 0), opt.get("cap", 0.0)
    pos = np.arange(n - new, n)
    ref, size = attn_ref.attention(q, k, v, pos, np.zeros(new), prefix, window, dim ** -0.5, cap, sl)
    got = syn.attn_prefill(cache, on(q), int32([0, new]), pages, int32([n]), cap=cap, window=window,
                           slopes=None if sl is None else on(sl), prefix=int32([prefix]) if prefix else None).double().cpu().numpy()
    ok = np.abs(got - ref) <= prefill_bound(t, size, np.abs(v).max(), ref, False)
    seen, cols = pos >= bad, slice(3, 4) if t == F16 else slice(0, 32)
    assert ok[~seen].all()
    assert not np.isfinite(got[seen][:, :, cols]).any()
    ok[:, :, cols] = True
    assert ok[seen].all()
    assert syn.device_status() == syn.OK


def test_long_rows_computed_again_in_time(syn):
    """A CTA whose rows are all computed again over a long cache is waited for by its other warps: no
    wait runs out, and its rows are right.  (Deterministic mode: one CTA has all the keys.)"""
    import torch
    heads, dim, page, n = 32, 64, 64, 200000
    gen = torch.Generator(device="cuda").manual_seed(5)
    cache = syn.KVCache.empty(F16, 1, dim, page, n // page)
    cache.k.normal_(generator=gen)
    cache.v.normal_(generator=gen)
    q = torch.randn((5, heads, dim), device="cuda", generator=gen).half()
    bad = n - 1  # seen by the last token alone
    cache.v[bad // page, 0, bad % page, 11] = float("inf")
    pages = torch.arange(n // page, dtype=torch.int32, device="cuda").view(1, -1)
    old = syn.set_deterministic(True)
    try:
        got = syn.attn_prefill(cache, q, int32([0, 5]), pages, int32([n]))
    finally:
        syn.set_deterministic(old)
    assert syn.device_status(clear=True) == syn.OK
    k, v = (x.view(n, dim).double() for x in (cache.k, cache.v))
    for i in (0, 3):
        p = torch.softmax((q[i].double() @ k[:n - 4 + i].T) / 8, -1)
        want = p @ v[:n - 4 + i]
        # sums of 2e5 terms in fp32, some 2^-24 of the sum of their sizes each, beside prefill's own bound
        assert (got[i].double() - want).abs().max() <= v[:-1].abs().max() * (2.0 ** -11 + 2.0 ** -24 * 16 * 30)
    assert torch.isinf(got[4, :, 11]).all() and torch.isfinite(got[4, :, :11]).all()


@pytest.mark.parametrize("new", [60, 270])
def test_cached_keys_past_fp16(syn, new):
    """Keys of a Q8_0 cache that fp16 does not hold (a scale above 516) are finite all the same: rows
    that see one are right, in one or the other way of expanding."""
    rng = np.random.default_rng([new, 53])
    heads, dim, page, n = 8, 64, 16, new + 60
    kc, kd, kx = q8_rows(rng.standard_normal((n, dim)))
    vc, vd, vx = q8_rows(rng.standard_normal((n, dim)))
    j = n - 20
    kc[j, :32] = 0
    kc[j, 7] = 127
    kd[j, 0] = 1500.0
    kx[j, :32] = kc[j, :32] * 1500.0
    cache = syn.KVCache(Q8_0, 1, dim, page, q8_pool(kc, kd, page), q8_pool(vc, vd, page))
    q = rng.standard_normal((new, heads, dim)).astype(np.float16)
    q[:, ::2, 7] = -(2.0 ** -14)  # (the score of that key: near -1.5 for half of the heads, of all sizes for the others)
    pos = np.arange(n - new, n)
    ref, size = attn_ref.attention(q, kx[:, None], vx[:, None], pos, np.zeros(new), 0, 0, dim ** -0.5, 30.0, None)
    got = syn.attn_prefill(cache, on(q), int32([0, new]), int32(np.arange(-(-n // page))[None]), int32([n]), cap=30.0).double().cpu().numpy()
    assert (np.abs(got - ref) <= prefill_bound(Q8_0, size, np.abs(vx).max(), ref, False)).all()
    assert syn.device_status() == syn.OK


# ---- page tables far wider than the lengths ------------------------------------------------

@pytest.mark.parametrize("width,want", [(8191, 2), (8192, 1)])
def test_expansion_keeps_to_its_room(syn, width, want):
    """The workspace of the expansion is 2 GiB at the most, the page table in it counted."""
    import torch
    kv, dim, page = 8, 128, 64
    cache = syn.KVCache.empty(Q8_0, kv, dim, page, 8)
    pages = torch.zeros((1, width), dtype=torch.int32, device="cuda")
    pages[0, :8] = torch.arange(8)
    side = torch.cuda.Stream()
    q = torch.zeros((300, 8 * kv, dim), dtype=torch.float16, device="cuda")
    call = syn.prepare_attn_prefill(cache, q, int32([0, 300]), pages, int32([400]), cap=5.0, stream=side)
    small = syn.prepare_attn_prefill(cache, q[:3], int32([0, 3]), pages, int32([400]), cap=5.0, stream=side)
    small()  # (the workspace for partial results)
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    assert launches(syn, call) == want
    torch.cuda.synchronize()
    assert before - torch.cuda.mem_get_info()[0] <= 2 ** 31 + 2 ** 22
    syn.check(syn.syn_release(), "syn_release")


@pytest.mark.parametrize("n_seq,width", [(2, 4096), (300, 64)])
@pytest.mark.parametrize("window", [0, 40])
def test_expansion_of_few_pages_of_a_wide_table(syn, n_seq, width, window):
    """A Q8_0 cache expanded ahead of the prefill gives the same bits whatever room its page table has
    behind the lengths, and whatever ids stand there."""
    import torch
    rng = np.random.default_rng([n_seq, width, 51])
    heads, dim, page = 16, 64, 16
    new = [int(x) for x in rng.integers(100, 400, n_seq)]
    lens = [m + int(rng.integers(0, 200)) if i % 7 else m // 2 for i, m in enumerate(new)]
    cache, pages, _ = make_cache(syn, rng, Q8_0, 1, dim, page, lens)
    q = on(rng.standard_normal((sum(new), heads, dim)).astype(np.float16))
    opt = {"slopes": on(2.0 ** -np.arange(1, heads + 1).astype(np.float32)), "window": window}
    starts = int32(np.concatenate([[0], np.cumsum(new)]))
    narrow = syn.prepare_attn_prefill(cache, q, starts, pages, int32(lens), **opt)
    assert launches(syn, narrow) == 2
    wide = torch.randint(-9, 10 ** 6, (n_seq, width), dtype=torch.int32, device="cuda")
    for s, n in enumerate(lens):
        wide[s, :-(-n // page)] = pages[s, :-(-n // page)]
    assert torch.equal(syn.attn_prefill(cache, q, starts, wide, int32(lens), **opt), narrow())
    assert syn.device_status() == syn.OK


# ---- pages that no query sees --------------------------------------------------------------

@pytest.mark.parametrize("t,new", WAYS)
@pytest.mark.parametrize("page", [8, 16, 64])
def test_pages_that_no_query_sees_may_be_gone(syn, t, new, page):
    """A server gives back the pages that have left the window: their ids in the table are no error, and
    an id outside the pool in a page that a query sees still is one."""
    import torch
    rng = np.random.default_rng([t, new, page, 47])
    heads, window = 8, 37
    n = 700 + page // 2 + 3
    cache, pages, _ = make_cache(syn, rng, t, 1, 64, page, [n])
    q = on(rng.standard_normal((new, heads, 64)).astype(np.float16))
    slopes = on(2.0 ** -np.arange(1, heads + 1).astype(np.float32))
    opt = {"window": window, "slopes": slopes}
    calls = {"prefill": (new, lambda p: syn.attn_prefill(cache, q, int32([0, new]), p, int32([n]), **opt)),
             "decode": (1, lambda p: syn.attn_decode(cache, q[:1], p, int32([n]), **opt))}
    for name, (m, call) in calls.items():
        want = call(pages)
        low = n - m - window + 1  # the first row that some query sees
        gone = pages.clone()
        gone[0, :low // page] = -1
        assert torch.equal(call(gone), want), name
        assert syn.device_status(clear=True) == syn.OK, name
        gone[0, low // page] = -1
        call(gone)
        assert syn.device_status(clear=True) == syn.ERR_BOUNDS, name
    # a prefix is seen past the window: its pages stay, the ones between may go
    prefix = int32([page + 3])
    want = syn.attn_decode(cache, q[:1], pages, int32([n]), prefix=prefix, **opt)
    gone = pages.clone()
    gone[0, 2:(n - window) // page] = -1
    assert torch.equal(syn.attn_decode(cache, q[:1], gone, int32([n]), prefix=prefix, **opt), want)
    assert syn.device_status(clear=True) == syn.OK
    want = syn.attn_prefill(cache, q, int32([0, new]), pages, int32([n]), prefix=prefix, **opt)
    gone[0, 2:] = pages[0, 2:]
    gone[0, 2:(n - new - window + 1) // page] = -1
    assert torch.equal(syn.attn_prefill(cache, q, int32([0, new]), gone, int32([n]), prefix=prefix, **opt), want)
    assert syn.device_status(clear=True) == syn.OK


# ---- infinite values that a query sees ------------------------------------------------------

@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_decode_infinite_values(syn, dim):
    """An infinity or NaN among the values that a query sees reaches its column of the output alone (as an
    infinity or NaN); the other columns, heads and sequences are as they are."""
    rng = np.random.default_rng([dim, 48])
    heads, kv, page, lens = 8, 2, 16, [400, 90, 3000]
    cache, pages, seqs = make_cache(syn, rng, F16, kv, dim, page, lens)

    def put(s, row, h, e, x):
        cache.v[int(pages[s, row // page]), h, row % page, e] = x

    put(0, 17, 0, 5, float("inf")), put(0, 333, 0, 5, float("inf"))
    put(0, 200, 0, 9, float("-inf"))
    put(0, 40, 1, 1, float("inf")), put(0, 41, 1, 1, float("-inf"))
    put(0, 60, 1, 2, float("nan"))
    put(2, 2222, 0, 31, float("inf"))
    q = rng.standard_normal((3, heads, dim)).astype(np.float16)
    ref, size = reference(q, seqs, [np.array([n - 1]) for n in lens], [np.zeros(1)] * 3, [0] * 3, 0, dim ** -0.5, 0.0, None)
    got = syn.attn_decode(cache, on(q), pages, int32(lens)).double().cpu().numpy()
    g = heads // kv
    for s, heads_of, e in ((0, slice(0, g), 5), (0, slice(0, g), 9), (0, slice(g, None), 1), (0, slice(g, None), 2), (2, slice(0, g), 31)):
        assert not np.isfinite(got[s, heads_of, e]).any()
        got[s, heads_of, e] = ref[s, heads_of, e]
    assert (np.abs(got - ref) <= decode_bound(size, ref, False)).all()
    assert syn.device_status() == syn.OK


# ---- options at the ends of the float range --------------------------------------------------

@pytest.mark.parametrize("t,new", WAYS)
@pytest.mark.parametrize("cap", [1e-7, 1e-12, 1e-39, 1e38])
def test_caps_at_the_ends_of_the_range(syn, t, new, cap):
    """Scores of zero stay zero however small the cap is; a cap far above every score changes nothing."""
    rng = np.random.default_rng([t, new, 49])
    heads, n = 8, new + 30
    cache, pages, seqs = make_cache(syn, rng, t, 1, 64, 16, [n])
    q = rng.standard_normal((new, heads, 64)).astype(np.float16)
    q[::3] = 0
    cap = float(np.float32(cap))
    ref, size = attn_ref.attention(q, *seqs[0], np.arange(n - new, n), np.zeros(new), 0, 0, 0.125, 0.0 if cap > 1 else cap, None)
    got = syn.attn_prefill(cache, on(q), int32([0, new]), pages, int32([n]), cap=cap).double().cpu().numpy()
    assert (np.abs(got - ref) <= prefill_bound(t, size, np.abs(seqs[0][1]).max(), ref, False)).all()
    one = syn.attn_decode(cache, on(q[-4:]), pages.expand(4, -1).contiguous(), int32([n] * 4), cap=cap).double().cpu().numpy()
    last, size = attn_ref.attention(q[-4:], *seqs[0], np.array([n - 1] * 4), np.zeros(4), 0, 0, 0.125, 0.0 if cap > 1 else cap, None)
    assert (np.abs(one - last) <= decode_bound(size, last, False)).all()


@pytest.mark.parametrize("t,new", WAYS[:2])
@pytest.mark.parametrize("scale", [3e38, -3e38, 2.0 ** 34])
def test_scales_at_the_ends_of_the_range(syn, t, new, scale):
    """The key of the largest score takes all the weight; queries of zeros see every key alike."""
    rng = np.random.default_rng([t, new, 50])
    heads, n, dim = 8, new + 30, 64
    k = np.zeros((n, 1, dim), np.float16)
    k[:, 0, 0] = rng.permutation(n) - n // 2  # (products: whole numbers apart)
    codes = k[:, 0].astype(np.int8)
    v = rng.integers(-100, 100, (n, dim)).astype(np.int8)
    rows = -(-n // 16) * 16
    if t == F16:
        pad = lambda x: on(np.pad(x, ((0, rows - n), (0, 0))).astype(np.float16).reshape(-1, 1, 16, dim))  # noqa: E731
        cache = syn.KVCache(F16, 1, dim, 16, pad(codes), pad(v))
    else:
        one = np.ones((n, dim // 32), np.float16)
        cache = syn.KVCache(Q8_0, 1, dim, 16, q8_pool(codes, one, 16), q8_pool(v, one, 16))
    q = np.zeros((new, heads, dim), np.float16)
    q[:, 1::2, 0] = 2.0 ** -8
    pages = int32(np.arange(rows // 16)[None])
    got = syn.attn_prefill(cache, on(q), int32([0, new]), pages, int32([n]), scale=scale).double().cpu().numpy()
    one = syn.attn_decode(cache, on(q[-1:]), pages, int32([n]), scale=scale).double().cpu().numpy()
    for i in range(new):
        seen = codes[:n - new + i + 1, 0].astype(int) * (1 if scale > 0 else -1)
        top = v[seen.argmax()].astype(np.float64)
        mean = v[:len(seen)].astype(np.float64).mean(0)
        assert (got[i, 1::2] == top).all() and (np.abs(got[i, ::2] - mean) <= 100 * 2.0 ** -11).all()
    assert (one[0, 1::2] == top).all() and (np.abs(one[0, ::2] - mean) <= 100 * 2.0 ** -20).all()


# ---- the calling thread's own stream --------------------------------------------------------

def test_threads_on_their_own_default_streams(syn):
    """The handle of the per-thread default stream names another stream in every thread: split calls of
    two threads at once, each with a workspace of its own, give what they give one after the other."""
    import threading

    import torch
    rng = np.random.default_rng(54)
    heads, kv, dim, page, n = 8, 2, 128, 64, 30000
    cache, pages, _ = make_cache(syn, rng, F16, kv, dim, page, [n])
    qs = [on(rng.standard_normal((1, heads, dim)).astype(np.float16)) for _ in range(2)]
    ld = int32([n])
    want = [syn.attn_decode(cache, q, pages, ld) for q in qs]
    outs = [[torch.zeros_like(want[0]) for _ in range(100)] for _ in qs]
    torch.cuda.synchronize()
    gate, wrong = threading.Barrier(2), []

    def work(i):
        calls = [syn.prepare_attn_decode(cache, qs[i], pages, ld, out, stream=2) for out in outs[i]]  # cudaStreamPerThread
        try:
            gate.wait(20)
            for call in calls:
                call()
        except Exception as e:  # (told below)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong
    for i in range(2):
        for out in outs[i]:
            assert torch.equal(out, want[i])
    assert syn.device_status() == syn.OK


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_decode_scales_of_every_size(syn, dim):
    """Value scales from zero and subnormal numbers to fp16's largest, in any order, and the code -128."""
    rng = np.random.default_rng([dim, 55])
    n, heads, page = 333, 8, 16
    kc, kd, kx = q8_rows(0.5 * rng.standard_normal((n, dim)))
    vc = rng.integers(-128, 128, (n, dim)).astype(np.int8)
    vd = (2.0 ** rng.uniform(-24, 9, (n, dim // 32))).astype(np.float16)
    vd[rng.random(vd.shape) < 0.3] = 0
    vd[:40] = 0
    vd[120:] = (2.0 ** rng.uniform(-24, -9, (n - 120, dim // 32))).astype(np.float16)
    vx = (vc.reshape(n, -1, 32) * vd.astype(np.float64)[..., None]).reshape(n, dim)
    cache = syn.KVCache(Q8_0, 1, dim, page, q8_pool(kc, kd, page), q8_pool(vc, vd, page))
    q = rng.standard_normal((4, heads, dim)).astype(np.float16)
    lens = [n, 37, 70, n]
    first = np.array([0, 0, 41, 130], np.int32)  # (the second sees zeros alone, the last small scales alone)
    pages = int32(np.arange(-(-n // page))[None].repeat(4, 0))
    got = syn.attn_decode(cache, on(q), pages, int32(lens), first=on(first)).double().cpu().numpy()
    for i in range(4):
        ref, size = attn_ref.attention(q[i:i + 1], kx[first[i]:lens[i], None], vx[first[i]:lens[i], None], np.array([lens[i] - first[i] - 1]),
                                       np.zeros(1), 0, 0, dim ** -0.5, 0.0, None)
        assert (np.abs(got[i:i + 1] - ref) <= decode_bound(size, ref, False)).all(), i
    assert (got[1] == 0).all() and np.abs(got[3]).max() > 0


def test_a_graph_captured_on_the_threads_own_stream(syn):
    import torch
    rng = np.random.default_rng(56)
    cache, pages, _ = make_cache(syn, rng, F16, 2, 64, 16, [3000])
    q, ld = on(rng.standard_normal((1, 8, 64)).astype(np.float16)), int32([3000])
    want = syn.attn_decode(cache, q, pages, ld)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    step = syn.prepare_attn_decode(cache, q, pages, ld, out, stream=2)  # cudaStreamPerThread
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.ExternalStream(2)):
        step()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
