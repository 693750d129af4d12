"""syn_logprobs on the GPU against its definition in 64 bits.

Tolerances.  d = z - max z takes two roundings of 2^-24 of itself (three with a row's own scale).  A thread sums 16
powers at a time, then pieces, threads and CTAs join: fewer than 64 additions in a row, each 2^-24 of a sum of
positive numbers, and each power is off by 2^-22 and by what its exponent's rounding gives (|d| e^d <= 1/e): ln S is off by less
than 2^-17, S's own rounding included, at the largest vocabularies here.  So a log probability is off by at
most 2^-17 + 2^-22 |logp|, the entropy by as much for ln S and 2^-17 of T/S (whose terms add up in the same
way).  A capped logit is off by 2^-21 of the cap at most (tanh to 3e-7, its rounding), a difference of two by twice that,
which moves ln S by as much.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def syn():
    import torch
    assert torch.cuda.is_available()
    from gguf_block_quantized_gb300 import syn
    yield syn
    torch.cuda.synchronize()
    assert syn.device_status() == syn.OK


def reference(x, ids, n_top, scale=1.0, cap=0.0, scales=None, on=None):
    x = x.astype(np.float64)
    if on is not None:
        x = np.where(on, x, -np.inf)
    z = cap * np.tanh(x / cap) if cap else x
    z = np.where(x == -np.inf, -np.inf, z) * scale
    if scales is not None:
        z = z * scales.astype(np.float64)[:, None]
    top = z.max(1, keepdims=True)
    top[top == -np.inf] = 0
    s = np.exp(z - top).sum(1, keepdims=True)
    logp = z - top - np.log(np.where(s == 0, 1, s))
    p = np.exp(logp)
    out = {"entropy": -np.where(p > 0, p * np.where(p > 0, logp, 0), 0).sum(1)}
    if ids is not None:
        out["logprob"] = np.where(ids < 0, 0, np.take_along_axis(logp, np.maximum(ids, 0).astype(np.int64), 1))
    if n_top:
        order = np.argsort(-x, axis=1, kind="stable")[:, :n_top]
        got = np.take_along_axis(logp, order, 1)
        got = np.pad(got, ((0, 0), (0, n_top - got.shape[1])), constant_values=-np.inf)
        order = np.pad(order, ((0, 0), (0, n_top - order.shape[1])), constant_values=-1)
        out["top"], out["top_logprob"] = np.where(got == -np.inf, -1, order), got
    out["log_s"] = np.log(np.where(s == 0, 1, s))[:, 0]
    return out


def close(got, want, lax):
    got, want = got.cpu().numpy().astype(np.float64), want
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine])
    bound = (np.broadcast_to(2.0 ** -17 + lax, want.shape) + 2.0 ** -22 * np.abs(np.where(fine, want, 0)))[fine]
    off = np.abs(got[fine] - want[fine])
    assert (off <= bound).all(), float((off / bound).max())


def check(syn, logits, ids=None, n_top=0, scale=1.0, cap=0.0, scales=None, on=None, mask=None):
    import torch
    x = logits.float().cpu().numpy()
    i = None if ids is None else ids.cpu().numpy()
    want = reference(x, i, n_top, scale, cap, None if scales is None else scales.cpu().numpy(), on)
    got = syn.logprobs(logits, ids, n_top, scale=scale, cap=cap, scales=scales, mask=mask)
    torch.cuda.synchronize()
    largest = scale * (1.0 if scales is None else float(scales.max()))
    lax = 2.0 ** -19 * cap * largest
    ts = np.abs(want["log_s"] - want["entropy"])
    close(got.entropy, want["entropy"], lax * (2 + ts) + 2.0 ** -17 * ts)
    if ids is not None:
        close(got.logprob, want["logprob"], lax)
    if n_top:
        assert np.array_equal(got.top.cpu().numpy(), want["top"])
        close(got.top_logprob, want["top_logprob"], lax)
    return got


def bits_of(on):
    """Words of allowed tokens from a truth table (numpy)."""
    import torch
    n, v = on.shape
    words = -(-v // 32)
    padded = np.zeros((n, words * 32), bool)
    padded[:, :v] = on
    return torch.from_numpy(np.packbits(padded, axis=1, bitorder="little").view(np.int32).copy()).cuda()


def rows(rng, n, v, half):
    import torch
    x = (rng.standard_normal((n, v)) * 2.5).astype(np.float32)
    x[np.arange(n), rng.integers(0, v, n)] += 8
    return torch.from_numpy(x.astype(np.float16) if half else x).cuda()


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("n,v", [(1, 1), (3, 2), (2, 31), (5, 777), (1, 16384), (2, 16385), (3, 50257), (1, 128256), (40, 9973),
                                 (400, 4099), (700, 33), (160, 32771)])
def test_shapes(syn, n, v, half):
    import torch
    rng = np.random.default_rng([n, v, half])
    x = rows(rng, n, v, half)
    ids = torch.from_numpy(rng.integers(-1, v, (n, 3)).astype(np.int32)).cuda()
    for n_top in (0, 1, 5, 64):
        check(syn, x, ids, n_top)


@pytest.mark.parametrize("half", [False, True])
def test_rows_that_start_anywhere(syn, half):
    """Odd strides and offsets: 16-byte pieces that begin before a row or end behind it are not its."""
    import torch
    rng = np.random.default_rng(5)
    big = rows(rng, 6, 20011, half)
    big[:, :40] = torch.nan
    big[:, -40:] = torch.inf
    for a, b in ((40, 19971), (41, 19970), (43, 19000), (47, 48), (50, 57)):
        check(syn, big[:, a:b], torch.full((6, 1), b - a - 1, dtype=torch.int32, device="cuda"), 7)
    check(syn, big[1:2, 45:17000], None, 3)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("v", [100, 5000, 40000, 128256])
def test_ties_go_to_the_lowest_token(syn, v, half):
    import torch
    rng = np.random.default_rng(v)
    t = torch.float16 if half else torch.float32
    same = torch.zeros((2, v), dtype=t, device="cuda")
    same[1, ::2] = -0.0  # (which is as large as 0)
    check(syn, same, None, 64)
    few = torch.from_numpy(rng.integers(-2, 3, (9, v)).astype(np.float32)).cuda().to(t)
    check(syn, few, None, 64)
    check(syn, few, None, 1)
    one = torch.full((1, v), -3.0, dtype=t, device="cuda")
    one[0, v // 3:v // 3 + 40] = 5.0
    one[0, v // 2] = 6.0
    check(syn, one, None, 50)


@pytest.mark.parametrize("down", [False, True])
def test_ordered_rows(syn, down):
    """The largest in one thread's, one CTA's, the last piece's logits."""
    import torch
    x = torch.linspace(-9, 4, 128256, device="cuda")
    x = (x.flip(0) if down else x).view(1, -1)
    check(syn, x.repeat(2, 1), None, 64)
    check(syn, x.repeat(200, 1), None, 20)
    check(syn, x.repeat(700, 1)[:, :40000].contiguous(), None, 20)


@pytest.mark.parametrize("n", [2, 90, 320])
def test_mask_scales_and_cap(syn, n):
    import torch
    rng = np.random.default_rng(n)
    for v, half, cap in ((50257, False, 30.0), (50257, True, 0.0), (4096, False, 5.0), (33, False, 0.0)):
        x = rows(rng, n, v, half)
        on = rng.random((n, v)) < rng.random((n, 1)) ** 3
        on[0] = False
        on[1] = False
        on[1, v // 2] = True
        hidden = torch.from_numpy(~on).cuda()
        x = torch.where(hidden & (torch.rand(x.shape, device="cuda") < 0.3), torch.tensor(torch.nan, device="cuda"), x.float()).to(x.dtype)
        x = torch.where(hidden & (torch.rand(x.shape, device="cuda") < 0.3), torch.tensor(torch.inf, device="cuda"), x.float()).to(x.dtype)
        scales = torch.from_numpy(rng.uniform(0.25, 2, n).astype(np.float32)).cuda()
        ids = torch.from_numpy(rng.integers(-1, v, (n, 2)).astype(np.int32)).cuda()
        ids[1, 0] = v // 2
        wide = torch.full((n, -(-v // 32) + 5), -1, dtype=torch.int32, device="cuda")
        wide[:, :-(-v // 32)] = bits_of(on)
        for mask in (bits_of(on), wide):
            check(syn, x, ids, 9, scale=0.5, cap=cap, scales=scales, on=on, mask=mask)
        if v > 100:  # rows that do not start on a piece's boundary
            check(syn, x[:, 3:], ids.clamp(max=v - 4), 9, cap=cap, on=on[:, 3:], mask=bits_of(on[:, 3:]))


def test_infinities_and_nan(syn):
    import torch
    for v in (40, 20000, 128256):
        x = torch.randn((7, v), device="cuda")
        x[0, 5] = torch.nan
        x[1, v - 1] = torch.inf
        x[2] = -torch.inf
        x[3, 1:] = -torch.inf
        x[4, ::2] = -torch.inf
        x[5] = -3e38
        x[5, 7] = 3e38
        ids = torch.tensor([[7], [7], [7], [0], [2], [7], [v - 1]], dtype=torch.int32, device="cuda")
        got = syn.logprobs(x, ids, 3)
        for y in (got.logprob, got.entropy[:, None], got.top_logprob):
            assert torch.isnan(y[:2]).all() and not torch.isnan(y[2:]).any()
        assert (got.top[:3] == -1).all() and (got.top_logprob[2] == -torch.inf).all() and got.logprob[2, 0] == -torch.inf
        assert got.entropy[2] == 0 and got.entropy[3] == 0 and got.logprob[3, 0] == 0 and got.top[3].tolist() == [0, -1, -1]
        assert got.logprob[4, 0] == -torch.inf and got.entropy[5] == 0 and got.logprob[5, 0] == 0 and got.top[5, 0] == 7
        check(syn, x[6:], ids[6:], 3)
        for bad in (0.0, -1.0, torch.inf, torch.nan):
            got = syn.logprobs(x[6:], ids[6:], 3, scales=torch.tensor([bad], device="cuda"))
            assert torch.isnan(got.logprob).all() and torch.isnan(got.entropy).all() and (got.top == -1).all()


def test_ids_outside_the_vocabulary(syn):
    import torch
    x = torch.randn((2, 1000), device="cuda")
    ids = torch.tensor([[-1, -5, 3], [999, -(2 ** 31), 0]], dtype=torch.int32, device="cuda")
    check(syn, x, ids, 0)
    assert syn.device_status() == syn.OK
    ids[0, 1] = 1000
    got = syn.logprobs(x, ids)
    assert got.logprob[0, 1] == 0
    assert syn.device_status() == syn.ERR_BOUNDS
    check(syn, x, x.argmax(1).to(torch.int32)[:, None])
    assert syn.logprobs(x, x.argmax(1).to(torch.int32)).logprob.shape == (2,)


def test_rows_on_their_own(syn):
    """Deterministic mode: a row's bits do not depend on the others or the SMs; and a call repeats its bits in any mode."""
    import torch
    rng = np.random.default_rng(3)
    x = rows(rng, 170, 50257, False)
    ids = torch.zeros((170, 1), dtype=torch.int32, device="cuda")
    a, b = syn.logprobs(x, ids, 5), syn.logprobs(x, ids, 5)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    old = syn.set_deterministic(True)
    lim = syn.set_sm_limit(0)
    try:
        want = syn.logprobs(x, ids, 5)
        for n in (1, 3, 40):
            got = syn.logprobs(x[:n], ids[:n], 5)
            assert all(torch.equal(p[:n], q) for p, q in zip(want, got))
        syn.set_sm_limit(5)
        got = syn.logprobs(x, ids, 5)
        assert all(torch.equal(p, q) for p, q in zip(want, got))
    finally:
        syn.set_deterministic(old)
        syn.set_sm_limit(lim)
    lim = syn.set_sm_limit(2)
    try:
        check(syn, x[:9], ids[:9], 64)
    finally:
        syn.set_sm_limit(lim)


def test_captured_and_on_another_stream(syn):
    import torch
    rng = np.random.default_rng(4)
    x, ids = rows(rng, 3, 128256, False), torch.zeros((3, 1), dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step = syn.prepare_logprobs(x, ids, 5)
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
        for seed in (1, 2):
            x.copy_(rows(np.random.default_rng(seed), 3, 128256, False))
            ids.fill_(seed)
            graph.replay()
            graph.replay()
            side.synchronize()
            want = reference(x.cpu().numpy(), ids.cpu().numpy(), 5)
            assert np.array_equal(got.top.cpu().numpy(), want["top"])
            close(got.logprob, want["logprob"], 0)
