"""Pages and log probabilities in the checking builds: in the debug build every index check passes and results are those of
the product build; in the stall build, where no chunk of a long list says that it is loaded, the waits run out and are reported,
and the next call finds its counters as they should be."""
import ctypes
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F16, Q8_0 = 7, 1


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def stream():
    return torch.cuda.current_stream().cuda_stream


def random_cache(syn, t, kv, dim, page, n_pages, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    shape = (n_pages, kv, page, dim * 2) if t == F16 else (n_pages, kv, page * dim // 16 * 17)
    pools = [torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=gen) for _ in range(2)]
    return syn.KVCache(t, kv, dim, page, *(p.view(torch.float16) if t == F16 else p for p in pools)), pools


@pytest.fixture(scope="module")
def libs():
    from gguf_block_quantized_gb300 import build, syn
    dbg = syn.bind(build.build(variant="debug"))
    dbg.syn_device_status(1)
    syn.device_status()
    return syn, dbg


@pytest.mark.parametrize("t,kv,dim,page", [(F16, 2, 64, 16), (F16, 3, 96, 8), (F16, 1, 256, 64), (Q8_0, 2, 64, 16), (Q8_0, 5, 160, 8),
                                           (Q8_0, 8, 128, 64)])
@pytest.mark.parametrize("lens", [[40, 0, 17, 300], [2100], [1, 3000, 700, 5000]])
def test_a_run_of_calls_in_the_debug_build(libs, t, kv, dim, page, lens):
    """extend, fork, extend of shared pages (copied), compact (short and long lists), trim, copy."""
    syn, dbg = libs
    n, new = len(lens), np.array([5, 1, 2 * page, 3])[:len(lens)]
    width = -(-(max(lens) + 2 * page) // page) + 1
    n_pages, results = 2 * n * width, []
    for lib in (dbg, syn):
        rng = np.random.default_rng([kv, dim, n])
        cache, pools = random_cache(syn, t, kv, dim, page, n_pages, 3)
        c, s = ctypes.byref(cache.desc), stream()
        refs, pages, ln = torch.zeros(n_pages, dtype=torch.int32, device="cuda"), torch.full((n, width), -1, dtype=torch.int32, device="cuda"), i32([0] * n)
        first, second = i32(np.concatenate([[0], np.cumsum(lens)])), i32(np.concatenate([[0], np.cumsum(new)]))
        slots, slots2 = (torch.empty(int(x[-1]), dtype=torch.int64, device="cuda") for x in (first, second))
        fork, fork_ln = torch.empty_like(pages), torch.empty_like(ln)
        keep = [np.sort(rng.permutation(int(m))[:int(0.7 * m)]) for m in lens]
        starts, rows = i32(np.concatenate([[0], np.cumsum([len(k) for k in keep])])), i32(np.concatenate(keep))
        source, zero, out = i32([n - 1 - i for i in range(n)]), i32([0] * n), torch.empty_like(ln)
        src, dst = i32([0, 1]), i32([n_pages - 1, n_pages - 2])
        assert lib.syn_kv_extend(c, refs.data_ptr(), n, slots.numel(), pages.data_ptr(), width, ln.data_ptr(), first.data_ptr(), ln.data_ptr(),
                                 slots.data_ptr(), s) == syn.OK
        assert lib.syn_kv_fork(c, refs.data_ptr(), n, pages.data_ptr(), width, ln.data_ptr(), n, source.data_ptr(), fork.data_ptr(),
                               fork_ln.data_ptr(), s) == syn.OK
        assert lib.syn_kv_extend(c, refs.data_ptr(), n, slots2.numel(), fork.data_ptr(), width, fork_ln.data_ptr(), second.data_ptr(),
                                 fork_ln.data_ptr(), slots2.data_ptr(), s) == syn.OK
        zeros = torch.zeros_like(ln)
        assert lib.syn_kv_trim(c, refs.data_ptr(), n, fork.data_ptr(), width, zeros.data_ptr(), s) == syn.OK
        assert lib.syn_kv_compact(c, refs.data_ptr(), n, rows.numel(), pages.data_ptr(), width, zero.data_ptr(), starts.data_ptr(),
                                  rows.data_ptr(), out.data_ptr(), s) == syn.OK
        assert lib.syn_kv_trim(c, refs.data_ptr(), n, pages.data_ptr(), width, out.data_ptr(), s) == syn.OK
        assert lib.syn_kv_copy(c, c, 2, src.data_ptr(), dst.data_ptr(), s) == syn.OK
        assert lib.syn_device_status(1) == syn.OK
        results.append([refs, pages, out, slots, slots2, fork, fork_ln, *pools])
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("n,v,half", [(1, 128256, False), (3, 50257, True), (330, 128256, False), (330, 20011, True), (200, 900, False), (2, 1, True)])
def test_logprobs_in_the_debug_build(libs, n, v, half):
    syn, dbg = libs
    gen = torch.Generator(device="cuda").manual_seed(v)
    x = torch.randn((n, v + 3), device="cuda", generator=gen).to(torch.float16 if half else torch.float32)[:, 3:]
    mask = torch.randint(-2 ** 31, 2 ** 31, (n, -(-v // 32)), dtype=torch.int32, device="cuda", generator=gen)
    ids = torch.randint(-1, v, (n, 3), dtype=torch.int32, device="cuda", generator=gen)
    for cap, on, top in ((0.0, None, 0), (0.0, None, 64), (20.0, mask, 9)):
        opt = syn.LogitsDesc(int(half), 1.0, cap, None, None if on is None else on.data_ptr(), v + 3, 0)
        out = []
        for lib in (dbg, syn):
            p, e, best, q = (torch.full(s, 7, dtype=d, device="cuda") for s, d in (((n, 3), torch.float32), ((n,), torch.float32),
                                                                                 ((n, max(top, 1)), torch.int32), ((n, max(top, 1)), torch.float32)))
            assert lib.syn_logprobs(ctypes.byref(opt), n, v, x.data_ptr(), 3, ids.data_ptr(), p.data_ptr(), e.data_ptr(), top, best.data_ptr(),
                                    q.data_ptr(), stream()) == syn.OK
            assert lib.syn_device_status(1) == syn.OK
            out.append((p, e, best, q))
        for a, b in zip(*out):
            assert torch.equal(a.view(torch.int32), b.view(torch.int32))


def test_waits_of_a_long_list_run_out():
    from gguf_block_quantized_gb300 import build, syn
    stall = syn.bind(build.build(variant="stall"))
    stall.syn_device_status(1)
    page, n = 16, 6000
    rows, starts, base = i32(np.arange(1, n)), i32([0, n - 1]), i32([0])
    table, out = torch.randperm(n // page, device="cuda")[None].to(torch.int32), torch.empty(1, dtype=torch.int32, device="cuda")
    for _ in range(2):
        cache, pools = random_cache(syn, F16, 2, 64, page, n // page, 1)
        assert stall.syn_kv_compact(ctypes.byref(cache.desc), None, 1, n - 1, table.data_ptr(), n // page, base.data_ptr(), starts.data_ptr(),
                                    rows.data_ptr(), out.data_ptr(), stream()) == syn.OK
        assert stall.syn_device_status(1) == syn.ERR_TIMEOUT and stall.syn_device_status(1) == syn.OK
        assert out.item() == n - 1
        # the product library, on the same device
        cache, pools = random_cache(syn, F16, 2, 64, page, n // page, 2)
        before = [p[table[0].long()].transpose(1, 2).flatten(0, 1).clone() for p in pools]  # rows in order
        syn.kv_compact(cache, None, table, base, starts, rows)
        for p, x in zip(pools, before):
            assert torch.equal(p[table[0].long()].transpose(1, 2).flatten(0, 1)[:n - 1], x[1:])
        assert syn.device_status() == syn.OK
