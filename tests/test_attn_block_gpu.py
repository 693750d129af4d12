"""The attention block (products, append, attention, product) on the GPU, and the paged-cache
operators in the checking builds of the library."""
import os
import sys

import numpy as np
import pytest

import oracle
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_ref  # noqa: E402
from test_attn_gpu import make_cache, prefill_bound, decode_bound, reference  # noqa: E402

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F16, Q8_0 = 7, 1


# The products are within 1e-4 |x| |w| of exact ones (the library's tolerance) in either form, fp16 rounds
# q, k, v and p to 2^-11 each: the two forms of a token differ by a few 2^-11 of the largest output at the
# most, where each value is a mean over 2048 products.  Q8_0: the codes of a cached row can differ by one
# unit (1 / 127 of its block's largest value) where the two forms' products straddle a code's edge.
@pytest.mark.parametrize("t,bound", [(F16, 8 * 2.0 ** -11), (Q8_0, 8 * 2.0 ** -11 + 2.0 / 127)])
@pytest.mark.parametrize("prompt,steps,seqs", [(70, 3, 2), (300, 2, 1)])
def test_block_forms_agree(t, bound, prompt, steps, seqs):
    from gguf_block_quantized_gb300 import attn_block
    r = attn_block.run(t, prompt, steps, seqs)
    assert r["difference"] <= bound


def test_block_against_plain_form():
    """The whole block against the products' definition (the oracle's: converted activations) and
    64-bit attention, to the sum of its parts' tolerances: 2^-7 of the largest output (products
    1e-4 |x| |w| three times deep, fp16 2^-11)."""
    from gguf_block_quantized_gb300 import attn_block
    n, heads, kv, dim = 33, 32, 8, 64
    block, pages, slots = attn_block.llama1b_block(F16, 1, n, page=16)
    rng = np.random.default_rng(3)
    x = rng.standard_normal((n, 2048)).astype(np.float32)
    out = torch.empty((n, 2048), device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    block.prepare_prompt(torch.from_numpy(x).cuda(), out, pos, slots.view(-1), torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                         pages, torch.tensor([n], dtype=torch.int32, device="cuda"))()
    def product(name, y):
        t, blocks, n_out, n_in = block.w[name]
        return oracle.mul_mat(t, blocks.cpu().numpy(), n_out, n_in, y.astype(np.float32)).astype(np.float64)

    def rotated(y, h):
        return attn_ref.rotate(y.reshape(n, h, dim), np.arange(n)[None], dim, 500000.0, 0)

    q, k, v = rotated(product("q", x), heads), rotated(product("k", x), kv), product("v", x).reshape(n, kv, dim)
    y, _ = attn_ref.attention(q, k, v, np.arange(n), np.zeros(n), 0, 0, dim ** -0.5, 0.0, None)
    want = product("output", y.reshape(n, -1))
    assert np.abs(out.double().cpu().numpy() - want).max() <= 2.0 ** -7 * np.abs(want).max()


# ---- the checking builds -------------------------------------------------------------------

def _stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.fixture(scope="module")
def libs():
    from gguf_block_quantized_gb300 import build, syn
    return syn, {v: syn.bind(build.build(variant=v)) for v in ("debug", "stall")}


def _through(lib, prepared):
    """A prepared call's arguments through another build of the library."""
    rc = getattr(lib, prepared._name)(*prepared._args)
    assert rc == 0, lib.syn_strerror(rc).decode()
    return prepared._result


def _tokens(rng, n, heads, kv, dim):
    x = torch.from_numpy(rng.standard_normal((n, heads + 2 * kv, dim)).astype(np.float32)).cuda()
    return x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]


@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("heads,kv,dim,page", [(8, 2, 64, 16), (5, 1, 96, 8), (16, 2, 128, 64), (3, 1, 160, 32), (8, 1, 256, 256)])
def test_every_index_check_passes(libs, t, heads, kv, dim, page):
    """Append, read, decode and prefill with ragged sizes in the build whose kernels check their indices."""
    syn, lib = libs[0], libs[1]["debug"]
    lib.syn_device_status(1)
    rng = np.random.default_rng([t, heads, dim])
    lens, new = [1, 40, 300, 0, 129], [1, 33, 150, 0, 2]
    cache, pages, seqs = make_cache(syn, rng, t, kv, dim, page, lens)
    n = 77
    q, k, v = _tokens(rng, n, heads, kv, dim)
    other = syn.KVCache.empty(t, kv, dim, page, -(-100 // page))
    slots = torch.from_numpy(rng.permutation(100)[:n].astype(np.int64)).cuda()
    rope = syn.Rope(dim - 32 if dim > 64 else dim, layout=syn.ROPE_HALVES)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    got = _through(lib, syn.prepare_kv_append(other, rope, k, v, pos, slots, q=q))
    rk, rv = _through(lib, syn.prepare_kv_read(other, slots))
    mine = syn.KVCache.empty(t, kv, dim, page, other.n_pages)
    want = syn.kv_append(mine, rope, k, v, pos, slots, q=q)
    assert torch.equal(got, want) and torch.equal(mine.k, other.k) and torch.equal(mine.v, other.v)
    wk, wv = syn.kv_read(mine, slots)
    assert torch.equal(rk, wk) and torch.equal(rv, wv)
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qs = torch.from_numpy(rng.standard_normal((5, heads, dim)).astype(np.float16)).cuda()
    got = _through(lib, syn.prepare_attn_decode(cache, qs, pages, ld)).double().cpu().numpy()
    ref, size = reference(qs.cpu().numpy(), seqs, [np.arange(x - 1, x) if x else np.array([-1]) for x in lens], [np.zeros(1)] * 5,
                          [0] * 5, 0, dim ** -0.5, 0.0, None)
    assert (np.abs(got - ref) <= decode_bound(size, ref, False)).all()
    starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    qs = torch.from_numpy(rng.standard_normal((sum(new), heads, dim)).astype(np.float16)).cuda()
    got = _through(lib, syn.prepare_attn_prefill(cache, qs, starts, pages, ld)).double().cpu().numpy()
    ref, size = reference(qs.cpu().numpy(), seqs, [np.arange(x - m, x) for x, m in zip(lens, new)], [np.zeros(m) for m in new], [0] * 5,
                          0, dim ** -0.5, 0.0, None)
    vmax = max(np.abs(v).max() for _, v in seqs if v.size)
    assert (np.abs(got - ref) <= prefill_bound(t, size, vmax, ref, False)).all()
    st = lib.syn_device_status(1)
    assert st == syn.OK, lib.syn_strerror(st).decode()


def test_index_checks_cover_the_expanded_cache_and_splits(libs):
    syn, lib = libs[0], libs[1]["debug"]
    lib.syn_device_status(1)
    rng = np.random.default_rng(5)
    for t, lens, new in ((Q8_0, [700, 330], [300, 300]), (F16, [9000], [3])):
        cache, pages, _ = make_cache(syn, rng, t, 1, 64, 16, lens)
        starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q = torch.from_numpy(rng.standard_normal((sum(new), 8, 64)).astype(np.float16)).cuda()
        slopes = torch.full((8,), 0.01, device="cuda")
        p = syn.prepare_attn_prefill(cache, q, starts, pages, ld, slopes=slopes)
        got = _through(lib, p).clone()
        assert torch.equal(p(), got)
        one = torch.from_numpy(rng.standard_normal((len(lens), 8, 64)).astype(np.float16)).cuda()
        d = syn.prepare_attn_decode(cache, one, pages, ld, slopes=slopes)
        got = _through(lib, d).clone()
        assert (d() - got).abs().max().item() < 1e-5
    st = lib.syn_device_status(1)
    assert st == syn.OK, lib.syn_strerror(st).decode()


@pytest.mark.parametrize("t", [F16, Q8_0])
@pytest.mark.parametrize("dim", [64, 256])
def test_waits_that_run_out_are_reported(libs, t, dim):
    """In the build whose loads are never issued, append and prefill give up, report it and leave the
    device usable (and the counters of the calls to come at zero)."""
    syn, lib = libs[0], libs[1]["stall"]
    lib.syn_device_status(1)
    rng = np.random.default_rng(6)
    lens, new = [300, 2000], [100, 3]
    cache, pages, seqs = make_cache(syn, rng, t, 2, dim, 16, lens)
    q, k, v = _tokens(rng, 50, 4, 2, dim)
    other = syn.KVCache.empty(t, 2, dim, 16, 4)
    slots = torch.arange(50, device="cuda")
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 100, 103], dtype=torch.int32, device="cuda")
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qs = torch.from_numpy(rng.standard_normal((103, 4, dim)).astype(np.float16)).cuda()
    a = syn.prepare_kv_append(other, syn.Rope(dim), k, v, pos, slots, q=q)
    p = syn.prepare_attn_prefill(cache, qs, starts, pages, ld)
    for call in (a, p, p):
        _through(lib, call)
        assert lib.syn_device_status(1) == syn.ERR_TIMEOUT, call._name
        assert lib.syn_device_status(1) == syn.OK
    # decode waits for nothing but its own copies: it runs as ever, and so do the normal library's calls
    one = torch.from_numpy(rng.standard_normal((2, 4, dim)).astype(np.float16)).cuda()
    d = syn.prepare_attn_decode(cache, one, pages, ld)
    ref, size = reference(one.cpu().numpy(), seqs, [np.array([x - 1]) for x in lens], [np.zeros(1)] * 2, [0] * 2, 0, dim ** -0.5, 0.0, None)
    assert (np.abs(_through(lib, d).double().cpu().numpy() - ref) <= decode_bound(size, ref, False)).all()
    assert lib.syn_device_status(1) == syn.OK
    got = p().double().cpu().numpy()
    ref, size = reference(qs.cpu().numpy(), seqs, [np.arange(x - m, x) for x, m in zip(lens, new)], [np.zeros(m) for m in new], [0] * 2,
                          0, dim ** -0.5, 0.0, None)
    vmax = max(np.abs(v).max() for _, v in seqs)
    assert (np.abs(got - ref) <= prefill_bound(t, size, vmax, ref, False)).all()
    assert syn.device_status() == syn.OK
