"""The operators of speculative decoding in the checking builds: every index check of the debug build passes and the
results are those of the product build; in the stall build, whose attention never receives a tile, the waits run out and
are reported, and the device stays usable."""
import ctypes

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F16, Q8_0 = 7, 1


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _case(syn, t, dim, seed=1):
    rng = np.random.default_rng(seed)
    cache = syn.KVCache.empty(t, 2, dim, 16, 200)
    if t == F16:
        cache.k.normal_()
        cache.v.normal_()
    else:
        cache.k.random_(0, 60)
        cache.v.random_(0, 60)
    lens, new = [900, 33, 400], [20, 33, 70]
    pages = torch.randperm(200, device="cuda")[:3 * 57].view(3, 57).to(torch.int32)
    parents = _i32([int(rng.integers(-1, i)) if i else -1 for n in new for i in range(n)])
    q = torch.randn((sum(new), 8, dim), device="cuda").half()
    return cache, q, _i32([0, 20, 53, 123]), parents, pages, _i32(lens)


def _tree(lib, syn, case, out):
    cache, q, starts, parents, pages, lens = case
    d = syn.AttnDesc(q.shape[1], 0, q.shape[2] ** -0.5, 0.0, None, None, None, 0, 0, syn.OUT_F32)
    return lib.syn_attn_tree(ctypes.byref(cache.desc), ctypes.byref(d), 3, q.shape[0], q.data_ptr(), starts.data_ptr(),
                             parents.data_ptr(), pages.data_ptr(), pages.shape[1], lens.data_ptr(), out.data_ptr(), _stream())


@pytest.mark.parametrize("t,dim", [(F16, 64), (F16, 128), (Q8_0, 128), (F16, 256), (Q8_0, 256)])
def test_tree_in_the_debug_build(t, dim):
    from gguf_block_quantized_gb300 import build, syn
    dbg = syn.bind(build.build(variant="debug"))
    dbg.syn_device_status(1)
    case = _case(syn, t, dim)
    a, b = (torch.empty(case[1].shape, device="cuda") for _ in range(2))
    assert _tree(dbg, syn, case, a) == syn.OK and _tree(syn, syn, case, b) == syn.OK
    assert dbg.syn_device_status(1) == syn.OK and syn.device_status() == syn.OK
    assert torch.equal(a, b)


def test_pages_and_logprobs_in_the_debug_build():
    from gguf_block_quantized_gb300 import build, syn
    dbg = syn.bind(build.build(variant="debug"))
    dbg.syn_device_status(1)
    c, s = syn.KVCache.empty(Q8_0, 2, 64, 16, 600), _stream()
    refs, pages, lens = torch.zeros(600, dtype=torch.int32, device="cuda"), torch.full((2, 300), -1, dtype=torch.int32, device="cuda"), _i32([0, 0])
    starts, slots = _i32([0, 4500, 4533]), torch.empty(4533, dtype=torch.int64, device="cuda")
    rows = torch.arange(1, 4500, dtype=torch.int32, device="cuda")
    keep, out = _i32([0, 4499, 4499]), torch.empty(2, dtype=torch.int32, device="cuda")
    args = (ctypes.byref(c.desc), refs.data_ptr())
    assert dbg.syn_kv_extend(*args, 2, 4533, pages.data_ptr(), 300, lens.data_ptr(), starts.data_ptr(), lens.data_ptr(), slots.data_ptr(), s) == syn.OK
    zero = _i32([0, 0])
    assert dbg.syn_kv_compact(*args, 2, 4499, pages.data_ptr(), 300, zero.data_ptr(), keep.data_ptr(), rows.data_ptr(), out.data_ptr(), s) == syn.OK
    assert dbg.syn_kv_trim(*args, 2, pages.data_ptr(), 300, out.data_ptr(), s) == syn.OK
    x, y = torch.randn((3, 5001), device="cuda"), torch.empty(3, device="cuda")
    opt = syn.LogitsDesc(0, 1.0, 0.0, None, None, 0, 0)
    assert dbg.syn_logprobs(ctypes.byref(opt), 3, 5001, x.data_ptr(), 0, None, None, y.data_ptr(), 0, None, None, s) == syn.OK
    assert dbg.syn_device_status(1) == syn.OK
    assert out.tolist() == [4499, 0] and int(refs.sum()) == 282 and (slots >= 0).all()


@pytest.mark.parametrize("t,dim", [(F16, 128), (Q8_0, 64), (F16, 256)])
def test_waits_that_run_out(t, dim):
    from gguf_block_quantized_gb300 import build, syn
    stall = syn.bind(build.build(variant="stall"))
    stall.syn_device_status(1)
    case = _case(syn, t, dim)
    out = torch.empty(case[1].shape, device="cuda")
    want = syn.attn_tree(*case)
    for _ in range(2):
        assert _tree(stall, syn, case, out) == syn.OK
        assert stall.syn_device_status(1) == syn.ERR_TIMEOUT and stall.syn_device_status(1) == syn.OK
    assert torch.equal(syn.attn_tree(*case), want) and syn.device_status() == syn.OK
