"""What the paged-cache entry points refuse, and their host functions.  CPU only: every check here
answers before a GPU is touched."""
import ctypes
import math

import numpy as np
import pytest

F16, Q8_0 = 7, 1
P = 1 << 20  # any aligned non-null value
LAST = 2 ** 62


@pytest.fixture(scope="module")
def syn():
    import torch  # noqa: F401
    from gguf_block_quantized_gb300 import build
    build.build()
    from gguf_block_quantized_gb300 import syn
    return syn


def cache(syn, **kw):
    c = dict(type=F16, n_kv_heads=2, head_dim=64, page_size=16, n_pages=4, k=P, v=P, page_stride=0)
    c.update(kw)
    return syn.KVCacheDesc(*c.values())


def rope(syn, **kw):
    r = dict(n_rot=64, layout=1, n_axes=1, magnitude=1.0, turns=P, axis=None)
    r.update(kw)
    return syn.RopeDesc(*r.values())


def attn(syn, **kw):
    a = dict(n_heads=4, window=0, scale=0.125, cap=0.0, slopes=None, prefix=None, first=None, q_stride=0, out_stride=0,
             out_type=0)
    a.update(kw)
    return syn.AttnDesc(*a.values())


def append(syn, c=None, r=None, **kw):
    a = dict(n_tok=3, q=P, q_stride=0, n_heads=4, q_out=P, k=P, k_stride=0, v=P, v_stride=0, pos=P, slots=P)
    a.update(kw)
    return syn.syn_kv_append(c or cache(syn), r or rope(syn), *a.values(), None)


def decode(syn, c=None, d=None, **kw):
    a = dict(n_seq=2, q=P, pages=P, max_pages=2, lens=P, out=P)
    a.update(kw)
    return syn.syn_attn_decode(c or cache(syn), d or attn(syn), *a.values(), None)


def prefill(syn, c=None, d=None, **kw):
    a = dict(n_seq=2, n_tok=9, q=P, starts=P, pages=P, max_pages=2, lens=P, out=P)
    a.update(kw)
    return syn.syn_attn_prefill(c or cache(syn), d or attn(syn), *a.values(), None)


def test_tile_bytes(syn):
    assert syn.syn_kv_tile_bytes(F16, 64, 16) == 16 * 64 * 2
    assert syn.syn_kv_tile_bytes(Q8_0, 96, 8) == 8 * (96 + 3 * 2)
    for t, dim, page in [(2, 64, 16), (0, 64, 16), (F16, 48, 16), (F16, 0, 16), (F16, 288, 16), (F16, 64, 4), (F16, 64, 24),
                         (Q8_0, 64, 131072), (Q8_0, 64, 0), (Q8_0, -64, 16)]:
        assert syn.syn_kv_tile_bytes(t, dim, page) == -1, (t, dim, page)


@pytest.mark.parametrize("n_rot,base,scale,factors", [(8, 10000.0, 1.0, None), (64, 500000.0, 0.25, None),
                                                      (128, 1e6, 1.0, "some"), (8, 1.0, -3.7, None)])
def test_rope_turns(syn, n_rot, base, scale, factors):
    """Turns per position to 2^-52 of themselves (the double they are made from), whole turns off."""
    f = None if factors is None else (1 + np.arange(n_rot // 2, dtype=np.float32) / 7).astype(np.float32)
    out = np.zeros(n_rot // 2, np.uint64)
    assert syn.syn_rope_turns(n_rot, base, scale, None if f is None else f.ctypes.data, out.ctypes.data) == syn.OK
    for i in range(n_rot // 2):
        want = scale * base ** (-2.0 * i / n_rot) / (1.0 if f is None else float(f[i])) / (2 * math.pi)
        d = int(out[i]) / 2.0 ** 64 - (want - math.floor(want))
        assert abs(d - round(d)) <= 2.0 ** -50 * max(1.0, abs(want))


def test_rope_turns_refusals(syn):
    out = np.zeros(4, np.uint64)
    f = np.ones(4, np.float32)
    call = lambda n=8, base=1e4, scale=1.0, fac=None, o=out: syn.syn_rope_turns(  # noqa: E731
        n, base, scale, None if fac is None else fac.ctypes.data, None if o is None else o.ctypes.data)
    assert call(0, o=None) == syn.OK
    for kw in ({"n": -8}, {"n": 12}, {"n": 264}, {"base": 0.0}, {"base": math.inf}, {"base": math.nan}, {"scale": math.nan},
               {"scale": -math.inf}):
        assert call(**kw) == syn.ERR_SHAPE, kw
    for bad in (0.0, math.inf, math.nan):
        g = f.copy()
        g[3] = bad
        assert call(fac=g) == syn.ERR_RANGE
    assert call(o=None) == syn.ERR_NULL


CACHES = [({"type": 2}, "TYPE"), ({"type": 0}, "TYPE"), ({"head_dim": 48}, "SHAPE"), ({"head_dim": 512}, "SHAPE"),
          ({"page_size": 12}, "SHAPE"), ({"page_size": 4}, "SHAPE"), ({"n_kv_heads": 0}, "SHAPE"), ({"n_kv_heads": 2000}, "SHAPE"),
          ({"n_pages": 0}, "SHAPE"), ({"n_pages": 1 << 31}, "SHAPE"), ({"page_stride": 2 * 16 * 64 * 2 - 16}, "SHAPE"),
          ({"page_stride": 2 * 16 * 64 * 2 + 8}, "SHAPE"), ({"page_stride": -16}, "SHAPE"), ({"page_stride": LAST}, "SHAPE"),
          ({"k": None}, "NULL"), ({"v": None}, "NULL"), ({"k": P + 8}, "ALIGN"), ({"v": P + 2}, "ALIGN")]


@pytest.mark.parametrize("kw,err", CACHES)
def test_every_call_checks_the_cache(syn, kw, err):
    c = cache(syn, **kw)
    want = getattr(syn, "ERR_" + err)
    assert append(syn, c) == want and decode(syn, c) == want and prefill(syn, c) == want
    assert syn.syn_kv_read(c, 3, P, P, P, None) == want


def test_null_structures(syn):
    assert syn.syn_kv_append(None, rope(syn), 1, P, 0, 4, P, P, 0, P, 0, P, P, None) == syn.ERR_NULL
    assert syn.syn_kv_append(cache(syn), None, 1, P, 0, 4, P, P, 0, P, 0, P, P, None) == syn.ERR_NULL
    assert syn.syn_attn_decode(cache(syn), None, 1, P, P, 1, P, P, None) == syn.ERR_NULL
    assert syn.syn_attn_prefill(None, attn(syn), 1, 1, P, P, P, 1, P, P, None) == syn.ERR_NULL
    assert syn.syn_kv_read(None, 1, P, P, P, None) == syn.ERR_NULL


@pytest.mark.parametrize("kw,err", [
    ({"layout": 2}, "TYPE"), ({"layout": -1}, "TYPE"), ({"n_rot": 72}, "SHAPE"), ({"n_rot": 12}, "SHAPE"), ({"n_rot": -8}, "SHAPE"),
    ({"n_axes": 0}, "SHAPE"), ({"n_axes": 9}, "SHAPE"), ({"magnitude": math.inf}, "SHAPE"), ({"magnitude": math.nan}, "SHAPE"),
    ({"turns": None}, "NULL"), ({"turns": P + 4}, "ALIGN")])
def test_append_checks_the_rotation(syn, kw, err):
    assert append(syn, r=rope(syn, **kw)) == getattr(syn, "ERR_" + err)


@pytest.mark.parametrize("kw,err", [
    ({"n_tok": -1}, "SHAPE"), ({"n_tok": 1 << 31}, "SHAPE"), ({"n_heads": -1}, "SHAPE"), ({"n_heads": 1025}, "SHAPE"),
    ({"k_stride": 124}, "SHAPE"), ({"v_stride": 130}, "SHAPE"), ({"q_stride": 252}, "SHAPE"), ({"q_stride": 258}, "SHAPE"),
    ({"k_stride": LAST}, "SHAPE"), ({"v_stride": LAST}, "SHAPE"), ({"q_stride": LAST}, "SHAPE"), ({"k_stride": -128}, "SHAPE"),
    ({"k": None}, "NULL"), ({"v": None}, "NULL"), ({"slots": None}, "NULL"), ({"q": None}, "NULL"), ({"q_out": None}, "NULL"),
    ({"pos": None}, "NULL"), ({"k": P + 4}, "ALIGN"), ({"v": P + 8}, "ALIGN"), ({"q": P + 4}, "ALIGN"), ({"q_out": P + 2}, "ALIGN"),
    ({"slots": P + 4}, "ALIGN"), ({"pos": P + 2}, "ALIGN")])
def test_append_refusals(syn, kw, err):
    assert append(syn, **kw) == getattr(syn, "ERR_" + err)


def test_calls_of_nothing(syn):
    assert append(syn, n_tok=0, q=None, q_out=None, k=None, v=None, pos=None, slots=None) == syn.OK
    assert syn.syn_kv_read(cache(syn), 0, None, None, None, None) == syn.OK
    assert decode(syn, n_seq=0) == syn.OK
    assert prefill(syn, n_seq=0, n_tok=0) == syn.OK and prefill(syn, n_tok=0) == syn.OK


@pytest.mark.parametrize("args,err", [((-1, P, P, P), "SHAPE"), ((LAST, P, P, P), "SHAPE"), ((3, None, P, P), "NULL"),
                                      ((3, P, None, P), "NULL"), ((3, P, P, None), "NULL"), ((3, P + 4, P, P), "ALIGN"),
                                      ((3, P, P + 8, P), "ALIGN"), ((3, P, P, P + 2), "ALIGN")])
def test_read_refusals(syn, args, err):
    assert syn.syn_kv_read(cache(syn), *args, None) == getattr(syn, "ERR_" + err)


@pytest.mark.parametrize("kw,err", [
    ({"out_type": 2}, "TYPE"), ({"out_type": -1}, "TYPE"), ({"n_heads": 0}, "SHAPE"), ({"n_heads": 3}, "SHAPE"),
    ({"n_heads": 1026}, "SHAPE"), ({"window": -1}, "SHAPE"), ({"scale": math.nan}, "SHAPE"), ({"scale": math.inf}, "SHAPE"),
    ({"cap": -1.0}, "SHAPE"), ({"cap": math.inf}, "SHAPE"), ({"cap": math.nan}, "SHAPE"), ({"q_stride": 248}, "SHAPE"),
    ({"q_stride": 260}, "SHAPE"), ({"out_stride": 248}, "SHAPE"), ({"out_stride": 258}, "SHAPE"), ({"q_stride": LAST}, "SHAPE"),
    ({"out_stride": -256}, "SHAPE"), ({"slopes": P + 2}, "ALIGN"), ({"prefix": P + 1}, "ALIGN"), ({"first": P + 2}, "ALIGN")])
def test_attention_checks_its_options(syn, kw, err):
    want = getattr(syn, "ERR_" + err)
    assert decode(syn, d=attn(syn, **kw)) == want and prefill(syn, d=attn(syn, **kw)) == want


@pytest.mark.parametrize("kw,err", [
    ({"n_seq": -1}, "SHAPE"), ({"n_seq": 1 << 31}, "SHAPE"), ({"max_pages": 0}, "SHAPE"), ({"max_pages": 1 << 31}, "SHAPE"),
    ({"q": None}, "NULL"), ({"out": None}, "NULL"), ({"pages": None}, "NULL"), ({"lens": None}, "NULL"), ({"q": P + 8}, "ALIGN"),
    ({"out": P + 4}, "ALIGN"), ({"pages": P + 2}, "ALIGN"), ({"lens": P + 1}, "ALIGN")])
def test_attention_refusals(syn, kw, err):
    want = getattr(syn, "ERR_" + err)
    assert decode(syn, **kw) == want and prefill(syn, **kw) == want


@pytest.mark.parametrize("kw,err", [({"n_tok": -1}, "SHAPE"), ({"n_tok": 1 << 29}, "SHAPE"), ({"starts": None}, "NULL"),
                                    ({"starts": P + 2}, "ALIGN")])
def test_prefill_refusals(syn, kw, err):
    assert prefill(syn, **kw) == getattr(syn, "ERR_" + err)


def test_helpers_check_before_they_call(syn):
    """The torch helpers refuse tensors that the library would read otherwise than they lie."""
    import torch
    c = syn.KVCache.empty(F16, 2, 64, 16, 4, device="cpu")
    with pytest.raises(syn.SynError):
        syn.KVCache.empty(2, 2, 64, 16, 4, device="cpu")
    with pytest.raises(syn.SynError):
        syn.KVCache.empty(F16, 2, 40, 16, 4, device="cpu")
    for k, v in [(c.k, c.v[:3]), (c.k, c.v[:, :1]), (c.k.transpose(1, 2), c.v), (c.k[:0], c.v[:0]), (c.k, torch.stack([c.v] * 2, 1)[:, 0]),
                 (c.k[:1].expand(4, -1, -1, -1), c.v[:1].expand(4, -1, -1, -1))]:
        with pytest.raises(ValueError):
            syn.KVCache(F16, 2, 64, 16, k, v)
    with pytest.raises(ValueError):
        syn.Rope(64, factors=np.ones(31), device="cpu")
    with pytest.raises(ValueError):
        syn.Rope(64, axis=np.zeros(33), device="cpu")
    with pytest.raises(syn.SynError):
        syn.Rope(12, device="cpu")
    r = syn.Rope(64, device="cpu")
    k = torch.zeros((5, 2, 64))
    q = torch.zeros((5, 4, 64))
    pos, slots = torch.zeros(5, dtype=torch.int32), torch.zeros(5, dtype=torch.int64)
    ok = dict(k=k, v=k, pos=pos, slots=slots, q=q, stream=0)
    syn.prepare_kv_append(c, r, **ok)
    syn.prepare_kv_append(c, r, **{**ok, "k": torch.zeros((5, 6, 64))[:, 2:4]})
    for kw in ({"k": k.half()}, {"k": k[:, :1]}, {"v": k[:4]}, {"slots": slots[:4]}, {"slots": slots.int()}, {"pos": pos.long()},
               {"pos": pos[:4]}, {"q": q[:4]}, {"k": k[:1].expand(5, 2, 64)}, {"q": q.transpose(0, 1).contiguous().transpose(0, 1)},
               {"k": torch.zeros((5, 2, 128))[:, :, ::2]}, {"q_out": torch.zeros((5, 4, 64))},
               {"q_out": torch.zeros((5, 3, 64), dtype=torch.float16)}):
        with pytest.raises(ValueError):
            syn.prepare_kv_append(c, r, **{**ok, **kw})
    with pytest.raises(ValueError):
        syn.prepare_kv_append(c, syn.Rope(64, axis=[0, 1] * 16, device="cpu"), **ok)
    with pytest.raises(ValueError):
        syn.prepare_kv_read(c, slots.int(), stream=0)
    h = torch.zeros((5, 4, 64), dtype=torch.float16)
    pages, lens = torch.zeros((5, 2), dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    ok = dict(q=h, pages=pages, lens=lens, stream=0)
    syn.prepare_attn_decode(c, **ok)
    for kw in ({"q": q}, {"pages": pages[:4]}, {"pages": pages.view(-1)}, {"pages": pages.long()}, {"pages": torch.zeros((5, 4), dtype=torch.int32)[:, ::2]},
               {"lens": lens[:4]}, {"lens": lens.long()}, {"out": q[:4]}, {"out": q.double()}, {"slopes": torch.zeros(3)},
               {"slopes": torch.zeros(4).double()}, {"prefix": lens[:1]}, {"first": lens[:3]}, {"q": h[:1].expand(5, 4, 64)},
               {"out": torch.zeros((1, 4, 64)).expand(5, 4, 64)}):
        with pytest.raises(ValueError):
            syn.prepare_attn_decode(c, **{**ok, **kw})
    starts = torch.tensor([0, 2, 5], dtype=torch.int32)
    ok = dict(q=h, starts=starts, pages=pages[:2], lens=lens[:2], stream=0)
    syn.prepare_attn_prefill(c, **ok)
    for kw in ({"starts": starts[:2]}, {"starts": starts.long()}, {"first": lens[:2]}, {"prefix": lens}, {"pages": pages}):
        with pytest.raises(ValueError):
            syn.prepare_attn_prefill(c, **{**ok, **kw})
