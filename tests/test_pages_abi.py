"""What the calls on a cache's pages and syn_logprobs refuse, and what their torch helpers do.  CPU only:
every check here answers before a GPU is touched."""
import math

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


CALLS = {
    "syn_kv_fork": dict(refs=P, n_seq=2, pages=P, max_pages=3, lens=P, n_new=4, source=P, new_pages=P, new_lens=P),
    "syn_kv_extend": dict(refs=P, n_seq=2, n_tok=5, pages=P, max_pages=3, lens=P, starts=P, new_lens=P, slots=P),
    "syn_kv_compact": dict(refs=P, n_seq=2, n_rows=5, pages=P, max_pages=3, base=P, starts=P, rows=P, new_lens=P),
    "syn_kv_trim": dict(refs=P, n_seq=2, pages=P, max_pages=3, lens=P),
}


def call(syn, name, c=None, **kw):
    a = dict(CALLS[name])
    assert set(kw) <= set(a)
    a.update(kw)
    return getattr(syn, name)(c or cache(syn), *a.values(), None)


@pytest.mark.parametrize("kw,err", [({"type": 2}, "TYPE"), ({"head_dim": 48}, "SHAPE"), ({"page_size": 12}, "SHAPE"),
                                    ({"n_pages": 0}, "SHAPE"), ({"page_stride": LAST}, "SHAPE"), ({"k": None}, "NULL"),
                                    ({"v": P + 8}, "ALIGN")])
def test_every_call_checks_the_cache(syn, kw, err):
    bad, want = cache(syn, **kw), getattr(syn, "ERR_" + err)
    for name in CALLS:
        assert call(syn, name, bad) == want, name
    assert syn.syn_kv_copy(bad, cache(syn), 1, P, P, None) == want
    assert syn.syn_kv_copy(cache(syn), bad, 1, P, P, None) == want


@pytest.mark.parametrize("name", CALLS)
def test_null_and_alignment(syn, name):
    assert getattr(syn, name)(None, *CALLS[name].values(), None) == syn.ERR_NULL
    optional = {"syn_kv_extend": ("starts", "slots"), "syn_kv_compact": ("refs",)}.get(name, ())
    for k, v in CALLS[name].items():
        if v != P:
            continue
        if k not in optional:
            assert call(syn, name, **{k: None}) == syn.ERR_NULL, k
        assert call(syn, name, **{k: P + 2}) == syn.ERR_ALIGN, k
    if name == "syn_kv_extend":
        assert call(syn, name, slots=P + 4) == syn.ERR_ALIGN
        assert call(syn, name, starts=None, n_tok=3) == syn.ERR_SHAPE  # (one row each: as many as sequences)
        assert call(syn, name, n_seq=4097, n_tok=9000) == syn.ERR_SHAPE


@pytest.mark.parametrize("name", CALLS)
def test_sizes(syn, name):
    for k in ("n_seq", "max_pages", "n_new", "n_tok", "n_rows"):
        if k in CALLS[name]:
            for bad in (-1, LAST):
                assert call(syn, name, **{k: bad}) == syn.ERR_SHAPE, (k, bad)
    assert call(syn, name, max_pages=0) == syn.ERR_SHAPE


def test_calls_of_nothing(syn):
    for name, a in CALLS.items():
        none = {k: None if v == P else 0 for k, v in a.items()}
        assert call(syn, name, **none) == syn.OK, name
    assert syn.syn_kv_copy(cache(syn), cache(syn), 0, None, None, None) == syn.OK


def test_copy_refusals(syn):
    c = cache(syn)
    for kw, err in (({"type": Q8_0}, "TYPE"), ({"head_dim": 32}, "SHAPE"), ({"n_kv_heads": 1}, "SHAPE"), ({"page_size": 32}, "SHAPE")):
        assert syn.syn_kv_copy(c, cache(syn, **kw), 1, P, P, None) == getattr(syn, "ERR_" + err)
    for args, err in (((-1, P, P), "SHAPE"), ((LAST, P, P), "SHAPE"), ((1, None, P), "NULL"), ((1, P, None), "NULL"),
                      ((1, P + 1, P), "ALIGN"), ((1, P, P + 2), "ALIGN")):
        assert syn.syn_kv_copy(c, c, *args, None) == getattr(syn, "ERR_" + err)


def logprobs(syn, opt=None, **kw):
    d = dict(type=0, scale=1.0, cap=0.0, scales=None, mask=None, stride=0, mask_stride=0)
    d.update(opt or {})
    a = dict(n_rows=2, n_vocab=100, logits=P, n_ids=1, ids=P, logprob=P, entropy=P, n_top=3, top=P, top_logprob=P)
    a.update(kw)
    return syn.syn_logprobs(syn.LogitsDesc(*d.values()), *a.values(), None)


@pytest.mark.parametrize("opt,kw,err", [
    ({"type": 2}, {}, "TYPE"), ({"type": -1}, {}, "TYPE"), ({"scale": 0.0}, {}, "SHAPE"), ({"scale": -1.0}, {}, "SHAPE"),
    ({"scale": math.nan}, {}, "SHAPE"), ({"scale": math.inf}, {}, "SHAPE"), ({"cap": -1.0}, {}, "SHAPE"),
    ({"cap": math.inf}, {}, "SHAPE"), ({"stride": 99}, {}, "SHAPE"), ({"stride": -100}, {}, "SHAPE"), ({"stride": LAST}, {}, "SHAPE"),
    ({"mask_stride": 3}, {}, "SHAPE"), ({"mask_stride": LAST}, {}, "SHAPE"), ({"scales": P + 2}, {}, "ALIGN"),
    ({"mask": P + 1}, {}, "ALIGN"), ({"type": 1}, {"logits": P + 1}, "ALIGN"), ({}, {"logits": P + 2}, "ALIGN"),
    ({}, {"n_rows": -1}, "SHAPE"), ({}, {"n_rows": LAST}, "SHAPE"), ({}, {"n_vocab": 0}, "SHAPE"), ({}, {"n_vocab": LAST}, "SHAPE"),
    ({}, {"n_ids": -1}, "SHAPE"), ({}, {"n_ids": 1 << 17}, "SHAPE"), ({}, {"n_top": -1}, "SHAPE"), ({}, {"n_top": 65}, "SHAPE"),
    ({}, {"logits": None}, "NULL"), ({}, {"ids": None}, "NULL"), ({}, {"logprob": None}, "NULL"), ({}, {"top": None}, "NULL"),
    ({}, {"top_logprob": None}, "NULL"), ({}, {"ids": P + 2}, "ALIGN"), ({}, {"logprob": P + 2}, "ALIGN"),
    ({}, {"entropy": P + 2}, "ALIGN"), ({}, {"top": P + 2}, "ALIGN"), ({}, {"top_logprob": P + 2}, "ALIGN")])
def test_logprobs_refusals(syn, opt, kw, err):
    assert logprobs(syn, opt, **kw) == getattr(syn, "ERR_" + err)


def test_logprobs_of_nothing(syn):
    import torch
    assert syn.syn_logprobs(None, 0, 1, None, 0, None, None, None, 0, None, None, None) == syn.ERR_NULL
    assert logprobs(syn, n_rows=0, logits=None, ids=None, logprob=None, entropy=None, top=None, top_logprob=None) == syn.OK
    got = syn.logprobs(torch.zeros((0, 50)), torch.zeros((0, 2), dtype=torch.int32), 3, stream=0)
    assert got.logprob.shape == (0, 2) and got.entropy.shape == (0,) and got.top.shape == (0, 3)
    assert syn.logprobs(torch.zeros((0, 50)), stream=0).logprob is None


def test_helpers_refuse(syn):
    """Shapes, types and devices that the library would read otherwise."""
    import torch
    c = syn.KVCache.empty(F16, 2, 64, 16, 4, device="cpu")
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    refs, pages, lens, kw = i(4), i(2, 3), i(2), {"stream": 0}
    for a in ((i(5), i(2), pages, lens), (refs, i(2).long(), pages, lens), (refs, i(2), i(3, 3), lens), (refs, i(2), i(2, 6)[:, ::2], lens),
              (refs, i(2), pages, lens, i(2, 4)), (refs, i(2), pages, lens, i(2, 3), i(3)), (refs, i(2), pages.to("meta"), lens)):
        with pytest.raises(ValueError):
            syn.kv_fork(c, *a, **kw)
    slots = torch.zeros(2, dtype=torch.int64)
    for a, more in (((i(3), pages, lens), {}), ((refs, i(6), lens), {}), ((refs, pages, lens.long()), {}), ((refs, pages, lens, i(3)), {}),
                    ((refs, pages, lens), {"slots": slots[:1]}), ((refs, pages, lens), {"slots": i(2)}), ((refs, pages, lens), {"starts": i(3)}),
                    ((refs, pages, lens), {"starts": i(2), "n_tok": 2}), ((refs, pages, lens), {"starts": i(3), "n_tok": 3, "slots": slots})):
        with pytest.raises(ValueError):
            syn.kv_extend(c, *a, **more, **kw)
    for a in ((i(2), pages, lens, i(3), i(1)), (refs, pages, lens, i(2), i(1)), (refs, pages, lens, i(3), i(1).long()),
              (refs, pages, lens, i(3), i(1, 1)), (refs, pages, lens, i(3), i(1), i(1))):
        with pytest.raises(ValueError):
            syn.kv_compact(c, *a, **kw)
    for a in ((i(3), pages, lens), (refs, pages, i(3)), (refs, pages.float(), lens)):
        with pytest.raises(ValueError):
            syn.kv_trim(c, *a, **kw)
    with pytest.raises(ValueError):
        syn.kv_copy(c, c, i(2), i(3), **kw)
    x = torch.zeros((2, 50))
    for a, more in (((x.double(),), {}), ((x[0],), {}), ((x.t(),), {}), ((x[:1].expand(2, 50),), {}), ((x, i(3, 1)), {}), ((x, i(2, 1).long()), {}),
                    ((x, i(2, 1, 1)), {}), ((x, i(4, 2)[::2]), {}), ((x,), {"scales": torch.zeros(3)}), ((x,), {"scales": torch.zeros(2).half()}),
                    ((x,), {"mask": i(2, 1)}), ((x,), {"mask": i(1, 2)}), ((x,), {"mask": i(2, 2).bool()}), ((x,), {"mask": i(2, 2, 2)}),
                    ((x, i(2, 1).to("meta")), {})):
        with pytest.raises(ValueError):
            syn.logprobs(*a, **more, **kw)
    for more in ({"n_top": 65}, {"n_top": -1}, {"scale": 0.0}, {"cap": -1.0}):
        with pytest.raises(syn.SynError):
            syn.logprobs(x, **more, **kw)


def tree(syn, c=None, **kw):
    d = dict(n_heads=4, window=0, scale=0.125, cap=0.0, slopes=None, prefix=None, first=None, q_stride=0, out_stride=0, out_type=0)
    a = dict(n_seq=2, n_tok=9, q=P, starts=P, parents=P, pages=P, max_pages=2, lens=P, out=P)
    for k, v in kw.items():
        assert k in d or k in a
        (d if k in d else a)[k] = v
    return syn.syn_attn_tree(c or cache(syn), syn.AttnDesc(*d.values()), *a.values(), None)


@pytest.mark.parametrize("kw,err", [
    ({"n_heads": 3}, "SHAPE"), ({"n_heads": 0}, "SHAPE"), ({"window": -1}, "SHAPE"), ({"scale": math.nan}, "SHAPE"), ({"cap": -1.0}, "SHAPE"),
    ({"q_stride": 100}, "SHAPE"), ({"out_stride": LAST}, "SHAPE"), ({"out_type": 2}, "TYPE"), ({"n_seq": -1}, "SHAPE"),
    ({"n_tok": -1}, "SHAPE"), ({"n_tok": 1 << 30}, "SHAPE"), ({"max_pages": 0}, "SHAPE"), ({"max_pages": LAST}, "SHAPE"), ({"q": None}, "NULL"),
    ({"starts": None}, "NULL"), ({"parents": None}, "NULL"), ({"pages": None}, "NULL"), ({"lens": None}, "NULL"), ({"out": None}, "NULL"),
    ({"q": P + 8}, "ALIGN"), ({"starts": P + 2}, "ALIGN"), ({"parents": P + 2}, "ALIGN"), ({"pages": P + 1}, "ALIGN"), ({"lens": P + 2}, "ALIGN"),
    ({"out": P + 4}, "ALIGN"), ({"first": P + 2}, "ALIGN"), ({"prefix": P + 2}, "ALIGN"), ({"slopes": P + 2}, "ALIGN")])
def test_tree_refusals(syn, kw, err):
    assert tree(syn, **kw) == getattr(syn, "ERR_" + err)


def test_tree_checks_its_structures(syn):
    import torch
    assert tree(syn, cache(syn, type=3)) == syn.ERR_TYPE and tree(syn, cache(syn, k=None)) == syn.ERR_NULL
    assert syn.syn_attn_tree(cache(syn), None, 1, 1, P, P, P, P, 1, P, P, None) == syn.ERR_NULL
    assert tree(syn, n_tok=0) == syn.OK and tree(syn, n_seq=0, n_tok=0) == syn.OK
    c = syn.KVCache.empty(F16, 2, 64, 16, 4, device="cpu")
    q, i = torch.zeros((3, 4, 64), dtype=torch.float16), lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    for a in ((q, i(2), i(3), i(2, 3), i(2)), (q, i(3), i(4), i(2, 3), i(2)), (q, i(3), i(3).long(), i(2, 3), i(2)), (q, i(3), i(3), i(1, 3), i(2)),
              (q.float(), i(3), i(3), i(2, 3), i(2)), (q, i(3), i(3).to("meta"), i(2, 3), i(2))):
        with pytest.raises(ValueError):
            syn.attn_tree(c, *a, stream=0)
