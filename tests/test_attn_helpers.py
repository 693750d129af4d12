"""What the torch helpers of the paged cache take and refuse.  CPU only: they check before they call."""
import pytest

F16, Q8_0 = 7, 1


@pytest.fixture(scope="module")
def syn():
    import torch  # noqa: F401
    from gguf_block_quantized_gb300 import build
    build.build()
    from gguf_block_quantized_gb300 import syn
    return syn


def test_pools_hold_what_the_cache_says(syn):
    """Types and shapes of the pools, not their bytes alone."""
    import torch
    half, byte = torch.zeros((3, 2, 16, 64), dtype=torch.float16), torch.zeros((3, 2, 16 * 64 // 16 * 17), dtype=torch.uint8)
    c = syn.KVCache(F16, 2, 64, 16, half, half.clone())
    assert c.n_pages == 3 and c.desc.page_stride == 2 * 16 * 64 * 2
    assert syn.KVCache(Q8_0, 2, 64, 16, byte, byte.clone()).desc.page_stride == byte.stride(0)
    both = torch.zeros((3, 2, 2, 16, 64), dtype=torch.float16)
    assert syn.KVCache(F16, 2, 64, 16, both[:, 0], both[:, 1]).desc.page_stride == 2 * 2 * 16 * 64 * 2
    syn.KVCache(F16, 2, 64, 16, half[:1], half[1:2])
    for t, k in [(F16, half.to(torch.bfloat16)), (F16, half.to(torch.int16)), (F16, half.view(torch.uint8)), (F16, half.flatten(1)),
                 (F16, torch.zeros((3, 2, 16, 32))), (F16, torch.zeros((3, 16, 2, 64), dtype=torch.float16)),
                 (F16, torch.zeros((3, 2, 64, 16), dtype=torch.float16)), (Q8_0, byte.view(torch.int8)),
                 (Q8_0, byte.view(torch.float16)), (Q8_0, byte.flatten(1)), (Q8_0, half), (F16, byte)]:
        with pytest.raises(ValueError):
            syn.KVCache(t, 2, 64, 16, k, k.clone())
    for v in (half.to(torch.bfloat16), half.to("meta"), byte):
        with pytest.raises(ValueError):
            syn.KVCache(F16, 2, 64, 16, half, v)


def test_calls_of_no_tokens(syn):
    """Empty tensors, whose pointers are 0: such calls do nothing, as kv_append and kv_read of nothing."""
    import torch
    c = syn.KVCache.empty(F16, 2, 64, 16, 4, device="cpu")
    q, i32 = torch.zeros((0, 4, 64), dtype=torch.float16), lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    assert q.data_ptr() == 0
    none = {"stream": 0}
    for width in (3, 0):
        assert syn.attn_decode(c, q, i32(0, width), i32(0), **none).shape == q.shape
        assert syn.attn_prefill(c, q, i32(1), i32(0, width), i32(0), **none).shape == q.shape
        assert syn.attn_prefill(c, q, i32(3), i32(2, width), i32(2), **none).shape == q.shape
    half = torch.zeros((0, 4, 64), dtype=torch.float16)
    opt = {"slopes": torch.zeros(4), "prefix": i32(0), "first": i32(0), "window": 7, "cap": 3.0}
    assert syn.attn_decode(c, q, i32(0, 3), i32(0), half, **opt, **none) is half
    k = torch.zeros((0, 2, 64))
    assert syn.kv_append(c, syn.Rope(0, device="cpu"), k, k, None, torch.zeros(0, dtype=torch.int64), **none) is None
    assert syn.kv_read(c, torch.zeros(0, dtype=torch.int64), **none)[0].shape == (0, 2, 64)
    for bad in ({"window": -1}, {"cap": -1.0}):  # (the options are checked all the same)
        with pytest.raises(syn.SynError):
            syn.attn_decode(c, q, i32(0, 3), i32(0), **bad, **none)
