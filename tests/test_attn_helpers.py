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
