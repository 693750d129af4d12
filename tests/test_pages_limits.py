"""Sizes at the ends of what the calls on a cache's pages count with.  CPU only: refused before a GPU is touched."""
import pytest

F16 = 7
P = 1 << 20  # any aligned non-null value


@pytest.fixture(scope="module")
def syn():
    import torch  # noqa: F401
    from gguf_block_quantized_gb300 import build
    build.build()
    from gguf_block_quantized_gb300 import syn
    return syn


def test_chunks_of_a_long_list_are_counted_in_32_bits(syn):
    """Every CTA takes a chunk past the last, so the counter needs room above the number of chunks.  Heads of 256 values: a
    chunk has 32 rows of two tiles, so 32 heads make 32 groups and the longest list 2^31 - 1024 chunks."""
    rows = 2 ** 31 - 1025
    for kv, n in ((32, rows), (256, rows), (512, rows // 2)):
        cache = syn.KVCacheDesc(F16, kv, 256, 16, 4, P, P, 0)
        assert syn.syn_kv_compact(cache, P, 1, n, P, 3, P, P, P, P, None) == syn.ERR_SHAPE, kv
