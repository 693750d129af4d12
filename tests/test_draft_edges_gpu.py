"""The operators of drafted tokens where several of their parts meet: many candidates over several turns, long lists one
after the other, few SMs, values at the ends of their types."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

F16, Q8_0 = 7, 1


@pytest.fixture(scope="module")
def syn():
    import torch
    assert torch.cuda.is_available()
    from gguf_block_quantized_gb300 import syn
    yield syn
    torch.cuda.synchronize()
    assert syn.device_status() == syn.OK


def most_likely(x, n_top):
    """The tokens of the n_top largest, ties to the lower one."""
    import torch
    bits = (x.float() + 0.0).view(torch.int32)
    key = ((bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32) - torch.arange(x.shape[1], device="cuda")
    return torch.topk(key, n_top, 1).indices.to(torch.int32)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("rows,n_top", [(600, 40), (600, 50), (600, 64), (310, 57)])
def test_candidates_over_several_turns(syn, rows, n_top, half):
    """A CTA to a row of 128256 logits: 16 or 32 units a turn are read again, and more than 64 logits found, so that the list
    is cut between two turns."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(rows + n_top)
    for _ in range(4):
        x = torch.randn((rows, 128256), device="cuda", generator=gen)
        if half:
            x = x.half()  # (ties among the largest)
        want = most_likely(x, n_top)
        for _ in range(3):
            got = syn.logprobs(x, n_top=n_top)
            assert torch.equal(got.top, want)
            z = x.gather(1, want.long()).double() - torch.logsumexp(x.double(), 1, keepdim=True)
            # 2^-17 for ln S, 2^-22 of the log probability
            assert ((got.top_logprob - z).abs() <= 2.0 ** -17 + 2.0 ** -22 * z.abs()).all()
