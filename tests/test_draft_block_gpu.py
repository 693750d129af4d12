"""A speculative run of the attention block: pages forked and extended, trees of drafts verified, accepted paths packed, the
rest given back, against decoding one token at a time."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,prompt,tokens,seqs,nodes,page", [(7, 100, 12, 3, 9, 16), (1, 65, 10, 4, 26, 64), (7, 1, 9, 2, 1, 8)])
def test_drafts_give_what_single_tokens_give(t, prompt, tokens, seqs, nodes, page):
    """The same tokens, and log probabilities within the two forms' roundings: hidden values are sums of about 2048
    products of which the tree form rounds p and the values to fp16 (2^-11 each, Q8_0 keys and values too), so a logit of
    size z moves by a few 2^-11 z; logits here are within 16."""
    from gguf_block_quantized_gb300 import attn_block, syn
    r = attn_block.run_drafts(t, prompt, tokens, seqs, nodes, vocab=4000, page=page)
    assert syn.device_status() == syn.OK
    assert r["same"] and r["held"] == 0
    assert r["difference"] <= 16 * 8 * 2.0 ** -11
    assert r["per_step"] >= 1.0 and (nodes > 1 or r["per_step"] == 1.0)


def test_command(capsys, monkeypatch):
    import sys
    from gguf_block_quantized_gb300 import attn_block
    monkeypatch.setattr(sys, "argv", ["attn_block", "--prompt", "40", "--steps", "4", "--seqs", "2", "--draft", "7"])
    attn_block.main()
    assert "the same tokens: True" in capsys.readouterr().out
