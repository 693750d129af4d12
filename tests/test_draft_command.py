"""What the attention block's command refuses (CPU: before anything is built)."""
import sys

import pytest


@pytest.mark.parametrize("args", [["--prompt", "0"], ["--steps", "0"], ["--seqs", "0"], ["--draft", "-1"], ["--draft", "4", "--steps", "0"]])
def test_sizes_that_are_none(args, monkeypatch, capsys):
    from gguf_block_quantized_gb300 import attn_block
    monkeypatch.setattr(sys, "argv", ["attn_block", *args])
    with pytest.raises(SystemExit) as e:
        attn_block.main()
    assert e.value.code == 2 and "at least 1" in capsys.readouterr().err
