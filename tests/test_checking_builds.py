"""Every source with kernels has index checks, and its status word is read (CPU: the sources alone)."""
import os
import re

from gguf_block_quantized_gb300 import build


def test_every_kernel_file_is_checked():
    def text(name):
        with open(os.path.join(build.CSRC, name)) as f:
            return f.read()

    read = re.findall(r"syn::(debug_bounds_\w+)\(clear\)", text("api.cu"))
    kernels = 0
    for name in build.SOURCES:
        source = text(name)
        if "__global__" not in source:
            continue
        kernels += 1
        reader = re.findall(r"SYN_BOUNDS_READER\((\w+)\)", source)
        assert len(reader) == 1 and reader[0] in read, name
        assert "SYN_IN_BOUNDS(" in source, name
    assert kernels == len(read) == len(set(read))
