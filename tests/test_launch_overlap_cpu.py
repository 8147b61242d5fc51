"""The serving kernels start before the kernel ahead of them in the stream has ended,
so what that one may write is never read through the read-only path, which is for
memory that nobody writes while a kernel is resident (no GPU needed)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "swiglu_block_quantized_gb300", "csrc")


@pytest.mark.parametrize("name", ["kv_ops.cu", "kv_common.cuh", "norm.cu", "attention_tree.cu", "attention_few.cu",
                                  "tree_common.cuh"])
def test_only_the_frequency_table_is_read_only(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "ld.global.nc" not in code and "__restrict__" not in code
    for call in re.finditer(r"__ldg\(", code):
        assert "p.freqs" in code[call.start():call.start() + 60].split(";")[0], code[call.start():call.start() + 80]
