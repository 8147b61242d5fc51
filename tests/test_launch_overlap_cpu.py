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


# The kernels of before that read what the serving kernels write: activations (the
# norms), queries (the rotation) and cache rows.  Packed weights are nobody's output.
@pytest.mark.parametrize("name", ["gemv.cuh", "attention.cu", "attention_tc.cu", "tc_proj.cuh", "tc_small.cuh"])
def test_activations_queries_and_cache_rows_are_not_read_only(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    for call in re.finditer(r"__ldg\(", code):
        arg = code[call.start():call.start() + 90].split(";")[0]
        assert "p.row_bytes" in arg or "(row + o" in arg, arg   # packed weight rows
    for kernel in re.finditer(r"__global__[^{;]*\{", code):
        assert "__restrict__" not in kernel.group(0), kernel.group(0)
