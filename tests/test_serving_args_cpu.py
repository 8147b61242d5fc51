"""More arguments of the serving operators that the binding or the C ABI accepts or
refuses before touching the GPU (no GPU needed)."""
import ctypes

import pytest

import swiglu_block_quantized_gb300 as m

torch = pytest.importorskip("torch")
from test_serving_cpu import FR, cpu_binding, f16, i32   # noqa: E402,F401


def rows(strides, h=2, n=4, d=64):
    size = 1 + (h - 1) * strides[0] + (n - 1) * strides[1] + d - 1
    return f16(size).as_strided((h, n, d), (*strides, 1))


def test_rope_takes_rows_with_gaps(cpu_binding):
    # rows that do not overlap, however they lie: the next head's first row may start
    # in the gap behind this one's last
    for strides in ((280, 72), (64, 136), (256, 64), (72, 200), (400, 96), (64, 128)):
        with pytest.raises(AssertionError, match="m4q_rope was called"):
            m.rope(f16(2, 4, 64), i32(4), FR, out=rows(strides))
    for strides in ((272, 72), (64, 120), (248, 64), (0, 64), (64, 0), (56, 512)):
        with pytest.raises(ValueError, match="overlap"):
            m.rope(f16(2, 4, 64), i32(4), FR, out=rows(strides))


def test_norm_gate_of_another_shape(cpu_binding):
    # as many rows as columns: one value a row holds as many values as one a column,
    # and would be taken for it
    h, r, w = f16(64, 64), f16(64, 64), f16(64)
    for gate in (f16(64, 1), f16(1, 64, 1), f16(32, 128), f16(64, 32, 2)):
        with pytest.raises(ValueError, match="gate"):
            m.norm_residual(h, r, w, gate=gate)
    for gate in (f16(64), f16(1, 64), f16(64, 64), f16(8, 8, 64), f16(64 * 64)):
        with pytest.raises(AssertionError, match="m4q_norm_residual was called"):
            m.norm_residual(h, r, w, gate=gate)


def test_parents_of_another_shape(cpu_binding):
    # node by node instead of tree by tree: as many values, other trees
    kc = f16(2, 2, 8, 64)
    call = lambda p: m.attention_tree(f16(4, 6, 64), kc, kc, m.KV_F16, i32(2), p)   # noqa: E731
    for shape in ((3, 2), (6, 1), (1, 6), (2, 3, 1)):
        with pytest.raises(ValueError, match="parents"):
            call(i32(6).view(shape))
    for shape in ((2, 3), (6,)):
        with pytest.raises(AssertionError, match="m4q_attention_tree was called"):
            call(i32(6).view(shape))


def test_tree_scale_in_powers_of_two():
    # a finite scale whose product with log2(e) is not: every score would be NaN
    m.build()
    a = ctypes.c_void_p(0x100000)   # never dereferenced
    for scale in (3e38, -3e38, 2.4e38):
        assert m.load().m4q_attention_tree(a, a, a, m.KV_F16, 1, 4, 2, 3, 8, 64, a, a, scale, a, None, 0,
                                           None) == m.ERR_INVALID_ARG
