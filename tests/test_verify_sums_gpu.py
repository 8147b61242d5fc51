"""Sums of the longest rows that m4q_verify_tree takes, where many sequences leave one
CTA, and so tens of thousands of values a thread, to each row (GPU).  The rows are one
row expanded over the sequences, of equal values c: every sum is k c, which a pair of
fp32 values holds exactly, so u = k / V is exactly the border behind the k-th value and
the next token has to be k."""
import numpy as np
import pytest

import swiglu_block_quantized_gb300 as m

torch = pytest.importorskip("torch")
from test_attention_tree_gpu import ints   # noqa: E402

pytestmark = pytest.mark.gpu

# values of all 24 bits, with a short fraction, and of fp16's 11 bits
WIDE = [0.1, 1 / 3, 0.7310585975646973, 5.9604644e-08 * 1.2345678, 0.9999999403953552]
SHORT = [c // 2.0 ** -30 * 2.0 ** -30 for c in (0.0001, 0.0003333, 0.00073)]   # at most 21 bits
HALF = [0.0999755859375, 0.333251953125, 5.9604644775390625e-08, 2.0 ** -14 * 1.3779296875]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()
    m.load()
    yield
    assert m.check_device_status() == m.OK


def borders(b, v, seed):
    """Counts k in [0, v), the ends among them, and u = k / v (v a power of two)."""
    k = np.random.RandomState(seed).randint(0, v, b)
    k[:4] = [0, 1, v - 1, v // 2]
    return k, torch.tensor(k / v, dtype=torch.float32, device="cuda")


@pytest.mark.parametrize("v,b", [(2 ** 24, 200), (2 ** 24, 110), (2 ** 23, 160), (2 ** 23, 400), (2 ** 21, 200)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_samples_at_borders(dtype, v, b):
    for i, c in enumerate(WIDE if dtype is torch.float32 else HALF):
        k, u = borders(b, v, i)
        row = torch.full((v,), c, device="cuda").to(dtype)
        root = ints([[-1]] * b)
        _, count, token = m.verify_tree(row.expand(b, 1, v), None, root, root, u.view(b, 1))
        assert (count == 1).all()
        assert np.array_equal(token.cpu().numpy(), k), c


@pytest.mark.parametrize("v,b", [(2 ** 24, 200), (2 ** 24, 110), (2 ** 23 + 1, 160)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("children", [1, 2])
def test_rests_at_borders(dtype, v, b, children):
    # The last token has no share of the target, so as a child it is turned down whatever u is.  The
    # rest of the first 2^23 tokens, which have all of it, is p - q after one child and p - (1 + m) q
    # after two, m the sum of the rest before (p = 1 / 2^23, so that m is 3/4, or 1 where q is below
    # fp16's range, exactly).  c - c / 4 of all 24 bits has 26: with the 23 of k that is one more than
    # a pair of fp32 values holds, so there the border is off by up to 2^-48 of itself and its
    # neighbour may be taken; c of 21 bits has no such excuse.
    n = 2 ** 23
    for i, c in enumerate((WIDE + SHORT if dtype is torch.float32 else HALF) if children == 1 else [1.0 / n]):
        k, u = borders(b, n, i)
        p = torch.zeros(v, device="cuda", dtype=dtype)
        p[:n] = c
        q = p / 4
        q[v - 1] = 0.25
        root = ints([[-1] + [0] * children] * b)
        tokens = ints([[0] + [v - 1] * children] * b)
        us = torch.cat([u.view(b, 1), torch.full((b, children), 0.5, device="cuda")], 1)
        rows = (b, children + 1, v)
        _, count, token = m.verify_tree(p.expand(rows), q.expand(rows), tokens, root, us)
        assert (count == 1).all()
        off = np.abs(token.cpu().numpy().astype(np.int64) - k)
        assert off.max() <= (1 if children == 1 and c in WIDE and dtype is torch.float32 else 0), c
