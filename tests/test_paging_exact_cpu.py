"""What the tolerances of test_paging_exact_gpu tell apart (no GPU needed): mistakes
planted in the 64-bit result of long sequences, a piece lost or joined twice, one key
lost, a result of another size, are outside them."""
import pytest

torch = pytest.importorskip("torch")
import _paging_exact as exact   # noqa: E402

N, D = 20001, 64


def mean_of_stripes():
    v = exact.striped((N + 63) // 64, 64, D, 64, torch.float64).view(-1, D)[:N]
    w = torch.full((1, N), 1.0 / N, dtype=torch.float64)
    want = w @ v
    return w, v, want, exact.tolerance(w, v[None], want, torch.zeros(1), rounded=False)


def outside(o, want, tol):
    return bool(((o - want).abs() > tol).any())


@pytest.mark.parametrize("first,last", [(0, 1), (777, 778), (N - 1, N), (0, 8), (64, 128), (5000, 7000)])
@pytest.mark.parametrize("times", [0, 2])
def test_keys_lost_or_taken_twice(first, last, times):
    w, v, want, tol = mean_of_stripes()
    f = torch.ones(N, dtype=torch.float64)
    f[first:last] = times
    assert not outside(want, want, tol)
    assert outside((w * f) @ v / (w * f).sum(), want, tol)       # numbers and their sum
    assert outside((w * f) @ v, want, tol)                       # numbers alone


def test_another_size():
    w, v, want, tol = mean_of_stripes()
    assert outside(want * 0.999, want, tol) and outside(want * 0, want, tol)


def test_random_rows():
    # elementwise bounds of random rows are wide, as every weight's rounding may have one sign; their
    # root mean square is not
    g = torch.Generator().manual_seed(1)
    v = torch.randn(N, D, generator=g, dtype=torch.float64)
    w = torch.softmax(torch.randn(1, N, generator=g, dtype=torch.float64), -1)
    want = w @ v
    tol = exact.tolerance(w, v[None], want, torch.full((1,), 20.0))
    assert float(tol.max()) < 0.2 * float(want.square().mean().sqrt())
    rounded = (w * N).half().double() / N @ v
    assert float((rounded - want).square().mean().sqrt()) < 2.0 ** -11 * float(want.square().mean().sqrt())


@pytest.mark.parametrize("bits", [20, 24, 26])
def test_tail_without_weight(bits):
    # one key has all but the tail's weight, and values of 0
    w = torch.full((1, N), 2.0 ** -bits, dtype=torch.float64)
    w[0, 0] = 1
    w /= w.sum()
    v = torch.rand(N, D, dtype=torch.float64, generator=torch.Generator().manual_seed(2)) + 0.5
    v[0] = 0
    want = w @ v
    tol = exact.tolerance(w, v[None], want, torch.full((1,), 20.0))
    assert outside(want * 0, want, tol) and outside(want * 0.75, want, tol)
