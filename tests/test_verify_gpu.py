"""Drafted trees verified against the target's probabilities, against a 64-bit reference
(GPU).  There is one right answer wherever no decision lies within 2^-40 of its border
(the operator's differences and sums are good to 2^-44, the reference's to 2^-45 for the
rows here); ties between exactly representable sums go one way only."""
import math

import numpy as np
import pytest

import swiglu_block_quantized_gb300 as m

torch = pytest.importorskip("torch")
import _paging_ref as pref   # noqa: E402
from test_attention_tree_gpu import gen, ints   # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()
    m.load()
    yield
    assert m.check_device_status() == m.OK


def distributions(g, b, n, v, dtype, spread=2.0, error=0.8):
    x = torch.randn(b, n, v, generator=g, device="cuda") * spread
    y = x + error * torch.randn(b, n, v, generator=g, device="cuda")
    return torch.softmax(x, -1).to(dtype), torch.softmax(y, -1).to(dtype)


def drawn(g, draft, parents):
    """A token for every node, from its parent's draft distribution."""
    b, n, v = draft.shape
    rows = torch.gather(draft.double(), 1, parents.long().clamp(0, n - 1)[:, :, None].expand(b, n, v)).cumsum(-1)
    at = torch.rand(b, n, 1, generator=g, device="cuda", dtype=torch.float64) * rows[:, :, -1:]
    return torch.searchsorted(rows, at, right=True).clamp(max=v - 1)[:, :, 0].to(torch.int32)


def trees(r, b, n, kind):
    if kind == "chain":
        return [[i - 1 for i in range(n)] for _ in range(b)]
    if kind == "star":
        return [[-1] + [0] * (n - 1) for _ in range(b)]
    p = [[-1] + [int(r.randint(max(0, i - 4), i)) for i in range(1, n)] for _ in range(b)]
    if kind == "holes":
        for s in range(b):
            for i in range(1, n):
                if r.rand() < 0.3:
                    p[s][i] = [-1, -2, i, i + 2, 2 ** 31 - 1, -2 ** 31][r.randint(6)]
            if s % 5 == 4:
                p[s][0] = [-2, 0, 3, -2 ** 31][s % 4]
    return p


def compare(target, draft, tokens, parents, u, least=2.0 ** -40):
    got = m.verify_tree(target, draft, tokens, parents, u)
    want = pref.verify(target, draft, tokens, parents, u)
    assert want[3] > least, "an input on a border"
    for name, x, y in zip(("path", "count", "token"), got, want):
        assert x.dtype == torch.int32 and x.tolist() == y, name
    return want


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("kind", ["chain", "star", "random", "holes"])
@pytest.mark.parametrize("n", [1, 2, 5, 17])
@pytest.mark.parametrize("v", [1, 2, 31, 33, 1000, 5003])
def test_trees(dtype, kind, n, v):
    b = 9
    g, r = gen(n * 100 + v), np.random.RandomState(n + v)
    p, q = distributions(g, b, n, v, dtype)
    parents = ints(trees(r, b, n, kind))
    compare(p, q, drawn(g, q, parents), parents, torch.rand(b, n, generator=g, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("v", [32000, 65536, 128000, 150001, 262144 + 5])
def test_long_rows(dtype, v):
    b, n = 5, 6
    g, r = gen(v), np.random.RandomState(v)
    for kind, error in (("chain", 0.3), ("star", 2.0), ("random", 1.0)):
        p, q = distributions(g, b, n, v, dtype, error=error)
        parents = ints(trees(r, b, n, kind))
        compare(p, q, drawn(g, q, parents), parents, torch.rand(b, n, generator=g, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_longest_rows(dtype):
    v = 2 ** 24
    g = gen(3)
    for n in (1, 3):
        p, q = distributions(g, 1, n, v, torch.float32, spread=1.0)
        if dtype is torch.float16:   # (probabilities of fp16's range, not summing to 1)
            p, q = (p * 4096).half(), (q * 4096).half()
        parents = ints([[-1] + [0] * (n - 1)])
        compare(p, q, torch.randint(0, v, (1, n), generator=g, device="cuda").to(torch.int32), parents,
                torch.rand(1, n, generator=g, device="cuda"))


@pytest.mark.parametrize("b,n", [(1, 256), (300, 3), (2000, 1)])
def test_many(b, n):
    g, r = gen(b), np.random.RandomState(b)
    p, q = distributions(g, b, n, 203, torch.float32)
    parents = ints(trees(r, b, n, "random"))
    compare(p, q, drawn(g, q, parents), parents, torch.rand(b, n, generator=g, device="cuda"))


def test_every_token_is_drawn():
    # the next token over a grid of u: each one's share, at the borders' right sides
    v = 37
    g = gen(2)
    w = torch.randint(0, 3, (v,), generator=g, device="cuda").float()
    w[3] = w[20] = 0
    w[30] += 64 - w.sum()   # the sum is 64: every share and border is exact in fp32
    p = (w / 64).view(1, 1, v).expand(64, 1, v)
    u = torch.arange(64, device="cuda").float().view(64, 1) / 64
    root = ints([[-1]] * 64)
    _, count, token = m.verify_tree(p, None, root, root, u)
    want = torch.repeat_interleave(torch.arange(v, device="cuda"), w.long())
    assert torch.equal(token.long(), want) and (count == 1).all()


@pytest.mark.parametrize("v", [8, 700, 70000])
def test_ties(v):
    # exactly representable sums: u exactly at a border belongs to what comes after it
    p = torch.zeros(1, 2, v, device="cuda")
    q = torch.zeros_like(p)
    a, b = v // 3, v - 2
    p[0, 0, a], p[0, 0, b] = 0.25, 0.75
    q[0, 0, a], q[0, 0, b] = 0.5, 0.5
    p[0, 1, 1], p[0, 1, v - 1] = 0.5, 0.5
    for tok, u1, u0, path, token in ((a, 0.5, 0.0, [0, -1], b), (a, 0.49999997, 0.0, [0, 1], 1),
                                     (a, 0.25, 0.5, [0, 1], v - 1), (a, 0.25, 0.49999997, [0, 1], 1),
                                     (b, 0.99999994, 0.99999994, [0, 1], v - 1), (a, 0.75, 0.99999994, [0, -1], b)):
        got = m.verify_tree(p, q, ints([[0, tok]]), ints([[-1, 0]]), torch.tensor([[u0, u1]], device="cuda"))
        assert [x.tolist() for x in got] == [[path], [sum(x >= 0 for x in path)], [token]], (tok, u1, u0)


def test_siblings_of_one_token():
    # a token drawn twice: turned down once, its rest is 0, and it is turned down again
    v = 50
    g = gen(5)
    p, q = distributions(g, 40, 4, v, torch.float32, error=2.0)
    parents = ints([[-1, 0, 0, 0]] * 40)
    tokens = drawn(g, q, parents)[:, 1:2].expand(40, 4).contiguous()
    path = compare(p, q, tokens, parents, torch.rand(40, 4, generator=g, device="cuda"))[0]
    assert any(x[1] == -1 for x in path) and not any(x[1] in (2, 3) for x in path)


def test_values_that_are_no_probabilities():
    # NaN, infinities and negative values count as 0; rows of nothing give no token
    v, inf, nan = 70, math.inf, math.nan
    g = gen(6)
    p, q = distributions(g, 6, 3, v, torch.float32)
    bad = torch.tensor([nan, inf, -inf, -1.0, -0.0], device="cuda")
    p[:, :, 7:12] = bad
    q[:, :, 9:14] = bad
    p[4], q[5] = nan, -3.0
    for dtype in (torch.float32, torch.float16):
        parents = ints([[-1, 0, 1], [-1, 0, 0], [-1, 0, 1], [-1, 0, 0], [-1, 0, 0], [-1, 0, 1]])
        tokens = ints([[0, 5, 8], [0, 9, 10], [1, 13, 2], [0, 7, 1], [0, 3, 4], [0, 8, 20]])
        u = torch.rand(6, 3, generator=g, device="cuda")
        want = compare(p.to(dtype), q.to(dtype), tokens, parents, u)
        assert want[2][4] == -1 and want[1][4] == 1


def test_tokens_outside_the_vocabulary():
    v = 40
    g = gen(7)
    p, q = distributions(g, 5, 3, v, torch.float32)
    tokens = ints([[-7, -1, 3], [99, v, 3], [0, 2 ** 31 - 1, 3], [0, -2 ** 31, 3], [v, 5, v]])
    compare(p, q, tokens, ints([[-1, 0, 0]] * 5), torch.rand(5, 3, generator=g, device="cuda"))


def test_draft_covers_target():
    # equal rows: every token is taken; a draft above the target everywhere leaves nothing
    # of it, and the target itself is drawn from
    v = 129
    g = gen(8)
    p, _ = distributions(g, 4, 2, v, torch.float32)
    parents = ints([[-1, 0]] * 4)
    u = torch.rand(4, 2, generator=g, device="cuda")
    path, count, _ = m.verify_tree(p, p, drawn(g, p, parents), parents, u)
    assert (count == 2).all()
    u[:, 1] = 0.9999
    path, count, token = m.verify_tree(p, p * 2, drawn(g, p, parents), parents, u)
    assert (count == 1).all()
    sums = p[:, 0].double().cumsum(-1)
    assert token.tolist() == (sums <= u[:, :1].double() * sums[:, -1:]).sum(-1).tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_strides_and_alignments(dtype):
    # rows inside wider ones, at every start, in other orders; what lies between is not read
    b, n, v = 3, 4, 1001
    g, r = gen(9), np.random.RandomState(9)
    p, q = distributions(g, b, n, v, dtype)
    parents = ints(trees(r, b, n, "random"))
    tokens, u = drawn(g, q, parents), torch.rand(b, n, generator=g, device="cuda")
    want = [x.tolist() for x in m.verify_tree(p, q, tokens, parents, u)]
    assert want == list(pref.verify(p, q, tokens, parents, u)[:3])
    for lead in range(0, 9):
        for order in (0, 1):
            def widen(x, extra):
                shape = (b, n, v + extra) if order == 0 else (n, b, v + extra)
                w = torch.full(shape, 0.5, dtype=dtype, device="cuda")
                w = w if order == 0 else w.transpose(0, 1)
                w[:, :, lead:lead + v] = x
                return w[:, :, lead:lead + v]
            got = m.verify_tree(widen(p, 9), widen(q, 12), tokens, parents, u)
            assert [x.tolist() for x in got] == want, (lead, order)
    # one row for all nodes, one sequence for all
    same = p[:1, :1].expand(b, n, v)
    compare(same, q, tokens, parents, u)


def test_captured_and_on_streams():
    b, n, v = 4, 5, 3001
    g, r = gen(10), np.random.RandomState(10)
    p, q = distributions(g, b, n, v, torch.float32)
    parents = ints(trees(r, b, n, "random"))
    tokens, u = drawn(g, q, parents), torch.rand(b, n, generator=g, device="cuda")
    out = [torch.empty(k, dtype=torch.int32, device="cuda") for k in ((b, n), b, b)]
    m.verify_tree(p, q, tokens, parents, u, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = m.verify_tree(p, q, tokens, parents, u, out=out)
    for _ in range(4):
        u.copy_(torch.rand(b, n, generator=g, device="cuda"))
        parents.copy_(ints(trees(r, b, n, "holes")))
        tokens.copy_(drawn(g, q, parents))
        graph.replay()
        want = list(pref.verify(p, q, tokens, parents, u)[:3])
        assert [x.tolist() for x in res] == want
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        got = [m.verify_tree(p, q, tokens, parents, u, stream=s) for _ in range(3) for s in streams]
        torch.cuda.synchronize()
        for x in got:
            assert [y.tolist() for y in x] == want


@pytest.mark.parametrize("kind", ["chain", "star"])
def test_distribution_is_the_targets(kind):
    # what comes first after the root (the first node kept, else the next token) is
    # distributed as the target's own samples: each frequency within 6 standard
    # deviations of its probability
    b, n, v = 200000, 3, 8
    g = gen(12)
    p, q = distributions(g, 1, n, v, torch.float32, spread=1.0, error=1.5)
    parents = ints(trees(None, 1, n, kind)).expand(b, n).contiguous()
    pe, qe = p.expand(b, n, v), q.expand(b, n, v)
    rows = torch.gather(q, 1, parents[:1].long().clamp(min=0)[:, :, None].expand(1, n, v)).cumsum(-1)[0]   # [n, v]
    at = torch.rand(n, b, generator=g, device="cuda")
    tokens = torch.searchsorted(rows.contiguous(), at * rows[:, -1:], right=True).clamp(max=v - 1).t()
    tokens = tokens.to(torch.int32).contiguous()
    path, count, token = m.verify_tree(pe, qe, tokens, parents, torch.rand(b, n, generator=g, device="cuda"))
    first = torch.where(count > 1, tokens.gather(1, path[:, 1:2].long().clamp(min=0))[:, 0], token)
    share = torch.bincount(first.long(), minlength=v).double() / b
    want = p[0, 0].double()
    assert ((share - want).abs() <= 6 * (want * (1 - want) / b).sqrt()).all()
    assert (count > 1).any() and (count == 1).any()
