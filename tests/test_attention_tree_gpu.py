"""Attention of drafted trees over a batch of KV caches, against a 64-bit
reference that loops over sequences and nodes (GPU).

Tolerance of a value o = sum_j w_j v_j, from the arithmetic: a probability is
rounded to fp16 before the product with V (2^-11 of it; 2^-25 of the row's
reference where fp16 is subnormal, over n keys: 2^-25 n max|v|), its exponent
comes from an fp32 score (products and sums of at most 128 terms over sum |q k|
scale = span: below 2 span 2^-22 with the exponential's own 2^-22), the sums are
fp32 (2^-20), and the result is rounded once (2^-11 of it)."""
import math

import numpy as np
import pytest

import swiglu_block_quantized_gb300 as m

torch = pytest.importorskip("torch")
import _serving_ref as ref   # noqa: E402

pytestmark = pytest.mark.gpu

F16, Q8 = m.KV_F16, m.Q8_0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()
    m.load()
    yield
    assert m.check_device_status() == m.OK


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make_cache(g, codec, b, hkv, c, d, scale=1.0):
    x = torch.randn(b, hkv, c, d, generator=g, device="cuda") * scale
    return x.half() if codec == F16 else ref.pack(*ref.encode(x.double()))


def tree(n, seed, kind):
    """parents of n nodes: a chain, a star, a random tree, one with unused
    nodes (and children of unused ones), or none used."""
    r = np.random.RandomState(seed)
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] * n
    p = [int(r.randint(max(-1, i - 6), i)) if i else -1 for i in range(n)]
    if kind == "holes":
        for i in range(n):
            if r.rand() < 0.25:
                p[i] = [-2, i, i + 3, 2 ** 31 - 1, -2 ** 31][r.randint(5)]
    if kind == "none":
        p = [-2] * n
    return p


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check(o, want, tol, what=""):
    bad = ~((o.double() - want).abs() <= tol)
    if bad.any():
        i = bad.nonzero()[0]
        raise AssertionError("%s: %d of %d values off; first at %s: %r, not %r (tolerance %r)" % (
            what, int(bad.sum()), bad.numel(), i.tolist(), o[tuple(i)].item(), want[tuple(i)].item(),
            tol[tuple(i)].item()))


def run(codec, h, hkv, d, c, pasts, parents, seed=0, scale=None, kscale=1.0, **kw):
    b, n = len(pasts), len(parents[0])
    g = gen(seed)
    q = torch.randn(h, b * n, d, generator=g, device="cuda").half()
    kc, vc = make_cache(g, codec, b, hkv, c, d, kscale), make_cache(g, codec, b, hkv, c, d)
    o = m.attention_tree(q, kc, vc, codec, ints(pasts), ints(parents), scale=scale, **kw)
    want, tol = ref.tree_attention(q, kc, vc, codec, pasts, parents, float(d) ** -0.5 if scale is None else scale)
    check(o, want, tol, "h=%d/%d d=%d n=%d" % (h, hkv, d, n))
    return o


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,hkv", [(4, 4), (8, 2), (3, 1), (24, 4)])
@pytest.mark.parametrize("n,past", [(1, 0), (1, 1), (1, 127), (1, 128), (1, 700), (2, 126), (7, 0), (16, 300),
                                    (33, 250), (64, 129)])
def test_shapes(codec, d, h, hkv, n, past):
    run(codec, h, hkv, d, (past + n + 7) // 4 * 4, [past], [tree(n, n, "random")], seed=n + past)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("kind", ["chain", "star", "random", "holes", "none"])
@pytest.mark.parametrize("n", [1, 5, 65, 130, 256])
def test_trees(codec, kind, n):
    run(codec, 4, 2, 64, 520, [200], [tree(n, n, kind)], seed=n)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
def test_ragged_batch(codec, d):
    # sequences of every length, one empty with no used node, trees of
    # different sizes padded to one
    pasts = [0, 1, 63, 64, 500, 1000, 0, 129, 128, 127, 383, 777]
    n = 12
    parents = [tree(n, b, ["random", "holes", "chain", "star"][b % 4]) for b in range(len(pasts))]
    parents[6] = [-2] * n
    parents[3] = [-1] + [-2] * (n - 1)
    o = run(codec, 8, 2, d, 1012, pasts, parents, seed=d)
    assert (o.view(len(pasts), n, -1)[6] == 0).all()


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("h,hkv,n", [(16, 1, 40), (32, 1, 9), (71, 1, 3), (40, 8, 31), (8, 8, 200)])
def test_group_sizes(codec, h, hkv, n):
    run(codec, h, hkv, 128, 400, [180], [tree(n, 5, "random")], seed=h)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
def test_long_split(codec, d):
    # keys split over many CTAs, merged; without a workspace no split: the
    # same result up to the order of fp32 sums and the rounding of P
    pasts, n = [6000, 900], 8
    parents = [tree(n, 1, "random"), tree(n, 2, "random")]
    a = run(codec, 8, 2, d, 6016, pasts, parents, seed=3)
    b = run(codec, 8, 2, d, 6016, pasts, parents, seed=3, workspace=False)
    assert (a.double() - b.double()).abs().max() < 4e-3


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("scale", [0.0, -0.3, 0.9])
def test_scales(codec, scale):
    run(codec, 8, 2, 128, 900, [800], [tree(9, 4, "random")], seed=8, scale=scale, kscale=2.0)


def test_growing_scores():
    # keys that grow along the cache: the running maximum rises by far more
    # than 2^8 from tile to tile
    g = gen(31)
    h, hkv, d, c, n = 8, 2, 128, 1600, 6
    q = torch.randn(h, n, d, generator=g, device="cuda").half()
    ramp = torch.linspace(0.1, 14, c, device="cuda")[None, None, :, None]
    kc = (torch.randn(1, hkv, c, d, generator=g, device="cuda") * ramp).half()
    vc = make_cache(g, F16, 1, hkv, c, d)
    p = [tree(n, 3, "random")]
    for kk in (kc, kc.flip(2).contiguous()):
        o = m.attention_tree(q, kk, vc, F16, ints([1590]), ints(p))
        want, tol = ref.tree_attention(q, kk, vc, F16, [1590], p, d ** -0.5)
        check(o, want, tol, "growing")


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("past", [-5, -2 ** 31, 250, 256, 300, 2 ** 31 - 1])
def test_past_outside_the_cache(codec, past):
    # clamped to [0, C]; nodes whose row is past the end have no key
    run(codec, 4, 2, 64, 256, [past, 100], [tree(10, 2, "random"), tree(10, 3, "holes")], seed=5)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("past", [0, 70, 128, 300])
def test_poison_in_unseen_rows(codec, d, past):
    # NaN and infinities in every row that a node does not see change nothing:
    # the rows behind the tree, those of unused nodes, and other branches
    g = gen(41)
    h, hkv, n, c = 8, 2, 12, 448
    q = torch.randn(h, 2 * n, d, generator=g, device="cuda").half()
    kc, vc = make_cache(g, codec, 2, hkv, c, d), make_cache(g, codec, 2, hkv, c, d)
    pasts = [past, 33]
    parents = [[-1, -1, 0, 1, 2, 3, -2, 4, 5, 6, 7, 8], tree(n, 7, "random")]
    clean = m.attention_tree(q, kc, vc, codec, ints(pasts), ints(parents))
    want, tol = ref.tree_attention(q, kc, vc, codec, pasts, parents, d ** -0.5)
    check(clean, want, tol, "clean")
    bad = torch.tensor([0x7E00, 0x7C00, -0x400], dtype=torch.int16, device="cuda").view(torch.float16)

    def poison(cache, s, rows):
        for j, r in enumerate(rows):
            if codec == F16:
                cache[s, :, r] = bad[j % 3]
            else:
                cache[s, :, r, :2] = bad[j % 3:j % 3 + 1].view(torch.uint8)

    for cache in (kc, vc):
        poison(cache, 0, [r for s in (6, 9) for r in [past + s]] + list(range(past + n, c)))
        poison(cache, 1, list(range(33 + n, c)))
    o = m.attention_tree(q, kc, vc, codec, ints(pasts), ints(parents))
    assert torch.equal(o, clean)
    # the branch of node 1 (nodes 1, 3, 5, 8, 11 ...) poisoned: the others
    # keep their bits, and its own nodes show it
    used, seen = ref.used_and_seen(parents[0])
    poison(vc, 0, [past + 1])
    poison(kc, 0, [past + 3])
    o = m.attention_tree(q, kc, vc, codec, ints(pasts), ints(parents)).view(2, n, h, d)
    clean = clean.view(2, n, h, d)
    for i in range(n):
        if used[i] and 1 in seen[i]:
            # (a Q8_0 row is poisoned through the scale of its first block)
            assert not torch.isfinite(o[0, i, :, :32 if codec == Q8 else d]).any()
        else:
            assert torch.equal(o[0, i], clean[0, i])
    assert torch.equal(o[1], clean[1])


def test_infinite_value_of_one_dimension():
    # one infinite component of a seen V row reaches that component of the
    # nodes that see it, and nothing else
    g = gen(43)
    h, hkv, d, n, c, past = 4, 2, 64, 4, 256, 100
    q = torch.randn(h, n, d, generator=g, device="cuda").half()
    kc, vc = make_cache(g, F16, 1, hkv, c, d), make_cache(g, F16, 1, hkv, c, d)
    p = ints([[-1, 0, -1, 1]])
    clean = m.attention_tree(q, kc, vc, F16, ints([past]), p).view(n, h, d)
    vc[0, 1, past + 1, 5] = -math.inf        # node 1, KV head 1 (heads 2, 3)
    o = m.attention_tree(q, kc, vc, F16, ints([past]), p).view(n, h, d)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[1, 2:, 5] = hit[3, 2:, 5] = True
    assert (o[hit] == -math.inf).all() and torch.equal(o[~hit], clean[~hit])


@pytest.mark.parametrize("codec", [F16, Q8])
def test_one_token_matches_attention(codec):
    # trees of one node over one sequence are the causal decode call
    g = gen(51)
    h, hkv, d, c = 32, 8, 128, 640
    q = torch.randn(h, 1, d, generator=g, device="cuda").half()
    kc, vc = make_cache(g, codec, 1, hkv, c, d), make_cache(g, codec, 1, hkv, c, d)
    a = m.attention(q, kc[0], vc[0], codec, hkv, c, q_offset=500)
    b = m.attention_tree(q, kc, vc, codec, ints([500]), ints([[-1]]))
    assert (a.double() - b.double()).abs().max() < 2e-3
    assert torch.equal(b, m.attention_tree(q, kc[0], vc[0], codec, ints([500]), ints([-1])))


@pytest.mark.parametrize("codec", [F16, Q8])
def test_graph_follows_past_and_streams(codec):
    # a captured call reads past and parents at replay; eager calls on two
    # streams at once, each with its own workspace, give the same bits
    h, hkv, d, c, n, b = 8, 2, 128, 2048, 6, 3
    g = gen(61)
    q = torch.randn(h, b * n, d, generator=g, device="cuda").half()
    kc, vc = make_cache(g, codec, b, hkv, c, d), make_cache(g, codec, b, hkv, c, d)
    past, parents = ints([10, 20, 30]), ints([tree(n, s, "random") for s in range(b)])
    out = torch.empty(b * n, h * d, dtype=torch.float16, device="cuda")
    m.attention_tree(q, kc, vc, codec, past, parents, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.attention_tree(q, kc, vc, codec, past, parents, out=out)
    for pasts, seed in (([10, 20, 30], 0), ([2000, 0, 777], 5), ([1500, 1400, 1], 9)):
        past.copy_(ints(pasts))
        new = [tree(n, seed + s, "holes") for s in range(b)]
        parents.copy_(ints(new))
        graph.replay()
        want, tol = ref.tree_attention(q, kc, vc, codec, pasts, new, d ** -0.5)
        check(out, want, tol, "replay %s" % pasts)
        got = []
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(4):
            for s in streams:
                got.append(m.attention_tree(q, kc, vc, codec, past, parents, stream=s))
        torch.cuda.synchronize()
        for o in got:
            assert torch.equal(o, out)


@pytest.mark.parametrize("codec", [F16, Q8])
def test_cache_past_32_bits(codec):
    # the last sequence's rows start past 2^32 bytes
    d, hkv, b, n, h = 128, 4, 2, 3, 8
    rb = 2 * d if codec == F16 else d // 32 * 34
    c = 2 ** 33 // (b * hkv * rb) // 4 * 4 + 400
    past = c - n - 2
    g = gen(71)
    kc = torch.zeros(b, hkv, c, rb, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    tail = 300
    for cache in (kc, vc):
        part = make_cache(g, codec, b, hkv, tail, d)
        cache[:, :, c - tail:] = part.view(torch.uint8)
    q = torch.randn(h, b * n, d, generator=g, device="cuda").half() * 4
    kc, vc = (x.view(torch.float16) if codec == F16 else x for x in (kc, vc))
    parents = [tree(n, 1, "random")] * 2
    # keys of zeros have score 0 and value 0: the tail alone plus their count
    o = m.attention_tree(q, kc, vc, codec, ints([past, past]), ints(parents)).view(b, n, h, d)
    for s in range(b):
        _, seen = ref.used_and_seen(parents[s])
        k, v = (ref.values(x[s][:, c - tail:], codec).repeat_interleave(h // hkv, 0) for x in (kc, vc))
        for i in range(n):
            idx = torch.tensor(list(range(tail - n - 2)) + [tail - n - 2 + a for a in seen[i]], device="cuda")
            x = torch.einsum("hd,hjd->hj", q[:, s * n + i].double(), k[:, idx]) * d ** -0.5
            top = x.amax(-1, keepdim=True).clamp(min=0)
            w = (x - top).exp()
            zeros = (past - (tail - n - 2)) * (-top).exp()
            total = w.sum(-1, keepdim=True) + zeros
            want = torch.einsum("hj,hjd->hd", w, v[:, idx]) / total
            mag = torch.einsum("hj,hjd->hd", w, v[:, idx].abs()) / total
            assert ((o[s, i].double() - want).abs() <= 2.0 ** -9 * mag + 2.0 ** -20).all()
