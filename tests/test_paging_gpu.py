"""The operators of the paged serving loop against plain references (GPU): positions of
several axes, page plans, attention of one new token over pages, verification of drafted
trees.

Attention's tolerance is that of test_attention_tree_gpu (the same arithmetic: fp32
scores, sums and products, probabilities rounded to fp16), rotations' that of
test_kv_ops_gpu; plans and verified trees have one right answer.  A verified tree is
compared where no decision lies within 2^-40 of its border (the operator's sums are good
to 2^-44, the reference's to 2^-45 for the rows here)."""
import math

import numpy as np
import pytest

import swiglu_block_quantized_gb300 as m

torch = pytest.importorskip("torch")
import _paging_ref as pref   # noqa: E402
import _serving_ref as ref   # noqa: E402
from test_attention_tree_gpu import check, gen, ints, make_cache   # noqa: E402
from test_kv_ops_gpu import new_cache, randn, raw, rope_tol   # noqa: E402

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


# ---------------------------------------------------------------- several axes

@pytest.mark.parametrize("d,rot,sections", [(64, 64, [16, 8, 8]), (128, 128, [24, 20, 20]), (128, 96, [16, 32]),
                                            (64, 16, [1, 1, 1, 1, 1, 1, 1, 1])])
@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("dealt", [False, True])
@pytest.mark.parametrize("h,rows", [(1, 1), (5, 33), (32, 300)])
def test_rope_axes(d, rot, sections, inter, dealt, h, rows):
    if dealt and sections == [16, 32]:
        pytest.skip("the first axis has the rest")
    g = gen(d + rows)
    x = randn(g, rows, h, d).transpose(0, 1)
    pos = torch.randint(-2000, 200000, (len(sections), rows), generator=g, device="cuda").to(torch.int32)
    freqs, _ = m.rope_freqs(rot)
    axes = m.rope_axes(sections, dealt)
    y = m.rope(x, pos, freqs, layout=inter, mscale=1.5, axes=axes)
    # pair by pair: the rotation of one axis, and of its values alone
    want, size = torch.empty_like(x, dtype=torch.float64), torch.empty_like(x, dtype=torch.float64)
    first = torch.arange(0, rot, 2) if inter else torch.arange(rot // 2)
    second = first + (1 if inter else rot // 2)
    for a in range(len(sections)):
        wa, sa = ref.rotate(x, pos[a], ref.inv_freqs(rot), inter, 1.5)
        mine = (axes.cpu() == a).nonzero()[:, 0]
        for part in (first[mine], second[mine]):
            want[..., part], size[..., part] = wa[..., part], sa[..., part]
    want[..., rot:], size[..., rot:] = x[..., rot:].double(), 0
    assert ((y.double() - want).abs() <= rope_tol(want, size)).all()
    assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("inter", [0, 1])
def test_one_axis_is_rope(inter):
    # all pairs on one axis are rope's bits; a pair without an axis is not turned
    g = gen(7)
    x = randn(g, 6, 70, 128)
    pos = torch.randint(0, 2 ** 31 - 1, (3, 70), generator=g, device="cuda").to(torch.int32)
    freqs, _ = m.rope_freqs(128)
    for a in range(3):
        y = m.rope(x, pos, freqs, layout=inter, axes=torch.full((64,), a, dtype=torch.int32, device="cuda"))
        assert torch.equal(y, m.rope(x, pos[a].contiguous(), freqs, layout=inter))
    for bad in (-1, 3, 2 ** 31 - 1, -2 ** 31):
        axes = torch.full((64,), bad, dtype=torch.int32, device="cuda")
        assert torch.equal(m.rope(x, pos, freqs, layout=inter, axes=axes), x)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d,page", [(64, 8), (128, 24), (128, 64)])
def test_kv_write_axes_into_pages(codec, d, page):
    # the rows are those of a rotation first and a write after it (fp16), and of the
    # formula (Q8_0: quantised from the fp32 rotation, so within a code of the fp16 path);
    # everything else stays as it was
    g = gen(d + page)
    hkv, h, n, pages = 3, 6, 37, 11
    q, k, v = randn(g, h, n, d), randn(g, hkv, n, d), randn(g, hkv, n, d)
    pos = torch.randint(0, 5000, (3, n), generator=g, device="cuda").to(torch.int32)
    freqs, _ = m.rope_freqs(d)
    axes = m.rope_axes([d // 2 - 16, 8, 8])
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:n].to(torch.int32)
    slots[5], slots[11] = -1, pages * page
    kc, vc = (new_cache(codec, pages, hkv, page, d) for _ in range(2))
    qo = m.kv_write(k, v, kc, vc, codec, slots, pos=pos, freqs=freqs, axes=axes, q=q)
    assert torch.equal(qo, m.rope(q, pos, freqs, axes=axes))
    kr = m.rope(k, pos, freqs, axes=axes)
    k2, v2 = (new_cache(codec, pages, hkv, page, d) for _ in range(2))
    m.kv_write(kr, v, k2, v2, codec, slots)
    assert torch.equal(raw(vc), raw(v2))
    if codec == F16:
        assert torch.equal(raw(kc), raw(k2))
    else:
        a, b = (ref.values(c, Q8) for c in (kc, k2))
        # a code, and the rotation's own rounding, of a block of magnitude at most 8
        assert ((a - b).abs() <= 8 / 127 * 1.01).all()
        used = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
        used[slots[(slots >= 0) & (slots < pages * page)].long()] = True
        same = (raw(kc) == raw(k2)).all(-1).transpose(0, 1).reshape(hkv, -1)
        assert same[:, ~used].all()


# ---------------------------------------------------------------- page plans

def plan_state(r, b, page, width, pages, most):
    """A consistent state: every sequence holds its rows' pages and a few more."""
    past = [int(r.randint(0, most + 1)) for _ in range(b)]
    ids = list(map(int, r.permutation(pages)))
    held, table = [], []
    for s in range(b):
        h = min(width, -(-past[s] // page) + int(r.randint(0, 3)), len(ids))
        past[s] = min(past[s], h * page)
        table.append([ids.pop() for _ in range(h)] + [-1] * (width - h))
        held.append(h)
    free = ids + [int(x) for x in r.randint(0, pages, size=pages - len(ids))]
    return past, held, table, free, len(ids)


def run_plan(past, new, table, held, free, n_free, page, tokens, out=None):
    t, h, f, n = ints(table), ints(held), ints(free), ints([n_free])
    got = m.page_plan(ints(past), ints(new), t, h, f, n, page, tokens, out=out)
    return [x.tolist() for x in got] + [t.tolist(), h.tolist(), f.tolist(), n.tolist()[0]]


NAMES = ("slots", "pos", "lengths", "starts", "table", "held", "free", "n_free")


def check_plan(past, new, table, held, free, n_free, page, tokens):
    got = run_plan(past, new, table, held, free, n_free, page, tokens)
    want = pref.plan(past, new, table, held, free, n_free, page, tokens)
    for name, x, y in zip(NAMES, got, want):
        assert x == y, name
    return got


@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("b", [1, 3, 32, 33, 200, 1025])
def test_plan(b, page):
    r = np.random.RandomState(b * 100 + page)
    for ended, scarce, room in ((0.0, False, 1.0), (0.3, False, 1.0), (0.3, True, 1.0), (0.1, False, 0.6), (1.0, True, 1.0)):
        most = 5 * page
        width = 9
        pages = b * width if not scarce else b * 4 + 1
        past, held, table, free, n_free = plan_state(r, b, page, width, pages, most)
        new = [-1 - int(r.randint(5)) if r.rand() < ended else int(r.randint(0, 3 * page + 2)) for _ in range(b)]
        tokens = max(1, int(room * sum(max(n, 0) for n in new)) + (3 if room == 1.0 else 0))
        check_plan(past, new, table, held, free, n_free, page, tokens)


@pytest.mark.parametrize("tokens", [1, 2, 1023, 1024, 1025, 40000])
def test_plan_one_sequence(tokens):
    # a whole prompt, and the pages of it
    page, width = 16, 2600
    free = list(range(3000))[::-1]
    got = check_plan([0], [tokens], [[-1] * width], [0], free, 3000, page, tokens)
    assert got[0] == list(range(tokens)) and got[5] == [-(-tokens // page)]
    check_plan([5], [tokens], [[7, 9] + [-1] * (width - 2)], [2], free, 10, page, tokens + 5)


def test_plan_again_changes_nothing():
    r = np.random.RandomState(3)
    past, held, table, free, n_free = plan_state(r, 20, 8, 12, 300, 50)
    new = [int(r.randint(0, 20)) for _ in range(20)]
    a = run_plan(past, new, table, held, free, n_free, 8, 400)
    assert run_plan(past, new, a[4], a[5], a[6], a[7], 8, 400) == a


def test_plan_values_out_of_range():
    # counts and lengths outside their range count as the nearest in it; entries that are
    # no pages give no slots
    page, width, pages = 4, 3, 6
    table = [[2, 77, 5], [-9, 1, 0], [3, 3, 3], [4, -1, -1]]
    for past in ([-5, 2, 1, 0], [2 ** 31 - 1, 4, 11, -2 ** 31]):
        for held in ([9, 2, 3, -4], [3, -1, 2 ** 31 - 1, 1]):
            for n_free in (-3, 0, 2, 6, 99, 2 ** 31 - 1):
                for new in ([3, 5, 1, 2], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0], [-1, -1, -1, -1]):
                    check_plan(past, new, table, held, [5, 0, 1, 2, 3, 4], n_free, page, 40)


def test_plan_largest_pages():
    # past + new + page are past 32 bits
    big = 2 ** 31 - 1
    for page in (big, 2 ** 30):
        for past in (big, page, page - 1, 5, 0):
            check_plan([past], [40], [[-1]], [0], [0], 1, page, 40)


def test_plan_captured():
    # a captured plan follows the lengths; pages come and go over many steps, and no page
    # is ever held twice
    r = np.random.RandomState(11)
    b, page, width, pages, tokens = 7, 8, 10, 60, 90
    past, new = ints([0] * b), ints([0] * b)
    table, held = ints([[-1] * width for _ in range(b)]), ints([0] * b)
    free, n_free = ints(list(map(int, r.permutation(pages)))), ints([pages])
    state = ([[-1] * width for _ in range(b)], [0] * b, free.tolist(), pages)
    out = [torch.empty(k, dtype=torch.int32, device="cuda") for k in (tokens, tokens, b, b + 1)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = m.page_plan(past, new, table, held, free, n_free, page, tokens, out=out)
    at = [0] * b
    for step in range(60):
        want_new = [-1 if r.rand() < 0.15 else int(r.randint(0, 13)) for _ in range(b)]
        past.copy_(ints(at)), new.copy_(ints(want_new))
        graph.replay()
        want = pref.plan(at, want_new, *state, page, tokens)
        got = [x.tolist() for x in res] + [table.tolist(), held.tolist(), free.tolist(), n_free.tolist()[0]]
        assert got == list(want), step
        state = want[4:8]
        mine = [e for s in range(b) for e in want[4][s][:want[5][s]]]
        assert sorted(mine + want[6][:want[7]]) == list(range(pages))
        at = [0 if n < 0 else int(r.randint(max(0, x - 3), x + 1)) for x, n in zip(want[2], want_new)]


def test_plan_largest_batch():
    # 4096 sequences, more tokens than a cluster takes in one go
    r = np.random.RandomState(6)
    past, held, table, free, n_free = plan_state(r, 4096, 16, 12, 4096 * 10, 100)
    new = [int(r.randint(-1, 120)) for _ in range(4096)]
    check_plan(past, new, table, held, free, n_free, 16, 200000)


# ---------------------------------------------------------------- attention over pages

def tables(r, lengths, page, width, pages):
    """Block tables of distinct random pages; entries behind a sequence's last page are
    unusable."""
    ids = list(map(int, r.permutation(pages)))
    return [[ids.pop() for _ in range(-(-n // page))] + [[-1, pages, 2 ** 31 - 1, -2 ** 31][s % 4]] *
            (width - -(-n // page)) for s, n in enumerate(lengths)]


def pools(g, codec, pages, hkv, page, d, kscale=1.0):
    return make_cache(g, codec, pages, hkv, page, d, kscale), make_cache(g, codec, pages, hkv, page, d)


def run_paged(codec, h, hkv, d, page, lengths, seed=0, scale=None, kscale=1.0, spare=3, **kw):
    r = np.random.RandomState(seed)
    g = gen(seed)
    width = max(1, -(-max(lengths) // page)) + 1
    pages = sum(-(-n // page) for n in lengths) + spare
    kc, vc = pools(g, codec, pages, hkv, page, d, kscale)
    q = randn(g, h, len(lengths), d)
    table = ints(tables(r, lengths, page, width, pages))
    o = m.attention_paged(q, kc, vc, codec, table, ints(lengths), scale=scale, **kw)
    want, tol = pref.paged_attention(q, kc, vc, codec, table, lengths, float(d) ** -0.5 if scale is None else scale)
    check(o, want, tol, "h=%d/%d d=%d page=%d" % (h, hkv, d, page))
    return o


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,hkv", [(4, 4), (8, 2), (3, 1), (32, 8)])
@pytest.mark.parametrize("page", [8, 16, 24, 64, 256])
def test_paged_lengths(codec, d, h, hkv, page):
    run_paged(codec, h, hkv, d, page, [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300, 0],
              seed=page + d)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [0, 1, 5, 16, 40, 64, 100, 511, 700, 3000, 20001])
def test_paged_one_sequence(codec, d, n):
    run_paged(codec, 8, 2, d, 16, [n], seed=n)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("h,hkv", [(1, 1), (2, 1), (5, 1), (6, 1), (7, 1), (8, 1), (9, 1), (12, 1), (16, 1), (17, 1),
                                   (24, 1), (33, 1), (71, 1), (36, 3), (64, 8)])
def test_paged_groups(codec, h, hkv):
    for d in (64, 128):
        run_paged(codec, h, hkv, d, 32, [130, 0, 41, 700], seed=h)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
def test_paged_ragged_batches(codec, d):
    # many sequences of very different lengths, and long ones beside empty ones
    r = np.random.RandomState(d)
    run_paged(codec, 8, 2, d, 16, [int(x) for x in np.exp(r.uniform(0, 8, 300))], seed=1)
    run_paged(codec, 4, 1, d, 64, [0, 0, 15000, 0, 1, 0, 9000, 0, 0, 64], seed=2)
    run_paged(codec, 16, 8, d, 8, [3] * 40, seed=3)
    run_paged(codec, 4, 4, d, 128, [int(x) for x in r.randint(0, 40, 1500)], seed=4)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
def test_paged_without_workspace(codec, d):
    # the split joined, or no split: the same result up to fp32 sums and P's rounding
    lengths = [6000, 900, 0, 77]
    a = run_paged(codec, 8, 2, d, 16, lengths, seed=5)
    b = run_paged(codec, 8, 2, d, 16, lengths, seed=5, workspace=False)
    assert (a.double() - b.double()).abs().max() < 4e-3
    need = m.load().m4q_attention_paged_workspace(codec, 4, 8, 2, 440, 16, 376, d)
    for size in (16, max(16, need - 16), need + 1024):   # too small: no split
        c = run_paged(codec, 8, 2, d, 16, lengths, seed=5,
                      workspace=torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda"))
        assert torch.equal(c, a) or torch.equal(c, b)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("scale", [0.0, -0.3, 0.9])
def test_paged_scales(codec, scale):
    run_paged(codec, 8, 2, 128, 16, [800, 3], seed=8, scale=scale, kscale=2.0)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
def test_paged_growing_scores(codec, d):
    # keys that grow along the sequence: the running maximum rises by far more than 2^8
    g = gen(31)
    h, hkv, page, n = 8, 2, 16, 1600
    q = randn(g, h, 1, d)
    ramp = torch.linspace(0.1, 14, n, device="cuda").view(n // page, 1, page, 1)
    x = torch.randn(n // page, hkv, page, d, generator=g, device="cuda") * ramp
    kc = x.half() if codec == F16 else ref.pack(*ref.encode(x.double()))
    vc = make_cache(g, codec, n // page, hkv, page, d)
    for order in (range(n // page), range(n // page - 1, -1, -1)):
        table = ints([list(order)])
        for length in (n, n - 5):
            o = m.attention_paged(q, kc, vc, codec, table, ints([length]))
            want, tol = pref.paged_attention(q, kc, vc, codec, table, [length], d ** -0.5)
            check(o, want, tol, "growing")


@pytest.mark.parametrize("codec", [F16, Q8])
def test_paged_lengths_outside_the_table(codec):
    # clamped to [0, W * page]; entries that are no pages are not seen
    g = gen(9)
    h, hkv, d, page, pages = 4, 2, 64, 16, 20
    kc, vc = pools(g, codec, pages, hkv, page, d)
    table = ints([[0, 1, 2, 3], [4, -1, 5, 20], [-1, 2 ** 31 - 1, -2 ** 31, 99], [6, 7, 8, 9], [10, 11, 12, 13]])
    lengths = [2 ** 31 - 1, 64, 50, -1, -2 ** 31]
    q = randn(g, h, 5, d)
    o = m.attention_paged(q, kc, vc, codec, table, ints(lengths))
    want, tol = pref.paged_attention(q, kc, vc, codec, table, lengths, d ** -0.5)
    check(o, want, tol, "clamped")
    assert (o[2:] == 0).all()


BAD = [0x7E00, 0x7C00, -0x400]


def poison(cache, codec, rows):
    """Rows (page, place) of a pool made NaN, inf or -inf (Q8_0: their scales)."""
    bad = torch.tensor(BAD, dtype=torch.int16, device="cuda").view(torch.float16)
    for j, (p, r) in enumerate(rows):
        if codec == F16:
            cache[p, :, r] = bad[j % 3]
        else:
            cache[p, :, r].unflatten(-1, (-1, 34))[..., :2] = bad[j % 3:j % 3 + 1].view(torch.uint8)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [8, 40, 128])
def test_paged_poison_in_unseen_rows(codec, d, page):
    # whatever the rows behind the last one and the pages of nobody hold
    r, g = np.random.RandomState(page), gen(41)
    h, hkv, lengths = 8, 2, [1, 7, 20, 64, 129, 300, 0]
    width, pages = -(-300 // page) + 1, sum(-(-n // page) for n in lengths) + 2
    kc, vc = pools(g, codec, pages, hkv, page, d)
    rows = tables(r, lengths, page, width, pages)
    table, q = ints(rows), randn(g, h, len(lengths), d)
    clean = m.attention_paged(q, kc, vc, codec, table, ints(lengths))
    want, tol = pref.paged_attention(q, kc, vc, codec, table, lengths, d ** -0.5)
    check(clean, want, tol, "clean")
    seen = {(rows[s][j // page], j % page) for s, n in enumerate(lengths) for j in range(n)}
    for cache in (kc, vc):
        poison(cache, codec, [(p, i) for p in range(pages) for i in range(page) if (p, i) not in seen])
    assert torch.equal(m.attention_paged(q, kc, vc, codec, table, ints(lengths)), clean)
    # a seen row: its sequence shows it, the others do not
    poison(vc, codec, [(rows[4][0], 3)])
    o = m.attention_paged(q, kc, vc, codec, table, ints(lengths))
    assert not torch.isfinite(o[4]).any()
    rest = torch.arange(len(lengths), device="cuda") != 4
    assert torch.equal(o[rest], clean[rest])


def test_paged_infinite_value_of_one_dimension():
    g = gen(43)
    h, hkv, d, page = 4, 2, 64, 16
    kc, vc = pools(g, F16, 5, hkv, page, d)
    q, table, n = randn(g, h, 1, d), ints([[3, 0, 4, 1]]), ints([50])
    clean = m.attention_paged(q, kc, vc, F16, table, n).view(h, d)
    vc[0, 1, 7, 5] = -math.inf            # row 23, KV head 1 (heads 2, 3)
    o = m.attention_paged(q, kc, vc, F16, table, n).view(h, d)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[2:, 5] = True
    assert (o[hit] == -math.inf).all() and torch.equal(o[~hit], clean[~hit])


def test_paged_minus_infinite_scores():
    # a key whose score is -inf has no weight, wherever it stands
    g = gen(44)
    h, hkv, d, page, n = 4, 1, 64, 8, 40
    kc, vc = pools(g, F16, 5, hkv, page, d)
    q, table = randn(g, h, 1, d).abs() + 0.1, ints([[0, 1, 2, 3, 4]])
    for rows in ([0], [39], list(range(16)), list(range(24, 40)), [3, 17, 29]):
        k2 = kc.clone()
        for j in rows:
            k2[j // page, :, j % page] = -math.inf
        o = m.attention_paged(q, k2, vc, F16, table, ints([n])).double()
        keep = torch.tensor([j for j in range(n) if j not in rows], device="cuda")
        k, v = (x[:, 0].reshape(n, d)[keep].double() for x in (kc, vc))
        w = torch.softmax(torch.einsum("hd,jd->hj", q[:, 0].double(), k) * d ** -0.5, -1)
        want = (w @ v).reshape(1, h * d)
        assert ((o - want).abs() <= 2.0 ** -9 * (w @ v.abs()).reshape(1, h * d) + 2.0 ** -20).all(), rows


@pytest.mark.parametrize("codec", [F16, Q8])
def test_paged_matches_the_tree_over_caches(codec):
    # one sequence a page: the pool is a batch of caches, and the call the tree of one node
    g = gen(51)
    h, hkv, d, b, c = 16, 4, 128, 3, 640
    kc, vc = pools(g, codec, b, hkv, c, d)
    q, past = randn(g, h, b, d), [500, 3, 639]
    tree = m.attention_tree(q, kc, vc, codec, ints(past), ints([[-1]] * b))
    paged = m.attention_paged(q, kc, vc, codec, ints([[0], [1], [2]]), ints([x + 1 for x in past]))
    assert (tree.double() - paged.double()).abs().max() < 2e-3


@pytest.mark.parametrize("codec", [F16, Q8])
def test_paged_shared_pages_and_repeats(codec):
    # sequences with a common prefix, and a page named twice by one sequence
    g = gen(53)
    h, hkv, d, page = 8, 2, 64, 16
    kc, vc = pools(g, codec, 8, hkv, page, d)
    q = randn(g, h, 3, d)
    table, lengths = ints([[5, 6, 1, 0], [5, 6, 2, 0], [7, 7, 7, 7]]), [40, 47, 64]
    o = m.attention_paged(q, kc, vc, codec, table, ints(lengths))
    want, tol = pref.paged_attention(q, kc, vc, codec, table, lengths, d ** -0.5)
    check(o, want, tol, "shared")


@pytest.mark.parametrize("codec", [F16, Q8])
def test_paged_graph_follows_lengths_and_streams(codec):
    h, hkv, d, page, b, width = 8, 2, 128, 16, 3, 130
    g = gen(61)
    pages = 3 * width
    kc, vc = pools(g, codec, pages, hkv, page, d)
    q = randn(g, h, b, d)
    table = torch.randperm(pages, generator=g, device="cuda").view(b, width).to(torch.int32)
    lengths = ints([10, 20, 30])
    out = torch.empty(b, h * d, dtype=torch.float16, device="cuda")
    m.attention_paged(q, kc, vc, codec, table, lengths, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.attention_paged(q, kc, vc, codec, table, lengths, out=out)
    for now in ([10, 20, 30], [2000, 0, 777], [1500, 1400, 1], [2080, 2080, 2080]):
        lengths.copy_(ints(now))
        table.copy_(table.flip(0).clone())
        graph.replay()
        want, tol = pref.paged_attention(q, kc, vc, codec, table, now, d ** -0.5)
        check(out, want, tol, "replay %s" % now)
        got = []
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(4):
            for s in streams:
                got.append(m.attention_paged(q, kc, vc, codec, table, lengths, stream=s))
        torch.cuda.synchronize()
        for o in got:
            assert torch.equal(o, out)


@pytest.mark.parametrize("codec", [F16, Q8])
def test_paged_two_million_keys(codec):
    # a few pages named again and again, beside short sequences under the same wide table
    g = gen(67)
    h, hkv, d, page, width = 2, 1, 64, 8, 260000
    kc, vc = pools(g, codec, 5, hkv, page, d)
    q = randn(g, h, 3, d)
    table = torch.randint(0, 5, (3, width), generator=g, device="cuda").to(torch.int32)
    lengths = [2000003, 0, 77]
    o = m.attention_paged(q, kc, vc, codec, table, ints(lengths))
    want, tol = pref.paged_attention(q, kc, vc, codec, table, lengths, d ** -0.5)
    check(o, want, tol, "two million keys")


@pytest.mark.parametrize("codec", [F16, Q8])
def test_paged_pool_past_32_bits(codec):
    # pages on both sides of 2^32 bytes, and the pool's last one
    d, hkv, page, h = 128, 4, 64, 8
    rb = 2 * d if codec == F16 else d // 32 * 34
    pages = 2 ** 33 // (hkv * page * rb) + 40
    g = gen(71)
    edge = 2 ** 32 // (hkv * page * rb)
    use = [pages - 1, edge, 0, edge + 1, edge - 1, pages - 2]
    pool = [torch.zeros(pages, hkv, page, rb, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for c in pool:
        c[torch.tensor(use, device="cuda")] = make_cache(g, codec, len(use), hkv, page, d).view(torch.uint8)
    kc, vc = (c.view(torch.float16) if codec == F16 else c for c in pool)
    q, table = randn(g, h, 1, d), ints([use])
    o = m.attention_paged(q, kc, vc, codec, table, ints([6 * page - 3]))
    want, tol = pref.paged_attention(q, kc, vc, codec, table, [6 * page - 3], d ** -0.5)
    check(o, want, tol, "far pages")
