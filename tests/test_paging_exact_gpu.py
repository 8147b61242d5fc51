"""Attention over pages where errors would hide behind the length of a sequence (GPU):
tails of keys that weigh little each, sums over many keys, pieces that are lost or joined
twice, tables as wide as the call takes.  Tolerances: _paging_exact."""
import math

import pytest

import swiglu_block_quantized_gb300 as m

torch = pytest.importorskip("torch")
import _paging_exact as exact   # noqa: E402
import _serving_ref as ref   # noqa: E402
from test_attention_tree_gpu import check, gen, ints, make_cache   # noqa: E402
from test_kv_ops_gpu import randn   # noqa: E402

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


def pool(x, codec):
    """Rows of values as cache rows."""
    return x.half().contiguous() if codec == F16 else ref.pack(*ref.encode(x.double()))


def order(g, n, page):
    """Entries of ceil(n / page) pages in a random order."""
    return torch.randperm(-(-n // page), generator=g, device="cuda").to(torch.int32)[None]


def rms(x):
    return float(x.double().square().mean().sqrt())


# In the first chunk of every configuration each warp has one of these keys.
SINKS = [0, 16, 32, 48, 64, 96]


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [2000, 20001, 131001])
@pytest.mark.parametrize("bits", [20, 23.6, 26])
@pytest.mark.parametrize("whole", [False, True])
def test_tail_behind_keys_of_all_weight(codec, d, n, bits, whole):
    # Six keys have nearly all the weight and no values; the tail's, 2^-bits each and of one sign,
    # are the result.  whole: one CTA takes all keys.
    g = gen(n + d)
    page, h = 64, 3
    pages = -(-n // page)
    k = torch.zeros(pages * page, d, device="cuda")
    k[:, 5] = 0
    k[SINKS, 5] = 15.875
    v = torch.rand(pages * page, d, generator=g, device="cuda") + 0.5
    v[SINKS] = 0
    kc, vc = (pool(x.view(pages, 1, page, d), codec) for x in (k, v))
    q = torch.zeros(h, 1, d, device="cuda", dtype=torch.float16)
    q[:, 0, 5] = torch.tensor([1.0, 0.75, 1.125], device="cuda")
    scale = bits * math.log(2) / 15.875
    entries = torch.arange(pages, device="cuda", dtype=torch.int32)
    o = m.attention_paged(q, kc, vc, codec, entries[None], ints([n]), scale=scale, workspace=False if whole else None)
    want, tol = exact.sequence(q[:, 0], kc, vc, codec, entries, n, scale)
    check(o.view(h, d), want, tol, "tail of 2^-%s" % bits)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h", [1, 4, 12])
@pytest.mark.parametrize("n", [300, 20001, 131001])
@pytest.mark.parametrize("whole", [False, True])
def test_every_key_counts(codec, d, h, n, whole):
    # equal weights, and values that count the keys of a stripe
    g = gen(n)
    page = 16
    pages = -(-n // page)
    entries = order(g, n, page)
    vc = torch.empty(pages, 1, page, d, device="cuda")
    vc[entries[0].long()] = exact.striped(pages, page, d, 8).cuda()
    vc = pool(vc, codec)
    kc = torch.zeros_like(vc)
    q = randn(g, h, 1, d)
    o = m.attention_paged(q, kc, vc, codec, entries, ints([n]), workspace=False if whole else None)
    want, tol = exact.sequence(q[:, 0], kc, vc, codec, entries[0], n, d ** -0.5, rounded=False)
    check(o.view(h, d), want, tol, "stripes")


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("whole", [False, True])
def test_every_key_of_a_batch_counts(codec, d, whole):
    # the same for sequences of many lengths, whose parts the CTAs take one after the other
    g = gen(d)
    page, h, hkv = 32, 8, 2
    lengths = [0, 5000, 1, 64, 777, 0, 20000, 129, 3001, 128, 9999, 31, 8192, 65, 2, 12345]
    table = torch.full((len(lengths), -(-max(lengths) // page) + 1), -1, dtype=torch.int32, device="cuda")
    total = sum(-(-n // page) for n in lengths)
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    vc = torch.empty(total, hkv, page, d, device="cuda")
    for s, n in enumerate(lengths):
        w = -(-n // page)
        mine, ids = ids[:w], ids[w:]
        table[s, :w] = mine
        vc[mine.long()] = exact.striped(w, page, d, 8).cuda() if w else vc[:0]
    vc = pool(vc, codec)
    kc = torch.zeros_like(vc)
    q = randn(g, h, len(lengths), d)
    o = m.attention_paged(q, kc, vc, codec, table, ints(lengths), workspace=False if whole else None)
    for s, n in enumerate(lengths):
        if n == 0:
            assert (o[s] == 0).all()
            continue
        want, tol = exact.sequence(q[:, s], kc, vc, codec, table[s], n, d ** -0.5, rounded=False)
        check(o[s].view(h, d), want, tol, "sequence %d" % s)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("whole", [False, True])
def test_long_random_sequences(codec, d, whole):
    # Errors of weights rounded one by one add up as their squares do: 2^-11 / sqrt(3) of O in the
    # mean, as much again for the result's rounding.
    g = gen(d)
    n, page, h, hkv = 131001, 64, 8, 2
    entries = order(g, n, page)
    kc, vc = (make_cache(g, codec, -(-n // page), hkv, page, d) for _ in range(2))
    q = randn(g, h, 1, d)
    o = m.attention_paged(q, kc, vc, codec, entries, ints([n]), workspace=False if whole else None).view(h, d)
    want, tol = exact.sequence(q[:, 0], kc, vc, codec, entries[0], n, d ** -0.5)
    check(o, want, tol, "long")
    assert rms(o.double() - want) < 2.0 ** -11 * rms(want)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("whole", [False, True])
def test_two_million_keys_that_count(codec, whole):
    # five pages again and again: O is the mean of their values, of one sign each dim
    g = gen(3)
    d, page, n, h = 64, 8, 2000003, 2
    width = -(-n // page)
    vc = pool(torch.rand(5, 1, page, d, generator=g, device="cuda") + 0.5, codec)
    kc = torch.zeros_like(vc)
    table = torch.randint(0, 5, (1, width), generator=g, device="cuda").to(torch.int32)
    q = randn(g, h, 1, d)
    o = m.attention_paged(q, kc, vc, codec, table, ints([n]), workspace=False if whole else None).view(h, d)
    want, tol = exact.sequence(q[:, 0], kc, vc, codec, table[0], n, d ** -0.5, rounded=False)
    check(o, want, tol, "two million")


# Tables of nearly 2^31 rows: lengths near INT32_MAX, whose last chunk ends past 32 bits.
@pytest.mark.parametrize("codec,d,page", [(Q8, 64, 64), (F16, 128, 120), (F16, 64, 8), (Q8, 128, 24)])
@pytest.mark.parametrize("first", [True, False])
def test_widest_tables(codec, d, page, first):
    g = gen(page)
    width = (2 ** 31 - 1) // page
    rows = width * page
    v = torch.rand(5, page, d, generator=g, device="cuda") + 0.5
    vc = pool(v[:, None], codec)
    kc = torch.zeros_like(vc)
    table = torch.randint(0, 5, (3, width), generator=g, device="cuda").to(torch.int32)
    lengths = [rows, 5, 0] if first else [0, 5, 2 ** 31 - 1]
    q = randn(g, 1, 3, d)
    o = m.attention_paged(q, kc, vc, codec, table, ints(lengths))
    values = ref.values(vc[:, 0], codec)
    for s, n in enumerate(lengths):
        n = min(n, rows)
        if n == 0:
            assert (o[s] == 0).all()
            continue
        full, rest = divmod(n, page)
        times = torch.bincount(table[s, :full], minlength=5).double()
        want = torch.einsum("p,pd->d", times, values.sum(1))
        if rest:
            want += values[int(table[s, full]), :rest].sum(0)
        want /= n
        # equal weights and values of one sign (_paging_exact, without roundings of weights)
        tol = (2.0 ** -12 + 2.0 ** -11) * want + 2.0 ** -25
        check(o[s], want, tol, "%d rows" % n)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,hkv", [(8, 8), (48, 4)])
@pytest.mark.parametrize("whole", [False, True])
def test_long_parts_of_many_items(codec, d, h, hkv, whole):
    # so many long sequences that a CTA's parts of them take several runs, between short and empty
    # ones; the pages of a 64th of a sequence are one page, which has its own dim
    g = gen(h)
    page, b = 16, 90
    at = torch.arange(64, device="cuda")
    v = torch.nn.functional.one_hot(at, d).float()[:, None, None].expand(64, hkv, page, d)
    vc = pool(v, codec)
    kc = torch.zeros_like(vc)
    lengths = [[40000, 5, 33333, 0, 8192, 8193, 16400, 1, 24577, 300][s % 10] + 7 * (s // 10) * (s % 10 != 3)
               for s in range(b)]
    width = -(-max(lengths) // page)
    table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    for s, n in enumerate(lengths):
        w = -(-n // page)
        table[s, :w] = torch.arange(w, device="cuda") * 64 // max(w, 1)
    q = randn(g, h, b, d)
    o = m.attention_paged(q, kc, vc, codec, table, ints(lengths), workspace=False if whole else None).view(b, h, d)
    one = ref.values(vc[0, 0, 0], codec)[0]
    for s, n in enumerate(lengths):
        if n == 0:
            assert (o[s] == 0).all()
            continue
        rows = table[s].long().repeat_interleave(page)[:n]
        want = torch.zeros(d, dtype=torch.float64, device="cuda")
        want[:64] = torch.bincount(rows, minlength=64).double() * one / n
        check(o[s], want.expand(h, d), (2.0 ** -12 + 2.0 ** -11) * want.expand(h, d) + 2.0 ** -25, "sequence %d" % s)
