"""The paged serving loop's operators together (GPU): prompts planned, written and decoded
over pages that come and go, eager and captured; a step with drafted tokens verified and
kept; workspaces shared in turn; and every kernel in the bounds-checked build."""
import numpy as np
import pytest

import swiglu_block_quantized_gb300 as m
import synth

torch = pytest.importorskip("torch")
import _paging_ref as pref   # noqa: E402
import _serving_ref as ref   # noqa: E402
from test_attention_tree_gpu import check, gen, ints, make_cache   # noqa: E402
from test_bounds_gpu import run_both   # noqa: E402
from test_kv_ops_gpu import new_cache, randn, raw   # noqa: E402
from test_paging_gpu import plan_state, tables   # noqa: E402
from test_verify_gpu import distributions, drawn, trees   # noqa: E402

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


@pytest.fixture(scope="module")
def libs():
    m.build()
    m.build(bounds=True)
    checked = m.load(m.LIB_BOUNDS_PATH)
    assert checked.m4q_build_flags() == m.BUILD_BOUNDS
    return m.load(), checked


class Serving:
    """Sequences over a page pool beside the same ones over a cache of their own each; the
    buffers of a step keep their places, so that it can be captured."""

    def __init__(self, codec, b=5, page=16, pages=60, width=12, d=64, h=8, hkv=2, room=96):
        self.codec, self.b, self.page, self.d, self.h, self.hkv, self.room, self.width = codec, b, page, d, h, hkv, room, width
        self.kc, self.vc = (new_cache(codec, pages, hkv, page, d) for _ in range(2))
        self.own = [new_cache(codec, b, hkv, width * page, d) for _ in range(2)]
        self.table, self.held = ints([[-1] * width] * b), ints([0] * b)
        self.free, self.n_free = ints(list(range(pages))), ints([pages])
        self.past, self.new = ints([0] * b), ints([0] * b)
        self.freqs, _ = m.rope_freqs(d)
        self.axes = m.rope_axes([d // 2 - 16, 8, 8])
        self.x = [torch.empty(n, room, d, dtype=torch.float16, device="cuda") for n in (h, hkv, hkv)]
        self.host = [0] * b

    def step(self):
        """Plan, write every token of the step, attend with the last token of each sequence;
        the same into the caches of their own by slots made on the host side of the plan."""
        q, k, v = self.x
        slots, pos, lengths, starts = m.page_plan(self.past, self.new, self.table, self.held, self.free, self.n_free,
                                                  self.page, self.room)
        place = pos[None].expand(3, -1).contiguous()
        qt = m.kv_write(k, v, self.kc, self.vc, self.codec, slots, pos=place, freqs=self.freqs, axes=self.axes, q=q)
        t = torch.arange(self.room, device="cuda", dtype=torch.int32)
        seq = (t[:, None] >= starts[None, 1:]).sum(1).clamp(max=self.b - 1)
        mine = torch.where(slots >= 0, seq * (self.width * self.page) + pos, -1).to(torch.int32)
        m.kv_write(k, v, *self.own, self.codec, mine, pos=pos, freqs=self.freqs)
        last = (starts[1:].long() - 1).clamp(min=0)
        qs = qt[:, last].contiguous()
        o = m.attention_paged(qs, self.kc, self.vc, self.codec, self.table, lengths)
        tree = m.attention_tree(qs, *self.own, self.codec, (lengths - 1).clamp(min=0),
                                torch.where(lengths > 0, -1, -2).to(torch.int32))
        self.past.copy_(lengths)
        return o, tree, qs, lengths

    def check(self, out):
        o, tree, qs, lengths = out
        assert (o.double() - tree.double()).abs().max() < 3e-3
        want, tol = pref.paged_attention(qs, self.kc, self.vc, self.codec, self.table, lengths.tolist(), self.d ** -0.5)
        check(o, want, tol, "step")
        # the rows of a sequence, page by page, are those of its own cache
        for s, n in enumerate(lengths.tolist()):
            j = torch.arange(n, device="cuda")
            for pool, own in ((self.kc, self.own[0]), (self.vc, self.own[1])):
                rows = raw(pool)[self.table[s].long()[j // self.page], :, j % self.page].transpose(0, 1)
                assert torch.equal(rows, raw(own)[s, :, :n])


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("captured", [False, True])
def test_sequences_come_and_go(codec, captured):
    s, r, g = Serving(codec), np.random.RandomState(1), gen(3)
    graph = out = None
    if captured:
        s.step()
        s.past.zero_()
        s.held.zero_()
        s.table.fill_(-1)
        s.free.copy_(ints(list(range(60))))
        s.n_free.fill_(60)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = s.step()
    for step in range(25):
        # new prompts where a sequence is empty, single tokens, now and then an end
        new = [int(r.randint(1, 20)) if n == 0 else -1 if r.rand() < 0.1 or n > 150 else 1 for n in s.past.tolist()]
        s.new.copy_(ints(new))
        for x in s.x:
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        if captured:
            graph.replay()
        else:
            out = s.step()
        torch.cuda.synchronize()
        s.check(out)
        assert [bool(n > 0) for n in out[3].tolist()] == [n >= 0 for n in new]
    assert m.check_device_status() == m.OK


def test_pages_run_out():
    # tokens without a page are not written, and not seen
    s, g = Serving(F16, pages=7, b=4), gen(5)
    for x in s.x:
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    s.new.copy_(ints([40, 30, 25, 1]))     # 3 + 2 + 2 pages of 16, none for the last
    out = s.step()
    s.check(out)
    assert out[3].tolist() == [40, 30, 25, 0] and int(s.n_free) == 0
    s.new.copy_(ints([10, 5, 8, 1]))       # 2 more fit in the second's pages, 7 in the third's
    out = s.step()
    s.check(out)
    assert out[3].tolist() == [48, 32, 32, 0]


@pytest.mark.parametrize("codec", [F16, Q8])
def test_drafted_tokens_are_verified_and_kept(codec):
    # trees of drafted tokens over a batch of caches: attention, a head's probabilities,
    # verification; the kept nodes' rows move up, and the next step sees them
    b, n, h, hkv, d, c, v, hidden = 4, 7, 8, 2, 64, 256, 500, 512
    r, g = np.random.RandomState(2), gen(9)
    kc, vc = make_cache(g, codec, b, hkv, c, d), make_cache(g, codec, b, hkv, c, d)
    head = torch.from_numpy(synth.weights(synth.Q8_0, v + 4, hidden, seed=3, name="head")).cuda()   # (rows of 8)
    past = ints([100, 3, 57, 200])
    for step in range(4):
        parents = ints(trees(r, b, n, "random"))
        q, k, vv = randn(g, h, b * n, d), randn(g, hkv, b * n, d), randn(g, hkv, b * n, d)
        node = torch.arange(n, device="cuda")
        slots = (torch.arange(b, device="cuda")[:, None] * c + past[:, None] + node).to(torch.int32).view(-1)
        m.kv_write(k, vv, kc, vc, codec, slots)
        o = m.attention_tree(q, kc, vc, codec, past, parents)
        logits = m.gemm(o, head, synth.Q8_0, v + 4, hidden)[:, :v].float().view(b, n, v) * 0.02
        target = torch.softmax(logits, -1)
        draft = torch.softmax(logits + 0.7 * torch.randn(b, n, v, generator=g, device="cuda"), -1)
        tokens, u = drawn(g, draft, parents), torch.rand(b, n, generator=g, device="cuda")
        path, count, token = m.verify_tree(target, draft, tokens, parents, u)
        want = pref.verify(target, draft, tokens, parents, u)
        assert want[3] > 2.0 ** -40
        assert [path.tolist(), count.tolist(), token.tolist()] == list(want[:3])
        # kept node i of a sequence moves to row past + i; the rest of the tree is left behind
        i = torch.arange(n, device="cuda")
        kept = i < count[:, None]
        source = torch.where(kept, past[:, None] + path, -1)
        base = torch.arange(b, device="cuda")[:, None] * c
        rows = m.kv_read(kc, vc, codec, torch.where(kept, base + source, -1).to(torch.int32).view(-1))
        m.kv_write(*rows, kc, vc, codec, torch.where(kept, base + past[:, None] + i, -1).to(torch.int32).view(-1))
        now = m.kv_read(kc, vc, codec, torch.where(kept, base + past[:, None] + i, -1).to(torch.int32).view(-1))
        for a, x in zip(now, rows):
            assert (a.double() - x.double()).abs().max() <= (0 if codec == F16 else 0.06)
        past += count


def test_one_workspace_for_call_after_call():
    # calls of other shapes, one after the other on one stream, in one workspace
    ws = torch.full((2 ** 25,), 0xFF, dtype=torch.uint8, device="cuda")
    g, r = gen(11), np.random.RandomState(3)
    cases = []
    for codec, h, hkv, d, page, lengths in ((F16, 8, 2, 128, 16, [3000, 10]), (Q8, 16, 1, 64, 64, [5000]),
                                            (F16, 4, 4, 64, 8, [700, 0, 64, 900]), (Q8, 8, 8, 128, 32, [2500, 1])):
        width, pages = -(-max(lengths) // page), sum(-(-n // page) for n in lengths) + 1
        kc, vc = make_cache(g, codec, pages, hkv, page, d), make_cache(g, codec, pages, hkv, page, d)
        cases.append((randn(g, h, len(lengths), d), kc, vc, codec, ints(tables(r, lengths, page, width, pages)), ints(lengths)))
    alone = [m.attention_paged(*c) for c in cases]
    for _ in range(3):
        got = [m.attention_paged(*c, workspace=ws) for c in cases]
        torch.cuda.synchronize()
        for a, x in zip(alone, got):
            assert torch.equal(a, x)
    # and captured into one graph, replayed
    out = [torch.empty_like(a) for a in alone]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, o in zip(cases, out):
            m.attention_paged(*c, out=o, workspace=ws)
    for _ in range(3):
        for o in out:
            o.zero_()
        graph.replay()
        for a, x in zip(alone, out):
            assert torch.equal(a, x)


# ---------------------------------------------------------------- the bounds-checked build

@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("h,hkv,d,page,lengths", [
    (8, 2, 128, 16, [0, 1, 17, 300, 2000]), (8, 8, 64, 8, [7, 8, 9]), (17, 1, 128, 64, [1000, 0, 64]),
    (12, 1, 64, 256, [5000, 3]), (4, 2, 128, 24, [int(x) for x in np.random.RandomState(0).randint(0, 90, 700)])])
def test_bounds_paged(libs, codec, h, hkv, d, page, lengths):
    g, r = gen(page), np.random.RandomState(page)
    width, pages = -(-max(lengths) // page) + 1, sum(-(-n // page) for n in lengths)
    kc, vc = make_cache(g, codec, pages, hkv, page, d), make_cache(g, codec, pages, hkv, page, d)
    q, table = randn(g, h, len(lengths), d), ints(tables(r, lengths, page, width, pages))
    run_both(libs, lambda: m.attention_paged(q, kc, vc, codec, table, ints(lengths)))


def test_bounds_plan_and_verify(libs):
    r, g = np.random.RandomState(4), gen(13)
    for b, page, tokens in ((3, 4, 50), (300, 16, 5000), (1500, 8, 9000)):
        past, held, table, free, n_free = plan_state(r, b, page, 9, b * 9, 5 * page)
        new = [int(r.randint(-1, 2 * page)) for _ in range(b)]

        def plan():
            t, h, f, k = ints(table), ints(held), ints(free), ints([n_free])
            got = m.page_plan(ints(past), ints(new), t, h, f, k, page, tokens)
            return torch.cat([x.view(-1) for x in (*got, t, h, f, k)])
        run_both(libs, plan)
    for b, n, v in ((2, 6, 50000), (40, 3, 301), (1, 1, 7)):
        p, q = distributions(g, b, n, v, torch.float32)
        parents = ints(trees(r, b, n, "random"))
        tokens, u = drawn(g, q, parents), torch.rand(b, n, generator=g, device="cuda")
        run_both(libs, lambda: torch.cat([x.view(-1) for x in m.verify_tree(p, q, tokens, parents, u)]))


@pytest.mark.parametrize("codec", [F16, Q8])
def test_bounds_axes(libs, codec):
    g = gen(15)
    d, hkv, n, pages, page = 128, 3, 77, 9, 16
    k, v, q = randn(g, hkv, n, d), randn(g, hkv, n, d), randn(g, 5, n, d)
    pos = torch.randint(0, 9000, (3, n), generator=g, device="cuda").to(torch.int32)
    freqs, _ = m.rope_freqs(d)
    axes = m.rope_axes([24, 20, 20], dealt=True)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:n].to(torch.int32)

    def write():
        kc, vc = (new_cache(codec, pages, hkv, page, d) for _ in range(2))
        qo = m.kv_write(k, v, kc, vc, codec, slots, pos=pos, freqs=freqs, axes=axes, q=q)
        return torch.cat([raw(kc).view(-1), raw(vc).view(-1), qo.contiguous().view(torch.uint8).view(-1)])
    run_both(libs, write)
    run_both(libs, lambda: m.rope(q, pos, freqs, axes=axes))
