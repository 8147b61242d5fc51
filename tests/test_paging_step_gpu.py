"""Whole steps of a serving loop over pages with more than one layer, where every token of
a prompt and every drafted node attends (GPU): a row of m4q_attention_paged for each
token of a sequence, its table repeated; trees over the pages' rows read back into
caches."""
import numpy as np
import pytest

import swiglu_block_quantized_gb300 as m

torch = pytest.importorskip("torch")
import _paging_ref as pref   # noqa: E402
import _serving_ref as ref   # noqa: E402
from test_attention_tree_gpu import check, gen, ints   # noqa: E402
from test_kv_ops_gpu import new_cache, randn, raw   # noqa: E402
from test_verify_gpu import drawn, trees   # noqa: E402

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


class Model:
    """Two layers of attention over pages (random projections, a residual stream)."""

    def __init__(self, codec, b, page=16, pages=80, width=14, h=8, hkv=2, d=64, words=300):
        g = gen(11)
        self.codec, self.b, self.page, self.h, self.hkv, self.d, self.words = codec, b, page, h, hkv, d, words
        wide = h * d
        self.w = [torch.randn(wide, (h + 2 * hkv) * d, generator=g, device="cuda") * wide ** -0.5 for _ in range(2)]
        self.proj = [torch.randn(wide, wide, generator=g, device="cuda") * wide ** -0.5 for _ in range(2)]
        self.head = torch.randn(wide, words, generator=g, device="cuda") * wide ** -0.5
        self.embed = torch.randn(words, wide, generator=g, device="cuda")
        self.pools = [[new_cache(codec, pages, hkv, page, d) for _ in range(2)] for _ in range(2)]
        self.table, self.held = ints([[-1] * width] * b), ints([0] * b)
        self.free, self.n_free = ints(list(range(pages))), ints([pages])
        self.freqs, _ = m.rope_freqs(d)

    def forward(self, tokens, past, new, room):
        """tokens int64 [room], the sequences' new ones in turn -> probabilities [room, words]."""
        slots, pos, lengths, starts = m.page_plan(past, ints(new), self.table, self.held, self.free, self.n_free,
                                                  self.page, room)
        t = torch.arange(room, device="cuda")
        seq = (t[:, None] >= starts[None, 1:]).sum(1).clamp(max=self.b - 1)
        rows = self.table[seq]                                     # a row of the call for each token,
        seen = torch.where(slots >= 0, pos + 1, 0).to(torch.int32)   # which sees those up to itself
        x = self.embed[tokens]
        for layer in range(2):
            kc, vc = self.pools[layer]
            qkv = (torch.nn.functional.rms_norm(x, x.shape[1:]) @ self.w[layer]).half().view(room, -1, self.d)
            q, k, v = (y.transpose(0, 1) for y in qkv.split([self.h, self.hkv, self.hkv], 1))
            qt = m.kv_write(k, v, kc, vc, self.codec, slots, pos=pos, freqs=self.freqs, q=q)
            o = m.attention_paged(qt, kc, vc, self.codec, rows, seen)
            want, tol = pref.paged_attention(qt, kc, vc, self.codec, rows, seen.tolist(), self.d ** -0.5)
            check(o, want, tol, "layer %d" % layer)
            x = x + o.float() @ self.proj[layer]
        return torch.softmax(x @ self.head, -1), starts, lengths


@pytest.mark.parametrize("codec", [F16, Q8])
def test_prompts_and_drafted_chains(codec):
    b, n = 3, 4
    s, g, r = Model(codec, b), gen(5), np.random.RandomState(4)
    prompts = [37, 5, 60]
    room = 110
    tokens = torch.randint(0, s.words, (room,), generator=g, device="cuda")
    p, starts, past = s.forward(tokens, ints([0] * b), prompts, room)
    assert past.tolist() == prompts
    known = torch.stack([p[int(e) - 1].argmax() for e in starts[1:]])      # the last known token of each
    text = [[tokens[int(starts[i]) + j].item() for j in range(prompts[i])] for i in range(b)]
    chain = ints([[i - 1 for i in range(n)]] * b)
    for _ in range(5):
        # nodes: the last known token and n - 1 drafted ones, from distributions near the target's
        draft = torch.softmax(torch.randn(b, n, s.words, generator=g, device="cuda") * 1.5, -1)
        nodes = drawn(g, draft, chain)
        nodes[:, 0] = known
        flat = torch.zeros(room, dtype=torch.int64, device="cuda")
        flat[:b * n] = nodes.view(-1)
        p, starts, _ = s.forward(flat, past, [n] * b, room)
        assert starts.tolist() == [i * n for i in range(b + 1)]
        target, u = p[:b * n].view(b, n, s.words).contiguous(), torch.rand(b, n, generator=g, device="cuda")
        path, count, token = m.verify_tree(target, draft, nodes, chain, u)
        want = pref.verify(target, draft, nodes, chain, u)
        assert want[3] > 2.0 ** -40 and [path.tolist(), count.tolist(), token.tolist()] == list(want[:3])
        for i in range(b):
            text[i] += nodes[i, :int(count[i])].tolist()
        past = (past + count).to(torch.int32)      # rows of nodes turned down are written again
        known = token.long()
    # the pages hold the text's rows: layer 0's keys and values depend on each token alone
    for i in range(b):
        length = int(past[i])
        assert len(text[i]) == length
        x = s.embed[torch.tensor(text[i], device="cuda")]
        qkv = (torch.nn.functional.rms_norm(x, x.shape[1:]) @ s.w[0]).half().view(length, -1, s.d)
        v = qkv[:, s.h + s.hkv:].transpose(0, 1)
        j = torch.arange(length, device="cuda")
        rows = ref.values(raw(s.pools[0][1])[s.table[i].long()[j // s.page], :, j % s.page]
                          .view(s.pools[0][1].dtype).transpose(0, 1), codec)
        # (a product of another number of rows is rounded otherwise: fp16's step, and Q8_0's half step
        # of 1 / 127 of a block's largest)
        assert ((rows - v.double()).abs() <= 2.0 ** -9 * v.double().abs() + 2.0 ** -12
                + (v.double().abs().amax() / 200 if codec == Q8 else 0)).all()


@pytest.mark.parametrize("codec", [F16, Q8])
def test_trees_over_rows_read_back(codec):
    # a tree's nodes do not lie one behind the other, so its rows are read back from the pages into
    # fp16 caches, where m4q_attention_tree takes them
    b, n, page, h, hkv, d = 3, 7, 16, 8, 2, 64
    g, r = gen(8), np.random.RandomState(3)
    kc, vc = (new_cache(codec, 40, hkv, page, d) for _ in range(2))
    table, held, free, n_free = ints([[-1] * 10] * b), ints([0] * b), ints(list(range(40))), ints([40])
    pasts = [70, 0, 33]
    slots, _, _, _ = m.page_plan(ints([0] * b), ints(pasts), table, held, free, n_free, page, 128)
    m.kv_write(randn(g, hkv, 128, d), randn(g, hkv, 128, d), kc, vc, codec, slots)
    parents = ints(trees(r, b, n, "random"))
    slots, _, lengths, _ = m.page_plan(ints(pasts), ints([n] * b), table, held, free, n_free, page, b * n)
    q, k, v = randn(g, h, b * n, d), randn(g, hkv, b * n, d), randn(g, hkv, b * n, d)
    m.kv_write(k, v, kc, vc, codec, slots)
    c = 128
    j = torch.arange(c, device="cuda")
    entry = table.long()[:, (j // page).clamp(max=table.shape[1] - 1)]
    where = torch.where(j[None] < lengths[:, None], entry * page + j % page, -1).to(torch.int32).view(-1)
    own = [x.view(hkv, b, c, d).transpose(0, 1).contiguous() for x in m.kv_read(kc, vc, codec, where)]
    o = m.attention_tree(q, *own, F16, ints(pasts), parents)
    want, tol = ref.tree_attention(q, *own, F16, pasts, parents.tolist(), d ** -0.5)
    check(o, want, tol, "tree over pages")
    for s in range(b):      # and the caches hold the pages' rows
        got = pref.gather(kc, table[s], int(lengths[s]), codec)[0]
        assert torch.equal(own[0][s, :, :int(lengths[s])].double(), got)
