"""The serving operators together (GPU): a decoder layer's step with drafted
tokens, eager and captured, against 64-bit references of each operator on the
inputs it had; accepted nodes moved up in the cache; batches of more sequences
than a launch takes; workspaces of every size; streams; and every kernel in the
bounds-checked build.  Tolerances are those of test_kv_ops_gpu (rotation, rows,
norms) and _serving_ref.tree_attention."""
import numpy as np
import pytest

import swiglu_block_quantized_gb300 as m
import synth

torch = pytest.importorskip("torch")
import _serving_ref as ref   # noqa: E402
from test_attention_tree_gpu import check, gen, ints, make_cache, tree   # noqa: E402
from test_bounds_gpu import run_both   # noqa: E402
from test_kv_ops_gpu import check_rows, new_cache, raw, rope_tol   # noqa: E402

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


# ---------------------------------------------------------------- a layer

class Layer:
    """A decoder layer over a batch of caches; every buffer that a step hands
    on is kept under its name in `at`."""

    def __init__(self, codec, b, c, d, h=8, hkv=2, hidden=512, ff=768, rot=None, layout=m.ROPE_HALF):
        self.codec, self.h, self.hkv, self.d, self.hidden, self.layout = codec, h, hkv, d, hidden, layout
        self.rot = rot or d
        names = [("wq", h * d, hidden), ("wk", hkv * d, hidden), ("wv", hkv * d, hidden), ("wo", hidden, h * d),
                 ("wg", ff, hidden), ("wu", ff, hidden), ("wd", hidden, ff)]
        w = {n: torch.from_numpy(synth.weights(synth.Q8_0, r, k, seed=i, name=n)).cuda()
             for i, (n, r, k) in enumerate(names)}
        self.qkv = m.QuantQKV(w["wq"], w["wk"], w["wv"], m.Q8_0, hidden, d, h, hkv)
        self.proj = m.QuantLinear(w["wo"], m.Q8_0, hidden, h * d)
        self.mlp = m.QuantMLP(w["wg"], w["wu"], w["wd"], m.Q8_0, m.Q8_0, hidden, ff)
        g = gen(5)
        self.n1, self.n2, self.n3 = (torch.rand(hidden, generator=g, device="cuda").half() + 0.5 for _ in range(3))
        self.freqs, self.mscale = m.rope_freqs(self.rot, scaling=m.ROPE_YARN, factor=4.0, original=64.0)
        self.kc, self.vc = new_cache(codec, b, hkv, c, d), new_cache(codec, b, hkv, c, d)
        self.at = {}

    def step(self, r, pos, slots, past, parents):
        a = self.at
        a["r"], a["pos"], a["slots"], a["past"], a["parents"] = r, pos, slots, past, parents
        a["y"], _ = m.norm_residual(None, r, self.n1)
        a["q"], a["k"], a["v"] = self.qkv(a["y"])
        a["qt"] = m.kv_write(a["k"], a["v"], self.kc, self.vc, self.codec, slots, pos=pos, freqs=self.freqs,
                             layout=self.layout, mscale=self.mscale, q=a["q"])
        a["o"] = m.attention_tree(a["qt"], self.kc, self.vc, self.codec, past, parents)
        a["h"] = self.proj(a["o"])
        a["y2"], a["r2"] = m.norm_residual(a["h"], r, self.n2, w_post=self.n3)
        a["h2"] = self.mlp(a["y2"])
        _, a["r3"] = m.norm_residual(a["h2"], a["r2"], None)
        return a["r3"]

    def verify(self):
        """Each operator of the last step against its reference."""
        a = self.at
        pasts, parents, slots = a["past"].tolist(), a["parents"].tolist(), a["slots"].tolist()

        def norm(got_y, got_r, h, r, w_pre, w_post):
            want_y, want_r = ref.norm_residual(h, r, w_pre, w_post, None, 1.0, 1.0, 1e-6)
            terms = r.double().abs() + (want_r - r.double()).abs()
            if h is not None:
                assert ((got_r.double() - want_r).abs() <= 2.0 ** -17 * terms + 2.0 ** -24 * want_r.abs()).all()
            if w_pre is not None:
                rms = (want_r.square().mean(-1, keepdim=True) + 1e-6).sqrt()
                tol = 2.0 ** -17 * (terms / rms * w_pre.double().abs() + want_y.abs()) \
                    + 2.0 ** -11 * want_y.abs() + 2.0 ** -25
                assert ((got_y.double() - want_y).abs() <= tol).all()

        norm(a["y"], None, None, a["r"], self.n1, None)
        norm(a["y2"], a["r2"], a["h"], a["r"], self.n2, self.n3)
        norm(None, a["r3"], a["h2"], a["r2"], None, None)
        # the table's own frequencies in radians a position
        inv = self.freqs.cpu().double() * (2 * np.pi / 2.0 ** 64)
        want, size = ref.rotate(a["q"], a["pos"], inv, self.layout, self.mscale)
        assert ((a["qt"].double() - want).abs() <= rope_tol(want, size)).all()
        want, size = ref.rotate(a["k"], a["pos"], inv, self.layout, self.mscale)
        c = self.kc.shape[2]
        for i, s in enumerate(slots):
            if 0 <= s < self.kc.shape[0] * c:
                check_rows(self.kc[s // c, :, s % c], self.codec, want[:, i], size[:, i], 1)
                check_rows(self.vc[s // c, :, s % c], self.codec, a["v"][:, i].double(), 0 * size[:, i], 0)
        want, tol = ref.tree_attention(a["qt"], self.kc, self.vc, self.codec, pasts, parents, self.d ** -0.5)
        check(a["o"], want, tol, "tree")


def prompt(layer, lengths, seed=0):
    """Cache rows of a prompt for every sequence, in one padded write."""
    b, _, c, _ = layer.kc.shape
    most = max(lengths)
    g = gen(seed)
    r = torch.randn(b * most, layer.hidden, generator=g, device="cuda")
    slots = [s * c + i if i < lengths[s] else -1 for s in range(b) for i in range(most)]
    y, _ = m.norm_residual(None, r, layer.n1)
    _, k, v = layer.qkv(y)
    pos = ints([i for _ in range(b) for i in range(most)])
    m.kv_write(k, v, layer.kc, layer.vc, layer.codec, ints(slots), pos=pos, freqs=layer.freqs, layout=layer.layout,
               mscale=layer.mscale)
    return y


def depths(parents):
    used, seen = ref.used_and_seen(parents)
    return [len(s) for s in seen]


def drafted(layer, lengths, parents):
    """(pos, slots) of one step's nodes: unused ones are not written."""
    c = layer.kc.shape[2]
    pos, slots = [], []
    for s, p in enumerate(parents):
        for i, depth in enumerate(depths(p)):
            pos.append(lengths[s] + max(depth, 1) - 1)
            slots.append(s * c + lengths[s] + i if depth else -1)
    return ints(pos), ints(slots)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d,rot,layout", [(64, 32, m.ROPE_INTERLEAVED), (128, 128, m.ROPE_HALF)])
def test_layer_step(codec, d, rot, layout):
    b, c, n = 3, 1024, 7
    layer = Layer(codec, b, c, d, rot=rot, layout=layout)
    lengths = [900, 0, 33]
    prompt(layer, lengths)
    parents = [tree(n, 3 + s, ["random", "chain", "holes"][s]) for s in range(b)]
    pos, slots = drafted(layer, lengths, parents)
    r = torch.randn(b * n, layer.hidden, generator=gen(1), device="cuda")
    before = raw(layer.kc).clone()
    layer.step(r, pos, slots, ints(lengths), ints(parents))
    layer.verify()
    # rows that the step did not name are as they were
    touched = torch.zeros(b * c, dtype=torch.bool, device="cuda")
    touched[[s for s in slots.tolist() if s >= 0]] = True
    same = (raw(layer.kc) == before).all(-1).all(1).reshape(-1)
    assert same[~touched].all()


@pytest.mark.parametrize("codec", [F16, Q8])
def test_layer_step_captured(codec):
    # one captured step replayed over growing caches, its inputs changed in
    # place, another stream's eager step between the replays
    b, c, d, n = 2, 1280, 64, 5
    layer, other = Layer(codec, b, c, d), Layer(codec, b, c, d)
    r = torch.randn(b * n, layer.hidden, generator=gen(2), device="cuda")
    parents = [tree(n, 1, "random"), tree(n, 2, "random")]
    lengths = [40, 7]
    for x in (layer, other):
        prompt(x, lengths)
    pos, slots = drafted(layer, lengths, parents)
    past, par = ints(lengths), ints(parents)
    keep = raw(layer.kc).clone(), raw(layer.vc).clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer.step(r, pos, slots, past, par)
    torch.cuda.synchronize()
    raw(layer.kc).copy_(keep[0])
    raw(layer.vc).copy_(keep[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(r, pos, slots, past, par)
    for lengths, seed in (([40, 7], 0), ([1100, 600], 4), ([1270, 0], 6)):
        for x in (layer, other):
            prompt(x, lengths, seed)
        new = [tree(n, seed + s, "holes") for s in range(b)]
        npos, nslots = drafted(layer, lengths, new)
        pos.copy_(npos), slots.copy_(nslots), past.copy_(ints(lengths)), par.copy_(ints(new))
        r.normal_(generator=gen(seed))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            eager = other.step(r, npos, nslots, ints(lengths), ints(new))
        torch.cuda.synchronize()
        layer.verify()
        assert torch.equal(layer.at["r3"], eager)
        assert torch.equal(raw(layer.kc), raw(other.kc))


@pytest.mark.parametrize("codec", [F16, Q8])
def test_accepted_nodes_move_up(codec):
    # the accepted path's rows written again right after the context give the
    # cache that a plain run of those tokens would have left, bit for bit
    b, c, d, n = 2, 512, 128, 6
    layer = Layer(codec, b, c, d)
    lengths = [130, 20]
    prompt(layer, lengths)
    parents = [[-1, 0, 0, 2, 1, 3], [-1, -1, 1, 0, 2, 4]]
    path = [[0, 2, 3, 5], [1, 2, 4, 5]]
    pos, slots = drafted(layer, lengths, parents)
    r = torch.randn(b * n, layer.hidden, generator=gen(3), device="cuda")
    layer.step(r, pos, slots, ints(lengths), ints(parents))
    k, v = layer.at["k"], layer.at["v"]
    moved = [-1] * (b * n)
    for s in range(b):
        for i, node in enumerate(path[s]):
            moved[s * n + node] = s * c + lengths[s] + i
    m.kv_write(k, v, layer.kc, layer.vc, codec, ints(moved), pos=pos, freqs=layer.freqs, mscale=layer.mscale)
    plain = Layer(codec, b, c, d)
    prompt(plain, lengths)
    for s in range(b):
        rows = [s * n + node for node in path[s]]
        m.kv_write(k[:, rows], v[:, rows], plain.kc, plain.vc, codec,
                   ints([s * c + lengths[s] + i for i in range(4)]), pos=ints([lengths[s] + i for i in range(4)]),
                   freqs=plain.freqs, mscale=plain.mscale)
        upto = lengths[s] + 4
        for x, y in ((layer.kc, plain.kc), (layer.vc, plain.vc)):
            assert torch.equal(raw(x)[s, :, :upto], raw(y)[s, :, :upto])
    # the next token sees the same either way, whatever the rejected rows hold
    q = torch.randn(8, b, d, generator=gen(4), device="cuda").half()
    now = ints([x + 3 for x in lengths])
    one = ints([[-1]] * b)
    assert torch.equal(m.attention_tree(q, layer.kc, layer.vc, codec, now, one),
                       m.attention_tree(q, plain.kc, plain.vc, codec, now, one))


@pytest.mark.parametrize("codec", [F16, Q8])
def test_read_rows_are_those_attention_reads(codec):
    # a cache read back to fp16 and attended to as an fp16 cache
    g = gen(8)
    b, hkv, h, c, d, n = 2, 2, 8, 900, 64, 4
    kc, vc = make_cache(g, codec, b, hkv, c, d), make_cache(g, codec, b, hkv, c, d)
    q = torch.randn(h, b * n, d, generator=g, device="cuda").half()
    kr, vr = m.kv_read(kc, vc, codec, torch.arange(b * c, dtype=torch.int32, device="cuda"))
    kr, vr = (x.view(hkv, b, c, d).transpose(0, 1).contiguous() for x in (kr, vr))
    past, par = ints([800, 3]), ints([tree(n, s, "random") for s in range(b)])
    # one answer for both; the bits may differ, as a Q8_0 tile's keys are summed
    # in another order: both are held to the tolerance of the fp16 rows' answer
    want, tol = ref.tree_attention(q, kr, vr, F16, past.tolist(), par.tolist(), d ** -0.5)
    check(m.attention_tree(q, kc, vc, codec, past, par), want, tol, "cache")
    check(m.attention_tree(q, kr, vr, F16, past, par), want, tol, "rows read")


# ---------------------------------------------------------------- batches, workspaces, streams

@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("n,c", [(1, 64), (2, 1024), (40, 128)])
def test_more_sequences_than_a_launch(codec, n, c):
    b, h, hkv, d = 300, 2, 1, 64
    g = gen(n)
    kc, vc = make_cache(g, codec, b, hkv, c, d), make_cache(g, codec, b, hkv, c, d)
    q = torch.randn(h, b * n, d, generator=g, device="cuda").half()
    pasts = [(37 * s) % (c - n + 3) for s in range(b)]
    parents = [tree(n, s, "holes" if s % 3 else "random") for s in range(b)]
    o = m.attention_tree(q, kc, vc, codec, ints(pasts), ints(parents))
    want, tol = ref.tree_attention(q, kc, vc, codec, pasts, parents, d ** -0.5)
    check(o, want, tol, "300 sequences")


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("n", [3, 64])
def test_workspaces(codec, n):
    h, hkv, d, c, b = 8, 2, 128, 4096, 2
    g = gen(9)
    kc, vc = make_cache(g, codec, b, hkv, c, d), make_cache(g, codec, b, hkv, c, d)
    q = torch.randn(h, b * n, d, generator=g, device="cuda").half()
    pasts, parents = [4000, 1500], [tree(n, s, "random") for s in range(b)]
    want, tol = ref.tree_attention(q, kc, vc, codec, pasts, parents, d ** -0.5)
    size = m.load().m4q_attention_tree_workspace(codec, b, h, hkv, n, c, d)
    assert size > 0

    def call(ws):
        o = m.attention_tree(q, kc, vc, codec, ints(pasts), ints(parents), workspace=ws)
        check(o, want, tol, "workspace")
        return o

    own = call(None)
    # a workspace of the size asked for, whatever it holds, with a guard behind
    ws = torch.full((size + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(call(ws[:size]), own)
    assert (ws[size:] == 0xFF).all()
    # none, or one byte short: no split, and nothing is written to it
    short = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    assert torch.equal(call(False), call(short[:size - 1]))
    assert (short == 0xA5).all()


def test_on_another_stream():
    # work of the given stream only: inputs made there are seen
    s = torch.cuda.Stream()
    g = gen(10)
    b, h, hkv, d, c = 2, 4, 2, 64, 1024
    k, v, q = (torch.randn(x, 64, d, generator=g, device="cuda").half() for x in (hkv, hkv, h))
    big = torch.randn(4096, 4096, device="cuda")
    freqs, _ = m.rope_freqs(64)
    pos, slots = ints(list(range(64))), ints([64 * (i % 2) * 16 + i // 2 for i in range(64)])
    past, par = ints([31, 31]), ints([[-1], [-1]])
    torch.cuda.synchronize()

    def steps(stream):
        kc, vc = (torch.zeros(b, hkv, c, d, dtype=torch.float16, device="cuda") for _ in range(2))
        x = q + 0
        qt = m.kv_write(k, v, kc, vc, F16, slots, pos=pos, freqs=freqs, q=x, stream=stream)
        q1 = m.rope(x, pos, freqs, stream=stream)
        rows = m.kv_read(kc, vc, F16, slots, stream=stream)
        o = m.attention_tree(qt[:, 62:].contiguous(), kc, vc, F16, past, par, stream=stream)
        y, r = m.norm_residual(o, o, torch.ones(h * d, dtype=torch.float16, device="cuda"), stream=stream)
        return [qt, q1, *rows, o, y, r]

    want = steps(None)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(8):
            big = big @ big * 1e-4
        got = steps(s)
    s.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)


def test_refuses_another_device_and_mixed_types():
    q = torch.zeros(4, 2, 64, dtype=torch.float16, device="cuda")
    kc = torch.zeros(1, 2, 16, 64, dtype=torch.float16, device="cuda")
    for bad in (lambda: m.attention_tree(q.cpu(), kc, kc, F16, ints([1]), ints([-1, 0])),
                lambda: m.attention_tree(q, kc, kc.cpu(), F16, ints([1]), ints([-1, 0])),
                lambda: m.attention_tree(q, kc, kc, F16, torch.tensor([1], dtype=torch.int32), ints([-1, 0])),
                lambda: m.kv_write(q[:2], q[2:], kc, kc.cpu(), F16, ints([0, 1])),
                lambda: m.kv_read(kc, None, F16, torch.tensor([1], dtype=torch.int32)),
                lambda: m.norm_residual(None, q.cpu(), q[0, 0]),
                lambda: m.rope(q, ints([0, 1]).cpu(), m.rope_freqs(64)[0]),
                lambda: m.attention_tree(q.float(), kc, kc, F16, ints([1]), ints([-1, 0])),
                lambda: m.kv_write(q[:2].bfloat16(), q[2:], kc, kc, F16, ints([0, 1])),
                lambda: m.attention_tree(q, kc, kc, Q8, ints([1]), ints([-1, 0]))):
        with pytest.raises((TypeError, ValueError)):
            bad()


# ---------------------------------------------------------------- bounds-checked build

@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d,rot,layout,rows", [(64, 64, 0, 1), (64, 16, 1, 37), (128, 96, 0, 300), (128, 128, 1, 5)])
def test_bounds_rows(libs, codec, d, rot, layout, rows):
    g = gen(rows)
    hkv, h, b, c = 3, 5, 2, 200
    qkv = torch.randn(rows, h + 2 * hkv, d, generator=g, device="cuda").half().transpose(0, 1)
    q, k, v = qkv[:h], qkv[h:h + hkv], qkv[h + hkv:]
    freqs, _ = m.rope_freqs(rot)
    pos = ints([7 * i - 3 for i in range(rows)])
    slots = ints([(b * c - 1 - i) if i % 4 else -i for i in range(rows)])

    def fn():
        kc, vc = new_cache(codec, b, hkv, c, d), new_cache(codec, b, hkv, c, d)
        qt = m.kv_write(k, v, kc, vc, codec, slots, pos=pos, freqs=freqs, layout=layout, q=q)
        back = m.kv_read(kc, vc, codec, slots)
        x = m.rope(q, pos, freqs, layout=layout)
        return torch.cat([t.contiguous().view(torch.uint8).flatten() for t in (qt, kc, vc, *back, x)])

    run_both(libs, fn)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("h,hkv,d,n,c,pasts", [
    (4, 4, 64, 1, 4, [0]), (4, 4, 64, 1, 4, [3]), (8, 2, 128, 8, 132, [124, 0, 131]), (8, 2, 64, 33, 300, [300, 77]),
    (6, 2, 128, 256, 400, [144, 3]), (32, 8, 128, 1, 2052, [2051, 5, 1000]), (8, 1, 128, 64, 8000, [7900]),
    (4, 1, 64, 24, 3000, [2990, 1, 128])])
def test_bounds_tree(libs, codec, h, hkv, d, n, c, pasts):
    g = gen(c)
    b = len(pasts)
    kc, vc = make_cache(g, codec, b, hkv, c, d), make_cache(g, codec, b, hkv, c, d)
    q = torch.randn(h, b * n, d, generator=g, device="cuda").half()
    past, par = ints(pasts), ints([tree(n, s, "holes") for s in range(b)])
    run_both(libs, lambda: torch.cat([m.attention_tree(q, kc, vc, codec, past, par),
                                      m.attention_tree(q, kc, vc, codec, past, par, workspace=False)]))


@pytest.mark.parametrize("d", [8, 512, 1000, 4096, 32768])
@pytest.mark.parametrize("r32", [0, 1])
def test_bounds_norm(libs, d, r32):
    g = gen(d)
    h, gate = (torch.randn(5, d, generator=g, device="cuda").half() for _ in range(2))
    r = torch.randn(5, d, generator=g, device="cuda")
    r = r if r32 else r.half()
    w = torch.ones(d, dtype=torch.float16, device="cuda")

    def fn():
        y, r2 = m.norm_residual(h, r, w, w_post=w, gate=gate)
        return torch.cat([y.float(), r2.float()])

    run_both(libs, fn)
