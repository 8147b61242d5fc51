"""Serving calls one right after the other, in a captured graph, over the same few
buffers and rows with other values each time: what a call reads is what the call
before it wrote, not what an earlier one left in a cache on the way (GPU)."""
import pytest

import swiglu_block_quantized_gb300 as m

torch = pytest.importorskip("torch")
import _serving_ref as ref   # noqa: E402
from test_attention_tree_gpu import gen, ints   # noqa: E402

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


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_written_and_read_in_turn(codec, d):
    steps, hkv, n, c = 40, 2, 24, 64
    g = gen(d)
    k, v = (torch.randn(steps, hkv, n, d, generator=g, device="cuda").half() for _ in range(2))
    row = d if codec == F16 else d // 32 * 34
    kc, vc = (torch.zeros(1, hkv, c, row, dtype=torch.float16 if codec == F16 else torch.uint8, device="cuda")
              for _ in range(2))
    slots = ints(list(range(n)))
    out = [(torch.empty(hkv, n, d, dtype=torch.float16, device="cuda"),
            torch.empty(hkv, n, d, dtype=torch.float16, device="cuda")) for _ in range(steps)]

    def run():
        for i in range(steps):
            m.kv_read(kc, vc, codec, slots, k_out=out[i][0], v_out=out[i][1])   # the step before's rows
            m.kv_write(k[i], v[i], kc, vc, codec, slots)
            m.kv_read(kc, vc, codec, slots, k_out=out[i][0], v_out=out[i][1])

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(5):
        for o in out:
            o[0].zero_(), o[1].zero_()
        graph.replay()
        for i in range(steps):
            for x, o in ((k[i], out[i][0]), (v[i], out[i][1])):
                want = x if codec == F16 else ref.values(ref.pack(*ref.encode(x.double())), Q8).half()
                assert torch.equal(o, want), i


@pytest.mark.parametrize("n", [1, 16])   # few rows, many rows
def test_queries_turned_into_one_buffer(n):
    # one buffer of queries, turned anew for each attention call
    steps, h, hkv, d, c = 24, 8, 2, 64, 256
    g = gen(n)
    x = torch.randn(steps, h, n, d, generator=g, device="cuda").half()
    kc, vc = (torch.randn(1, hkv, c, d, generator=g, device="cuda").half() for _ in range(2))
    freqs, _ = m.rope_freqs(d)
    pos, past, par = ints(list(range(n))), ints([100]), ints([[-1] * n])
    q = torch.empty(h, n, d, dtype=torch.float16, device="cuda")
    out = torch.empty(steps, n, h * d, dtype=torch.float16, device="cuda")
    ws = torch.empty(2 ** 24, dtype=torch.uint8, device="cuda")

    def run(i):
        m.rope(x[i], pos, freqs, out=q)
        m.attention_tree(q, kc, vc, F16, past, par, out=out[i], workspace=ws)

    want = []
    for i in range(steps):
        run(i)
        torch.cuda.synchronize()
        want.append(out[i].clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(steps):
            run(i)
    for _ in range(5):
        out.zero_()
        graph.replay()
        for i in range(steps):
            assert torch.equal(out[i], want[i]), i
