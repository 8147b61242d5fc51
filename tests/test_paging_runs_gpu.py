"""Attention over pages where parts take several runs (csrc/attention_paged.cu): the
bounds-checked build, a captured graph, two streams at once (GPU)."""
import numpy as np
import pytest

import swiglu_block_quantized_gb300 as m

torch = pytest.importorskip("torch")
from test_attention_tree_gpu import gen, ints, make_cache   # noqa: E402
from test_bounds_gpu import run_both   # noqa: E402
from test_kv_ops_gpu import randn   # noqa: E402

pytestmark = pytest.mark.gpu

F16, Q8 = m.KV_F16, m.Q8_0
LENGTHS = [8192, 0, 8193, 70001, 5, 16385, 30000, 64]


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


def inputs(codec, h, hkv, d, page, seed=0):
    g = gen(seed + d)
    pages = 200
    kc, vc = make_cache(g, codec, pages, hkv, page, d), make_cache(g, codec, pages, hkv, page, d)
    width = -(-max(LENGTHS) // page)
    table = torch.randint(0, pages, (len(LENGTHS), width), generator=g, device="cuda").to(torch.int32)
    table[3, 100:110] = -1          # entries that are no pages, within a run
    return randn(g, h, len(LENGTHS), d), kc, vc, codec, table, ints(LENGTHS)


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("h,hkv,d,page", [(8, 2, 128, 16), (12, 1, 64, 40), (17, 1, 128, 64), (4, 4, 64, 8)])
@pytest.mark.parametrize("whole", [False, True])
def test_bounds(libs, codec, h, hkv, d, page, whole):
    args = inputs(codec, h, hkv, d, page)
    run_both(libs, lambda: m.attention_paged(*args, workspace=False if whole else None))


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("whole", [False, True])
def test_captured_and_on_two_streams(codec, whole):
    calls = [inputs(codec, 8, 2, 64, 16, seed) for seed in (1, 2)]
    kw = {"workspace": False} if whole else {}
    alone = [m.attention_paged(*c, **kw) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        got = []
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(m.attention_paged(*c, **kw))
        torch.cuda.synchronize()
        for a, o in zip(alone, got):
            assert torch.equal(a, o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [m.attention_paged(*c, **kw) for c in calls]
    lengths = calls[0][-1]
    for n in (LENGTHS, [int(x) for x in np.random.RandomState(3).randint(0, 70001, len(LENGTHS))], LENGTHS):
        lengths.copy_(ints(n))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], m.attention_paged(*calls[0], **kw)) and torch.equal(out[1], alone[1])
