"""A prefix of whole pages that sequences share under page plans (GPU): how it is taken
over and given back, so that no page is free twice."""
import pytest

import swiglu_block_quantized_gb300 as m

torch = pytest.importorskip("torch")
import _paging_ref as pref   # noqa: E402
from test_attention_tree_gpu import check, gen, ints   # noqa: E402
from test_kv_ops_gpu import new_cache, randn, raw   # noqa: E402

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
def test_shared_prefix(codec):
    # Two sequences take over the whole pages of a third's prefix.  Each ends with its own pages
    # alone, the third last, and every page is free once.
    page, pages, h, hkv, d, b, width = 16, 30, 4, 2, 64, 4, 8
    g = gen(6)
    kc, vc = (new_cache(codec, pages, hkv, page, d) for _ in range(2))
    table, held, free, n_free = ints([[-1] * width] * b), ints([0] * b), ints(list(range(pages))), ints([pages])
    past = ints([0] * b)

    def step(new, room=64):
        slots, _, lengths, starts = m.page_plan(past, ints(new), table, held, free, n_free, page, room)
        m.kv_write(randn(g, hkv, room, d), randn(g, hkv, room, d), kc, vc, codec, slots)
        q = randn(g, h, b, d)
        o = m.attention_paged(q, kc, vc, codec, table, lengths)
        want, tol = pref.paged_attention(q, kc, vc, codec, table, lengths.tolist(), d ** -0.5)
        check(o, want, tol, "shared")
        past.copy_(lengths)
        named = free[:int(n_free)].tolist()
        for s in range(b):
            named += table[s, shared[s]:int(held[s])].tolist()
        assert sorted(named) == list(range(pages))

    shared = [0] * b
    step([50, 0, 0, 0])
    for s in (1, 2):                       # 3 whole pages of the first sequence's 50 rows
        table[s, :3] = table[0, :3]
        held[s], past[s], shared[s] = 3, 48, 3
    before = raw(kc)[table[0, :3].long()].clone()
    step([1, 20, 5, 7])
    step([1, 1, 17, 1])
    assert torch.equal(raw(kc)[table[0, :3].long()], before)
    assert table[1, :3].tolist() == table[2, :3].tolist() == table[0, :3].tolist()
    for s in (2, 1):
        mine = int(held[s]) - 3
        table[s, :mine] = table[s, 3:3 + mine].clone()
        table[s, mine:] = -1
        held[s], shared[s] = mine, 0
        step([1 if i != s and int(past[i]) else -1 if i == s else 0 for i in range(b)])
    step([-1, 0, 0, -1])
    assert int(n_free) == pages and sorted(free.tolist()) == list(range(pages))
