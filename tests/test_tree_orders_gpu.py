"""Tree attention when its copies land late (GPU): calls whose caches are read from
memory for the first time, or again after the L2 cache was filled with something
else, give the reference's values and the same bits each time.  What they would
miss is walked on the CPU by test_tree_barriers_cpu."""
import pytest

import swiglu_block_quantized_gb300 as m

torch = pytest.importorskip("torch")
import _serving_ref as ref   # noqa: E402
from test_attention_tree_gpu import check, gen, ints, make_cache, tree   # noqa: E402

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


def repeated(codec, h, hkv, d, c, pasts, n, seed):
    b = len(pasts)
    g = gen(seed)
    q = torch.randn(h, b * n, d, generator=g, device="cuda").half()
    kc, vc = make_cache(g, codec, b, hkv, c, d), make_cache(g, codec, b, hkv, c, d)
    parents = [tree(n, seed + s, "holes" if s % 2 else "random") for s in range(b)]
    past, par = ints(pasts), ints(parents)
    want, tol = ref.tree_attention(q, kc, vc, codec, pasts, parents, d ** -0.5)
    other = torch.empty(2 ** 26, device="cuda")   # 256 MB, more than L2
    first = None
    for i in range(8):
        other.fill_(i)
        o = m.attention_tree(q, kc, vc, codec, past, par)
        if first is None:
            first = o
            check(o, want, tol, "h=%d/%d d=%d n=%d" % (h, hkv, d, n))
        else:
            assert torch.equal(o, first), "call %d" % i


# 17 to 32 rows a KV head over a Q8_0 cache: two blocks of 16 rows, one decode group a
# kind; long runs, many runs of few tiles, and runs of one
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,hkv,n,c,pasts", [
    (17, 1, 1, 20000, [19000]), (24, 1, 1, 4096, [4095, 17, 2600]), (32, 8, 8, 2048, [2000, 1, 130, 900, 513]),
    (12, 4, 7, 640, [600] * 60), (8, 8, 31, 128, [90] * 40)])
def test_few_rows_in_two_blocks(d, h, hkv, n, c, pasts):
    repeated(Q8, h, hkv, d, c, pasts, n, 7)


# more than 32 rows over fp16 caches at D = 128: three K stages for two issuers
@pytest.mark.parametrize("h,hkv,n,c,pasts", [
    (32, 8, 24, 9000, [8900, 4000]), (8, 1, 64, 20000, [19900]), (16, 4, 16, 768, [700, 3, 350, 128] * 15),
    (4, 1, 256, 520, [200])])
def test_many_rows_fp16(h, hkv, n, c, pasts):
    repeated(F16, h, hkv, 128, c, pasts, n, 11)


# D = 64: three score buffers, the halves of a row a tile apart
@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("h,hkv,n,c,pasts", [
    (32, 8, 24, 9000, [8900, 4000, 1]), (8, 1, 64, 20000, [19900]), (16, 4, 16, 768, [700, 3, 350, 128] * 15)])
def test_many_rows_of_64(codec, h, hkv, n, c, pasts):
    repeated(codec, h, hkv, 64, c, pasts, n, 13)
