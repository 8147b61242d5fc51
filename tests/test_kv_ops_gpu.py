"""Rotary positions, the KV cache's rows written and read back, and the
residual norms, against 64-bit references (GPU).

Tolerances.  A rotated value is rounded once to fp16 (2^-11 of it, 2^-25 where
fp16 is subnormal); before that its angle is off by at most 2^-32 turn and
the fp32 remainder of at most 1/8 turn (together 2^-24 rad), sine, cosine and
magnitude factor by 4 x 2^-24, the two products and their sum by 3 x 2^-24, all
relative to |a| + |b|: 2^-21 (|a| + |b|) covers them.  Cache rows from
unrotated values have one right answer, bit for bit.  Norms: fp32 sums of D
squares in a tree (at most V + 10 additions deep for a thread's V vectors of
8: 42 x 2^-24), a reciprocal root (2^-22) and four products: 2^-17 relative to
the terms covers them, then one rounding."""
import math

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


def randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).half()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rope_tol(y, size):
    return 2.0 ** -11 * y.abs() + 2.0 ** -21 * size + 2.0 ** -25


def row_bytes(codec, d):
    return 2 * d if codec == F16 else d // 32 * 34


def new_cache(codec, b, hkv, c, d, fill=0x35):
    """A cache whose every byte is `fill`."""
    if codec == F16:
        return torch.full((b, hkv, c, 2 * d), fill, dtype=torch.uint8, device="cuda").view(torch.float16)
    return torch.full((b, hkv, c, row_bytes(codec, d)), fill, dtype=torch.uint8, device="cuda")


def raw(cache):
    return cache.view(torch.uint8)


# ---------------------------------------------------------------- rope

POSITIONS = [0, 1, -1, 7, 4095, 131071, 1000003, 2 ** 31 - 1, -2 ** 31, -77777]


@pytest.mark.parametrize("d,rot", [(64, 16), (64, 64), (64, 48), (128, 128), (128, 32), (128, 112)])
@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("h,rows", [(1, 1), (3, 17), (32, 5), (2, 300)])
def test_rope(d, rot, inter, h, rows):
    g = gen(d + rot + rows)
    x = randn(g, h, rows, d)
    pos = ints([POSITIONS[i % len(POSITIONS)] + (i // 10 if abs(POSITIONS[i % 10]) < 2 ** 30 else 0)
                for i in range(rows)])
    freqs, ms = m.rope_freqs(rot)
    assert ms == 1.0
    y = m.rope(x, pos, freqs, layout=inter)
    want, size = ref.rotate(x, pos, ref.inv_freqs(rot), inter)
    # positions past 2^24 make 64-bit angles themselves inexact: 2^-52 of the angle
    slack = size * (pos.double().abs() * 2.0 ** -51)[:, None]
    assert ((y.double() - want).abs() <= rope_tol(want, size) + slack).all()
    assert torch.equal(y[..., rot:], x[..., rot:])


def test_rope_strided_and_in_place():
    g = gen(3)
    h, rows, d, rot = 6, 41, 128, 64
    freqs, _ = m.rope_freqs(rot, 500000.0)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda") + 100
    by_token = randn(g, rows, h * d + 32)             # a row-major projection with wider rows
    x = by_token[:, 16:16 + h * d].unflatten(1, (h, d)).transpose(0, 1)
    y = m.rope(x, pos, freqs, mscale=1.25)
    assert y.is_contiguous()
    want, size = ref.rotate(x, pos, ref.inv_freqs(rot, 500000.0), 0, 1.25)
    assert ((y.double() - want).abs() <= rope_tol(want, size)).all()
    keep = by_token.clone()
    out = m.rope(x, pos, freqs, mscale=1.25, out=x)   # in place, strided
    assert out is x and torch.equal(x, y)
    assert torch.equal(by_token[:, :16], keep[:, :16]) and torch.equal(by_token[:, 16 + h * d:], keep[:, 16 + h * d:])
    assert m.rope(x[:, :0], pos[:0], freqs).shape == (h, 0, d)


@pytest.mark.parametrize("inter", [0, 1])
def test_rope_many_heads_a_thread(inter):
    # enough tokens that a thread walks several heads with one set of sines
    g = gen(5)
    h, rows, d = 33, 4100, 64
    x = randn(g, h, rows, d)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    freqs, _ = m.rope_freqs(d)
    want, size = ref.rotate(x, pos, ref.inv_freqs(d), inter)
    assert ((m.rope(x, pos, freqs, layout=inter).double() - want).abs() <= rope_tol(want, size)).all()


def test_rope_undone_by_the_negative_position():
    # a position and its negative undo each other up to two roundings
    g = gen(6)
    x = randn(g, 4, 50, 128)
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 7919
    freqs, _ = m.rope_freqs(128)
    back = m.rope(m.rope(x, pos, freqs), -pos, freqs)
    _, size = ref.rotate(x, pos, ref.inv_freqs(128), 0)
    assert ((back.double() - x.double()).abs() <= 2.0 ** -10 * size + 2.0 ** -11 * x.double().abs()).all()


# ---------------------------------------------------------------- cache write and read

def check_rows(cache, codec, want, size, turned):
    """Cache rows against 64-bit values: exact where nothing was turned."""
    got = ref.values(cache, codec)
    if codec == F16:
        if not turned:
            assert torch.equal(got, want)
        assert ((got - want).abs() <= rope_tol(want, size)).all()
        return
    d, q = ref.encode(want)
    if not turned:
        assert torch.equal(cache, ref.pack(d, q))
        return
    # the scale is that of the 64-bit rotation, or the next fp16 either way;
    # a value is off by half a step, its fp32 error and one fp16 rounding
    b = cache.unflatten(-1, (-1, 34))
    gd = b[..., :2].contiguous().view(torch.int16)[..., 0].int()
    assert ((gd - d.view(torch.int16).int()).abs() <= 1).all()
    step = (d.double() * (1 + 2.0 ** -10) + 2.0 ** -24).repeat_interleave(32, -1)
    assert ((got - want).abs() <= step / 2 + 2.0 ** -20 * size + 2.0 ** -11 * want.abs() + 2.0 ** -25).all()


@pytest.mark.parametrize("codec", [F16, Q8])
@pytest.mark.parametrize("d,rot,inter", [(64, 0, 0), (64, 16, 0), (64, 64, 0), (64, 48, 1), (128, 128, 0),
                                         (128, 48, 0), (128, 64, 1), (128, 0, 0)])
@pytest.mark.parametrize("b,hkv,c,rows", [(1, 1, 4, 1), (1, 8, 40, 33), (3, 2, 24, 50), (2, 5, 8, 7)])
def test_kv_write(codec, d, rot, inter, b, hkv, c, rows):
    g = gen(rows + d + rot)
    h = 2 * hkv
    qkv = randn(g, h + 2 * hkv, rows, d)
    q, k, v = qkv[:h], qkv[h:h + hkv], qkv[h + hkv:]
    # distinct rows in any order, with padding in between
    order = torch.randperm(b * c, generator=torch.Generator().manual_seed(rows)).tolist()
    slots = [order.pop() if order and i % 5 != 3 else [-1, b * c, 2 ** 31 - 1, -2 ** 31][i % 4] for i in range(rows)]
    pos = ints([3 * i + 11 for i in range(rows)])
    kc, vc = new_cache(codec, b, hkv, c, d), new_cache(codec, b, hkv, c, d)
    if rot:
        freqs, _ = m.rope_freqs(rot)
        qo = m.kv_write(k, v, kc, vc, codec, ints(slots), pos=pos, freqs=freqs, layout=inter, q=q)
        assert torch.equal(qo, m.rope(q, pos, freqs, layout=inter))
        want, size = ref.rotate(k, pos, ref.inv_freqs(rot), inter)
    else:
        assert m.kv_write(k, v, kc, vc, codec, ints(slots)) is None
        want, size = k.double(), torch.zeros_like(k, dtype=torch.float64)
    named = torch.zeros(b * c, dtype=torch.bool, device="cuda")
    for i, s in enumerate(slots):
        if 0 <= s < b * c:
            named[s] = True
            check_rows(kc[s // c, :, s % c], codec, want[:, i], size[:, i], rot)
            check_rows(vc[s // c, :, s % c], codec, v[:, i].double(), size[:, i] * 0, 0)
    fresh = raw(new_cache(codec, b, hkv, c, d))
    for cache in (kc, vc):   # rows that no slot names are as they were
        same = (raw(cache) == fresh).all(-1).all(1).reshape(-1)
        assert same[~named].all()
    # read back: every written row, one twice, and slots outside
    at = [s for s in slots if 0 <= s < b * c]
    at = ints(at + at[:1] + [-1, b * c])
    kr, vr = m.kv_read(kc, vc, codec, at)
    for cache, got in ((kc, kr), (vc, vr)):
        rows_at = cache.transpose(0, 1).flatten(1, 2)[:, at[:-2].long()]
        assert torch.equal(got[:, :-2].double(), ref.values(rows_at, codec))
        assert (got[:, -2:] == 0).all()
    only_v = m.kv_read(None, vc, codec, at)
    assert only_v[0] is None and torch.equal(only_v[1], vr)


def test_q8_0_block_edges():
    # blocks of zeros, of the smallest subnormals, of values whose scale is
    # subnormal, of the largest fp16, of exact ties (codes to even), and one
    # with an infinity and one with a NaN (decode to NaN, others unharmed)
    d, rows = 64, 8
    x = torch.zeros(1, rows, d, device="cuda", dtype=torch.float64)
    x[0, 1, :32] = 2.0 ** -24
    x[0, 1, 32:] = torch.linspace(-1, 1, 32, dtype=torch.float64, device="cuda") * 180 * 2.0 ** -24
    x[0, 2] = torch.linspace(-65504, 65504, d, dtype=torch.float64, device="cuda")
    step = 2.0 ** -6
    x[0, 3, :32] = (torch.arange(32, device="cuda") - 15.5) * step          # ties of d = 2^-6
    x[0, 3, 0] = 127 * step
    x[0, 3, 32:] = (torch.arange(32, device="cuda") - 16.5) * 3 * step      # ties of d = 3 x 2^-6
    x[0, 3, 40] = -127 * 3 * step
    x[0, 4] = 1.0
    x[0, 5] = -0.0
    x[0, 6, 32:] = 5 * 2.0 ** -20
    x = x.half()
    x[0, 6, 3], x[0, 7, 40] = math.inf, math.nan
    kc, vc = new_cache(Q8, 1, 1, rows, d), new_cache(Q8, 1, 1, rows, d)
    m.kv_write(x, x, kc, vc, Q8, torch.arange(rows, dtype=torch.int32, device="cuda"))
    assert torch.equal(kc, vc)
    dd, qq = ref.encode(x[:, :6].double())
    assert torch.equal(kc[0, :, :6], ref.pack(dd, qq))
    assert qq.abs().max() == 127
    got, _ = m.kv_read(kc, vc, Q8, torch.arange(rows, dtype=torch.int32, device="cuda"))
    assert got[0, 6, :32].isnan().all() and not got[0, 6, 32:].isnan().any()
    assert got[0, 7, 32:].isnan().all() and (got[0, 7, :32] == 0).all()


@pytest.mark.parametrize("codec", [F16, Q8])
def test_offsets_past_32_bits(codec):
    # caches whose last rows start past 2^32 bytes
    d, hkv, b = 128, 4, 2
    c = 2 ** 32 // (b * hkv * row_bytes(codec, d)) // 4 * 4 + 400
    kc, vc = new_cache(codec, b, hkv, c, d, 0), new_cache(codec, b, hkv, c, d, 0)
    assert kc.numel() * kc.element_size() > 2 ** 32
    g = gen(9)
    k, v = randn(g, hkv, 3, d), randn(g, hkv, 3, d)
    slots = ints([b * c - 1, 0, c - 2])
    m.kv_write(k, v, kc, vc, codec, slots)
    kr, vr = m.kv_read(kc, vc, codec, slots)
    if codec == F16:
        assert torch.equal(kr, k) and torch.equal(vr, v)
    else:
        dd, qq = ref.encode(k.double())
        assert torch.equal(kr.double(), ref.values(ref.pack(dd, qq), Q8))
    assert raw(kc[b - 1, hkv - 1, c - 2]).sum() == 0
    assert int((raw(kc[b - 1, :, c - 1]) != 0).any(-1).sum()) == hkv


# ---------------------------------------------------------------- norms

def check_norm(g, rows, d, r32, post, gate, y, rs=1.0, bs=1.0, scale=1.0):
    h = randn(g, rows, d, scale=scale)
    r = randn(g, rows, d, scale=2.0)
    r = r.float() * 1.0009765 if r32 else r
    w1 = randn(g, d) if post else None
    w2 = randn(g, d) if y else None
    gt = {0: None, 1: randn(g, d), 2: randn(g, rows, d)}[gate]
    got_y, got_r = m.norm_residual(h, r, w2, w_post=w1, gate=gt, res_scale=rs, branch_scale=bs, eps=1e-5)
    want_y, want_r = ref.norm_residual(h, r, w2, w1, gt, rs, bs, 1e-5)
    assert got_r.dtype == r.dtype and got_r.shape == r.shape
    # r': relative to the terms it is the sum of; y: that, carried on
    terms = rs * r.double().abs() + (want_r - rs * r.double()).abs()
    half = 2.0 ** -24 if r32 else 2.0 ** -11
    assert ((got_r.double() - want_r).abs() <= 2.0 ** -17 * terms + half * want_r.abs() + 2.0 ** -25).all()
    if y:
        rms = (want_r.square().mean(-1, keepdim=True) + 1e-5).sqrt()
        tol = 2.0 ** -17 * (terms / rms * w2.double().abs() + want_y.abs()) + 2.0 ** -11 * want_y.abs() + 2.0 ** -25
        assert ((got_y.double() - want_y).abs() <= tol).all()
    else:
        assert got_y is None


@pytest.mark.parametrize("d", [8, 64, 248, 256, 264, 520, 1024, 1032, 2048, 2056, 4096, 5000, 8192, 8200, 32768])
@pytest.mark.parametrize("rows", [1, 9])
def test_norm_widths(d, rows):
    for r32 in (0, 1):
        check_norm(gen(d + rows), rows, d, r32, 1, 2, 1, 0.9, 0.3)


@pytest.mark.parametrize("r32", [0, 1])
@pytest.mark.parametrize("post", [0, 1])
@pytest.mark.parametrize("gate", [0, 1, 2])
@pytest.mark.parametrize("y", [0, 1])
def test_norm_options(r32, post, gate, y):
    check_norm(gen(17), 37, 640, r32, post, gate, y, 1.0, -0.5)


def test_norm_alone_in_place_and_special_rows():
    g = gen(21)
    r, w, h = randn(g, 6, 2048), randn(g, 2048), randn(g, 6, 2048, scale=100.0)
    h[1] = 0                       # a row of zeros: eps alone
    h[2] = 60000                   # squares far beyond fp16
    r[3, 7] = math.inf
    h[4, 9] = math.nan
    y, same = m.norm_residual(None, r, w)
    assert same is r
    want, _ = ref.norm_residual(None, r, w, None, None, 1, 1, 1e-6)
    ok = [0, 1, 2, 4, 5]
    assert ((y[ok].double() - want[ok]).abs() <= 2.0 ** -10 * want[ok].abs() + 2.0 ** -20).all()
    y1, r1 = m.norm_residual(h, r, w, w_post=w)
    r2, h2 = r.clone(), h.clone()
    y2, r3 = m.norm_residual(h2, r2, w, w_post=w, r_out=r2, out=h2)
    assert r3 is r2 and y2 is h2
    for a, b in ((y1, y2), (r1, r2)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert torch.isfinite(r1[[0, 1, 2, 5]]).all() and torch.equal(r1[1], r[1])
    assert r1[4].isnan().all() and not torch.isfinite(y1[3]).all()
    assert m.norm_residual(h[:0], r[:0], w)[0].shape == (0, 2048)
