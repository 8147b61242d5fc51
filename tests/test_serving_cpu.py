"""The serving operators (rotary positions, KV cache rows, attention of drafted
trees, residual norms) reject bad arguments before touching the GPU, and the
table of rotary frequencies is right (no GPU needed)."""
import ctypes
import math

import pytest

import swiglu_block_quantized_gb300 as m

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    m.build()
    return m.load()


A = ctypes.c_void_p(0x100000)   # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x100008)
BYTE = ctypes.c_void_p(0x100002)


# ---------------------------------------------------------------- frequencies

def turns(f):
    """round(f / (2 pi) 2^64): 64-bit floats are exact to 2^-52 of it."""
    return f / (2 * math.pi) * 2.0 ** 64


def freqs_of(*args, **kw):
    t, ms = m.rope_freqs(*args, device="cpu", **kw)
    assert t.dtype == torch.int64
    return [int(v) for v in t], ms


def near(got, want):
    # a power (2^-52 relative on a host libm, taken as 8 of them), a division
    # and the rounding to an integer
    assert len(got) == len(want)
    for g, w in zip(got, want):
        assert abs(g - turns(w)) <= turns(w) * 2.0 ** -48 + 1, (g, turns(w))


def test_plain_linear_ntk(lib):
    plain = [10000.0 ** (-2 * i / 64) for i in range(32)]
    got, ms = freqs_of(64)
    assert ms == 1.0
    near(got, plain)
    near(freqs_of(64, scaling=m.ROPE_LINEAR, factor=4.0)[0], [f / 4 for f in plain])
    base = 10000.0 * 4.0 ** (64 / 62)
    near(freqs_of(64, scaling=m.ROPE_NTK, factor=4.0)[0], [base ** (-2 * i / 64) for i in range(32)])


@pytest.mark.parametrize("low,high,original,factor", [(1.0, 32.0, 4096.0, 16.0), (1.0, 4.0, 8192.0, 8.0), (0.0, 2.0, 100.0, 1.0)])
def test_bands_and_yarn(lib, low, high, original, factor):
    want = []
    for i in range(64):
        f = 500000.0 ** (-2 * i / 128)
        r = original * f / (2 * math.pi)
        g = min(1.0, max(0.0, (r - low) / (high - low)))
        want.append((1 - g) * f / factor + g * f)
    kw = dict(base=500000.0, factor=factor, original=original, low=low, high=high)
    bands, one = freqs_of(128, scaling=m.ROPE_BANDS, **kw)
    near(bands, want)
    assert one == 1.0
    yarn, ms = freqs_of(128, scaling=m.ROPE_YARN, **kw)
    assert yarn == bands and abs(ms - (0.1 * math.log(factor) + 1.0)) < 1e-6
    # a scaled table never turns faster than the plain one, nor slower than 1 /
    # factor of it (but for the roundings of the mix, each 2^-53)
    plain = freqs_of(128, 500000.0)[0]
    assert all(p / factor * (1 - 2.0 ** -48) - 1 <= b <= p * (1 + 2.0 ** -48) + 1 for b, p in zip(bands, plain))


def test_frequencies_refuse(lib):
    out, ms = (ctypes.c_int64 * 64)(), ctypes.c_float()
    call = lambda rot=64, base=1e4, sc=0, f=1.0, orig=0.0, lo=1.0, hi=32.0, o=out: lib.m4q_rope_freqs(   # noqa: E731
        rot, base, sc, f, orig, lo, hi, o, ctypes.byref(ms))
    assert call() == m.OK
    inf, nan = math.inf, math.nan
    for kw in (dict(rot=0), dict(rot=7), dict(rot=-2), dict(base=1.0), dict(base=inf), dict(base=nan), dict(sc=5),
               dict(sc=-1), dict(f=0.5), dict(f=nan), dict(f=inf), dict(o=None), dict(rot=2, sc=m.ROPE_NTK),
               dict(sc=m.ROPE_BANDS), dict(sc=m.ROPE_YARN, orig=100.0, lo=2.0, hi=2.0),
               dict(sc=m.ROPE_YARN, orig=100.0, lo=-1.0), dict(sc=m.ROPE_YARN, orig=inf),
               dict(sc=m.ROPE_BANDS, orig=1.0, hi=inf), dict(sc=m.ROPE_NTK, base=1e300, f=1e300)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    assert lib.m4q_rope_freqs(64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, out, None) == m.OK
    with pytest.raises(m.M4QError):
        m.rope_freqs(3, device="cpu")


# ---------------------------------------------------------------- the C ABI's refusals

def test_rope_refuses(lib):
    def call(x=A, xh=64, xr=64, h=2, n=3, d=64, pos=A, fr=A, rot=64, lay=0, ms=1.0, y=A, yh=64, yr=64):
        return lib.m4q_rope(x, xh, xr, h, n, d, pos, fr, rot, lay, ms, y, yh, yr, None)
    for kw in (dict(x=None), dict(y=None), dict(pos=None), dict(fr=None), dict(h=0), dict(n=0), dict(h=65536),
               dict(n=2 ** 31), dict(lay=2), dict(lay=-1), dict(ms=math.nan), dict(ms=math.inf)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    for kw in (dict(d=96), dict(d=0), dict(rot=8), dict(rot=0), dict(rot=80), dict(rot=24), dict(rot=-16)):
        assert call(**kw) == m.ERR_BAD_SHAPE, kw
    for kw in (dict(x=ODD), dict(y=ODD), dict(pos=BYTE), dict(fr=ctypes.c_void_p(0x100004)), dict(xh=65), dict(xr=4),
               dict(yh=-63), dict(yr=2)):
        assert call(**kw) == m.ERR_MISALIGNED, kw


def test_kv_write_refuses(lib):
    def call(k=A, kh=64, kr=64, v=A, vh=64, vr=64, hk=2, n=3, d=64, pos=A, fr=A, rot=64, lay=0, ms=1.0, sl=A, kc=A,
             vc=A, codec=m.KV_F16, b=1, c=8, q=A, qh=64, qr=64, h=4, qo=A):
        return lib.m4q_kv_write(k, kh, kr, v, vh, vr, hk, n, d, pos, fr, rot, lay, ms, sl, kc, vc, codec, b, c, q, qh,
                                qr, h, qo, None)
    for kw in (dict(k=None), dict(v=None), dict(sl=None), dict(kc=None), dict(vc=None), dict(qo=None), dict(fr=None),
               dict(pos=None), dict(b=0), dict(c=0), dict(hk=0), dict(n=0), dict(h=0), dict(h=65532), dict(lay=3),
               dict(ms=math.inf), dict(n=2 ** 31)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    assert call(codec=m.Q4_0) == m.ERR_UNSUPPORTED_CODEC
    for kw in (dict(d=96), dict(rot=8), dict(b=2 ** 20, c=2 ** 20), dict(c=2 ** 31), dict(codec=m.Q8_0, c=9, hk=1),
               dict(codec=m.Q8_0, c=5, d=128, hk=1)):
        assert call(**kw) == m.ERR_BAD_SHAPE, kw
    for kw in (dict(k=ODD), dict(v=ODD), dict(kc=ODD), dict(vc=ODD), dict(q=ODD), dict(qo=ODD), dict(sl=BYTE),
               dict(pos=BYTE), dict(kh=3), dict(vr=12), dict(qh=1)):
        assert call(**kw) == m.ERR_MISALIGNED, kw


def test_kv_read_refuses(lib):
    def call(kc=A, vc=A, codec=m.KV_F16, b=1, hk=2, c=8, d=64, sl=A, n=3, ko=A, vo=A):
        return lib.m4q_kv_read(kc, vc, codec, b, hk, c, d, sl, n, ko, vo, None)
    for kw in (dict(kc=None), dict(ko=None), dict(vc=None), dict(vo=None), dict(sl=None), dict(n=0), dict(n=2 ** 31),
               dict(kc=None, vc=None, ko=None, vo=None), dict(c=-4)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    assert call(codec=3) == m.ERR_UNSUPPORTED_CODEC
    assert call(d=32) == m.ERR_BAD_SHAPE
    for kw in (dict(kc=ODD), dict(vo=ODD), dict(sl=BYTE)):
        assert call(**kw) == m.ERR_MISALIGNED, kw


def test_attention_tree_refuses(lib):
    def call(q=A, kc=A, vc=A, codec=m.KV_F16, b=1, h=4, hk=2, n=3, c=8, d=64, past=A, par=A, sc=0.1, o=A, ws=None):
        return lib.m4q_attention_tree(q, kc, vc, codec, b, h, hk, n, c, d, past, par, sc, o, ws, 0, None)
    for kw in (dict(q=None), dict(kc=None), dict(vc=None), dict(past=None), dict(par=None), dict(o=None), dict(n=0),
               dict(n=257), dict(h=0), dict(b=0), dict(sc=math.nan), dict(sc=-math.inf), dict(b=2 ** 22, c=1, n=256)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    assert call(codec=m.MLX4) == m.ERR_UNSUPPORTED_CODEC
    for kw in (dict(h=5), dict(d=80), dict(c=2 ** 40), dict(codec=m.Q8_0, hk=1, c=3)):
        assert call(**kw) == m.ERR_BAD_SHAPE, kw
    for kw in (dict(q=ODD), dict(kc=ODD), dict(o=ODD), dict(past=BYTE), dict(par=BYTE), dict(ws=ODD)):
        assert call(**kw) == m.ERR_MISALIGNED, kw
    assert lib.m4q_attention_tree_workspace(m.KV_F16, 1, 5, 2, 3, 8, 64) == 0
    assert lib.m4q_attention_tree_workspace(m.Q4_0, 1, 4, 2, 3, 8, 64) == 0


def test_norm_residual_refuses(lib):
    def call(h=A, r=A, t=0, wp=A, g=A, gr=0, w=A, n=3, d=64, rs=1.0, bs=1.0, eps=1e-6, ro=A, y=A):
        return lib.m4q_norm_residual(h, r, t, wp, g, gr, w, n, d, rs, bs, eps, ro, y, None)
    for kw in (dict(r=None), dict(t=2), dict(t=-1), dict(h=None), dict(h=None, wp=None), dict(w=None), dict(y=None),
               dict(w=None, y=None, ro=None), dict(n=0), dict(d=0), dict(d=32776), dict(rs=math.nan), dict(bs=math.inf),
               dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(n=2 ** 31)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    assert call(d=68) == m.ERR_BAD_SHAPE
    for kw in (dict(h=ODD), dict(r=ODD), dict(wp=ODD), dict(g=ODD), dict(w=ODD), dict(ro=ODD), dict(y=ODD)):
        assert call(**kw) == m.ERR_MISALIGNED, kw
    assert call() == m.ERR_INVALID_ARG   # y is r_out


# ---------------------------------------------------------------- the binding's refusals

class _NoLaunch:
    def m4q_attention_tree_workspace(self, *a):
        return 0

    def m4q_status_string(self, code):
        return b"status"

    def __getattr__(self, name):
        raise AssertionError("%s was called: the binding did not reject its arguments" % name)


@pytest.fixture
def cpu_binding(monkeypatch):
    """CPU tensors pass for CUDA ones, and no compute call may be made."""
    def require(t, dtype, what):
        if not isinstance(t, torch.Tensor) or t.dtype != dtype:
            raise TypeError(what)
        if not t.is_contiguous():
            raise ValueError(what)

    def head_rows(x, what):
        if x.dim() != 3 or x.stride(2) != 1:
            raise ValueError(what)
        return (*x.shape, x.stride(0), x.stride(1))
    monkeypatch.setattr(m, "_require", require)
    monkeypatch.setattr(m, "_head_rows", head_rows)
    monkeypatch.setattr(m, "_one_device", lambda *a: None)
    monkeypatch.setattr(m, "load", lambda path=None: _NoLaunch())
    return m


def f16(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def i32(n):
    return torch.zeros(n, dtype=torch.int32)


FR = torch.zeros(32, dtype=torch.int64)


def test_rope_binding(cpu_binding):
    for bad in (lambda: m.rope(f16(4, 64), i32(4), FR), lambda: m.rope(f16(2, 4, 64), i32(3), FR),
                lambda: m.rope(f16(2, 4, 64), i32(4), FR, out=f16(2, 3, 64)),
                lambda: m.rope(f16(2, 4, 64), i32(4), FR, out=f16(1, 4, 64).expand(2, 4, 64)),
                lambda: m.rope(f16(2, 4, 64), i32(4), FR, out=f16(2, 256)[:, :100].as_strided((2, 4, 64), (128, 32, 1)))):
        with pytest.raises(ValueError):
            bad()
    x = f16(2, 4, 64)
    with pytest.raises(ValueError, match="other strides"):   # x's memory, seen token by token
        m.rope(x, i32(4), FR, out=x.view(4, 2, 64).transpose(0, 1))
    assert m.rope(f16(2, 0, 64), i32(0), FR).shape == (2, 0, 64)


def test_kv_binding(cpu_binding):
    kc = f16(2, 3, 8, 64)
    k = f16(3, 5, 64)
    w = lambda **kw: m.kv_write(**{**dict(k=k, v=k, kc=kc, vc=kc, kv_codec=m.KV_F16, slots=i32(5)), **kw})   # noqa: E731
    for kw in (dict(v=f16(3, 4, 64)), dict(k=f16(2, 5, 64), v=f16(2, 5, 64)), dict(slots=i32(4)), dict(freqs=FR),
               dict(freqs=FR, pos=i32(4)), dict(q=f16(6, 5, 64)), dict(q=f16(6, 4, 64), pos=i32(5), freqs=FR),
               dict(vc=f16(2, 3, 9, 64)), dict(kc=f16(2, 3, 8, 96), vc=f16(2, 3, 8, 96)),
               dict(q=f16(6, 5, 64), pos=i32(5), freqs=FR, q_out=f16(6, 5, 32))):
        with pytest.raises(ValueError):
            w(**kw)
    with pytest.raises(TypeError):
        w(kv_codec=m.Q8_0)
    with pytest.raises(m.M4QError):
        w(kv_codec=m.Q4_0)
    with pytest.raises(ValueError):   # 66 bytes a row: not whole blocks
        m.kv_read(torch.zeros(1, 1, 4, 66, dtype=torch.uint8), None, m.Q8_0, i32(1))
    with pytest.raises(ValueError):
        m.kv_read(None, None, m.KV_F16, i32(1))
    with pytest.raises(ValueError):
        m.kv_read(kc, kc, m.KV_F16, i32(2), k_out=f16(3, 3, 64))


def test_attention_tree_binding(cpu_binding):
    kc = f16(2, 2, 8, 64)
    t = lambda **kw: m.attention_tree(**{**dict(q=f16(4, 6, 64), kc=kc, vc=kc, kv_codec=m.KV_F16, past=i32(2),   # noqa: E731
                                                parents=i32(6)), **kw})
    for kw in (dict(q=f16(4, 5, 64)), dict(q=f16(4, 6, 128)), dict(past=i32(1)), dict(parents=i32(2)), dict(vc=None),
               dict(out=f16(6, 128))):
        with pytest.raises(ValueError):
            t(**kw)
    assert t(q=f16(4, 0, 64), parents=i32(0)).shape == (0, 256)


def test_norm_binding(cpu_binding):
    h, r, w = f16(3, 64), f16(3, 64), f16(64)
    for bad in (lambda: m.norm_residual(h[:2], r, w), lambda: m.norm_residual(h, r, f16(32)),
                lambda: m.norm_residual(h, r, w, w_post=f16(63)), lambda: m.norm_residual(h, r, w, gate=f16(2, 64)),
                lambda: m.norm_residual(None, r, w, w_post=w), lambda: m.norm_residual(None, r, None),
                lambda: m.norm_residual(None, r, w, gate=w), lambda: m.norm_residual(h, r, w, out=f16(2, 64)),
                lambda: m.norm_residual(h, r, w, r_out=f16(4, 64))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: m.norm_residual(h, r.double(), w), lambda: m.norm_residual(h.float(), r, w),
                lambda: m.norm_residual(h, r.float(), w, r_out=f16(3, 64))):
        with pytest.raises(TypeError):
            bad()


def test_a_missing_tensor_type_is_refused(lib):
    with pytest.raises(TypeError):
        m.rope(f16(2, 4, 64), i32(4), FR)                 # a CPU tensor
    with pytest.raises(TypeError):
        m.norm_residual(f16(2, 64), f16(2, 64), f16(64))
