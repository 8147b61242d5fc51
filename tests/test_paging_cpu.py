"""The operators of the paged serving loop (positions of several axes, page plans,
attention over pages, verification of drafted trees) refuse bad arguments before
touching the GPU, and the table of axes is right (no GPU needed)."""
import ctypes
import math

import pytest

import swiglu_block_quantized_gb300 as m

torch = pytest.importorskip("torch")
from test_serving_cpu import A, BYTE, FR, ODD, cpu_binding, f16, i32   # noqa: E402,F401


@pytest.fixture(scope="module")
def lib():
    m.build()
    return m.load()


def test_axes_table():
    assert m.rope_axes([2, 3], device="cpu").tolist() == [0, 0, 1, 1, 1]
    assert m.rope_axes([4, 0, 1], device="cpu").tolist() == [0, 0, 0, 0, 2]
    # in turn, the first axis takes what the others leave
    assert m.rope_axes([4, 2, 2], dealt=True, device="cpu").tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    assert m.rope_axes([5, 2, 1], dealt=True, device="cpu").tolist() == [0, 1, 2, 0, 1, 0, 0, 0]
    assert m.rope_axes([3], dealt=True, device="cpu").tolist() == [0, 0, 0]
    for bad in ([], [0, 0], [2, -1], [1] * 9):
        with pytest.raises(ValueError):
            m.rope_axes(bad, device="cpu")
    with pytest.raises(ValueError, match="dealt"):
        m.rope_axes([1, 4], dealt=True, device="cpu")


# ---------------------------------------------------------------- the C ABI

def test_rope_axes_refuses(lib):
    def call(x=A, xh=64, xr=64, h=2, n=3, d=64, pos=A, na=3, fr=A, ax=A, rot=64, lay=0, ms=1.0, y=A, yh=64, yr=64):
        return lib.m4q_rope_axes(x, xh, xr, h, n, d, pos, na, fr, ax, rot, lay, ms, y, yh, yr, None)
    for kw in (dict(x=None), dict(y=None), dict(pos=None), dict(fr=None), dict(ax=None), dict(na=0), dict(na=9),
               dict(na=-1), dict(h=0), dict(n=0), dict(n=2 ** 31), dict(lay=2), dict(ms=math.nan)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    for kw in (dict(d=96), dict(rot=8), dict(rot=80)):
        assert call(**kw) == m.ERR_BAD_SHAPE, kw
    for kw in (dict(x=ODD), dict(pos=BYTE), dict(ax=BYTE), dict(fr=ctypes.c_void_p(0x100004)), dict(xh=65)):
        assert call(**kw) == m.ERR_MISALIGNED, kw


def test_kv_write_axes_refuses(lib):
    def call(k=A, v=A, hk=2, n=3, d=64, pos=A, na=2, fr=A, ax=A, rot=64, lay=0, ms=1.0, sl=A, kc=A, vc=A,
             codec=m.KV_F16, b=1, c=8, q=A, h=4, qo=A):
        return lib.m4q_kv_write_axes(k, 64, 64, v, 64, 64, hk, n, d, pos, na, fr, ax, rot, lay, ms, sl, kc, vc, codec,
                                     b, c, q, 64, 64, h, qo, None)
    for kw in (dict(k=None), dict(sl=None), dict(fr=None), dict(ax=None), dict(fr=None, q=None), dict(na=0), dict(na=9),
               dict(pos=None), dict(b=0), dict(n=0), dict(lay=3)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    assert call(codec=m.Q4_0) == m.ERR_UNSUPPORTED_CODEC
    assert call(rot=8) == m.ERR_BAD_SHAPE
    for kw in (dict(k=ODD), dict(ax=BYTE), dict(pos=BYTE)):
        assert call(**kw) == m.ERR_MISALIGNED, kw


def test_page_plan_refuses(lib):
    names = ("past", "new", "table", "held", "free", "n_free", "slots", "pos", "lengths", "starts")

    def call(b=2, page=16, w=4, p=9, t=5, **kw):
        a = {n: A for n in names}
        a.update(kw)
        return lib.m4q_page_plan(a["past"], a["new"], b, page, a["table"], w, a["held"], a["free"], p, a["n_free"], t,
                                 a["slots"], a["pos"], a["lengths"], a["starts"], None)
    for n in names:
        assert call(**{n: None}) == m.ERR_INVALID_ARG, n
        assert call(**{n: BYTE}) == m.ERR_MISALIGNED, n
    for kw in (dict(b=0), dict(b=4097), dict(page=0), dict(page=-8), dict(w=0), dict(p=0), dict(t=0), dict(t=2 ** 31 - 1)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    for kw in (dict(page=2 ** 31), dict(p=2 ** 27), dict(w=2 ** 27), dict(page=2 ** 30, w=2), dict(p=2 ** 62)):
        assert call(**kw) == m.ERR_BAD_SHAPE, kw


def test_attention_paged_refuses(lib):
    def call(q=A, kc=A, vc=A, codec=m.KV_F16, b=2, h=4, hk=2, p=9, page=16, d=64, tab=A, w=3, le=A, sc=0.1, o=A, ws=None):
        return lib.m4q_attention_paged(q, kc, vc, codec, b, h, hk, p, page, d, tab, w, le, sc, o, ws, 0, None)
    for kw in (dict(q=None), dict(kc=None), dict(vc=None), dict(tab=None), dict(le=None), dict(o=None), dict(b=0),
               dict(h=0), dict(w=0), dict(p=0), dict(page=0), dict(hk=0), dict(sc=math.nan), dict(sc=math.inf),
               dict(sc=3e38), dict(sc=-2.4e38), dict(b=65536), dict(h=65536)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    assert call(codec=m.MLX4) == m.ERR_UNSUPPORTED_CODEC
    for kw in (dict(h=5), dict(d=80), dict(page=12), dict(page=4), dict(page=2 ** 40), dict(p=2 ** 40), dict(w=2 ** 28),
               dict(w=2 ** 60)):
        assert call(**kw) == m.ERR_BAD_SHAPE, kw
    for kw in (dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(o=ODD), dict(tab=BYTE), dict(le=BYTE), dict(ws=ODD)):
        assert call(**kw) == m.ERR_MISALIGNED, kw
    ws = lib.m4q_attention_paged_workspace
    assert ws(m.KV_F16, 2, 5, 2, 9, 16, 3, 64) == 0 and ws(m.Q4_0, 2, 4, 2, 9, 16, 3, 64) == 0
    assert ws(m.KV_F16, 2, 4, 2, 9, 12, 3, 64) == 0


def test_verify_tree_refuses(lib):
    def call(t=A, d=A, ty=0, b=2, n=3, v=100, tok=A, par=A, u=A, path=A, cnt=A, nxt=A):
        return lib.m4q_verify_tree(t, 300, 100, d, 300, 100, ty, b, n, v, tok, par, u, path, cnt, nxt, None)
    for kw in (dict(t=None), dict(d=None), dict(tok=None), dict(par=None), dict(u=None), dict(path=None),
               dict(cnt=None), dict(nxt=None), dict(ty=2), dict(ty=-1), dict(b=0), dict(b=2 ** 31), dict(n=0), dict(n=257),
               dict(v=0), dict(v=2 ** 24 + 1)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    for kw in (dict(t=BYTE), dict(d=BYTE), dict(t=ctypes.c_void_p(0x100001), ty=1), dict(tok=BYTE), dict(par=BYTE),
               dict(u=BYTE), dict(path=BYTE), dict(cnt=BYTE), dict(nxt=BYTE)):
        assert call(**kw) == m.ERR_MISALIGNED, kw


# ---------------------------------------------------------------- the binding

def test_rope_axes_binding(cpu_binding):
    x, pos, ax = f16(2, 4, 64), i32(12).view(3, 4), i32(32)
    with pytest.raises(AssertionError, match="m4q_rope_axes was called"):
        m.rope(x, pos, FR, axes=ax)
    for kw in (dict(pos=i32(12)), dict(pos=i32(12).view(4, 3)), dict(axes=i32(31)), dict(pos=i32(4))):
        with pytest.raises(ValueError):
            m.rope(x, **{**dict(pos=pos, freqs=FR, axes=ax), **kw})
    with pytest.raises(ValueError):   # positions of three axes without a table of axes
        m.rope(x, pos, FR)
    kc, k = f16(2, 3, 8, 64), f16(3, 4, 64)
    w = lambda **kw: m.kv_write(**{**dict(k=k, v=k, kc=kc, vc=kc, kv_codec=m.KV_F16, slots=i32(4), pos=pos, freqs=FR,   # noqa: E731
                                          axes=ax), **kw})
    with pytest.raises(AssertionError, match="m4q_kv_write_axes was called"):
        w()
    for kw in (dict(pos=i32(4)), dict(axes=i32(16)), dict(pos=None), dict(freqs=None, pos=None)):
        with pytest.raises(ValueError):
            w(**kw)


def test_page_plan_binding(cpu_binding):
    def call(**kw):
        return m.page_plan(**{**dict(past=i32(3), new=i32(3), table=i32(12).view(3, 4), held=i32(3), free=i32(20),
                                     n_free=i32(1), page=16, tokens=7), **kw})
    with pytest.raises(AssertionError, match="m4q_page_plan was called"):
        call()
    with pytest.raises(AssertionError, match="m4q_page_plan was called"):
        call(out=(i32(7), i32(7), i32(3), i32(4)))
    for kw in (dict(past=i32(2)), dict(new=i32(4)), dict(held=i32(0)), dict(n_free=i32(2)), dict(table=i32(12)),
               dict(tokens=0), dict(tokens=-3), dict(out=(i32(7), i32(7), i32(3), i32(3))), dict(out=(i32(7), i32(7), i32(3))), dict(table=i32(24).view(3, 8)[:, :4])):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(past=torch.zeros(3)), dict(free=torch.zeros(20, dtype=torch.int64))):
        with pytest.raises(TypeError):
            call(**kw)


def test_attention_paged_binding(cpu_binding):
    kc = f16(9, 2, 16, 64)
    call = lambda **kw: m.attention_paged(**{**dict(q=f16(4, 3, 64), kc=kc, vc=kc, kv_codec=m.KV_F16,   # noqa: E731
                                                    table=i32(6).view(3, 2), lengths=i32(3), workspace=False), **kw})
    with pytest.raises(AssertionError, match="m4q_attention_paged was called"):
        call()
    for kw in (dict(q=f16(4, 2, 64)), dict(q=f16(4, 3, 128)), dict(table=i32(6)), dict(table=i32(6).view(2, 3)),
               dict(lengths=i32(2)), dict(out=f16(3, 128)), dict(vc=None), dict(kc=kc[0], vc=kc[0]),
               dict(vc=f16(8, 2, 16, 64))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(TypeError):
        call(kv_codec=m.Q8_0)
    assert call(q=f16(4, 0, 64), table=i32(0).view(0, 2), lengths=i32(0)).shape == (0, 256)


def test_verify_tree_binding(cpu_binding, monkeypatch):
    def rows(x, what):
        return x.stride(0), x.stride(1)
    real = m._prob_rows
    monkeypatch.setattr(m, "_prob_rows", rows)
    p, n = torch.zeros(2, 3, 50), i32(6).view(2, 3)
    call = lambda **kw: m.verify_tree(**{**dict(target=p, draft=p, tokens=n, parents=n, u=torch.zeros(2, 3)), **kw})   # noqa: E731
    with pytest.raises(AssertionError, match="m4q_verify_tree was called"):
        call()
    for kw in (dict(draft=None), dict(draft=torch.zeros(2, 3, 49)), dict(tokens=i32(5)), dict(parents=i32(6).view(3, 2)),
               dict(u=torch.zeros(3, 2)), dict(out=(n, i32(2), i32(3))), dict(out=(n, i32(2)))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(draft=p.half()), dict(u=torch.zeros(2, 3).double())):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(AssertionError, match="m4q_verify_tree was called"):
        call(target=p[:, :1], draft=None, tokens=i32(2), parents=i32(2), u=torch.zeros(2))
    path, count, token = call(target=p[:0], draft=p[:0], tokens=i32(0), parents=i32(0), u=torch.zeros(0))
    assert path.shape == (0, 3) and count.shape == (0,) and token.shape == (0,)
    for bad in (p.double(), p[0], p):   # a type, a shape, a CPU tensor
        with pytest.raises((TypeError, ValueError)):
            real(bad, "target")


# ---------------------------------------------------------------- the kernels' loads

@pytest.mark.parametrize("name", ["attention_paged.cu", "page_plan.cu", "verify.cu"])
def test_nothing_is_read_only(name):
    # as test_launch_overlap_cpu: these kernels start before the one ahead of them ends
    import os
    import re
    with open(os.path.join(os.path.dirname(m.__file__), "csrc", name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "ld.global.nc" not in code and "__restrict__" not in code and "__ldg" not in code


def test_cpu_tensors_are_refused(lib):
    x, pos, n = f16(2, 4, 64), i32(12).view(3, 4), i32(6).view(2, 3)
    p, kc = torch.zeros(2, 3, 50), f16(9, 2, 16, 64)
    for call in (lambda: m.rope(x, pos, FR, axes=i32(32)),
                 lambda: m.kv_write(x, x, kc, kc, m.KV_F16, i32(4), pos=pos, freqs=FR, axes=i32(32)),
                 lambda: m.page_plan(i32(2), i32(2), n, i32(2), i32(9), i32(1), 16, 4),
                 lambda: m.attention_paged(x, kc, kc, m.KV_F16, i32(8).view(4, 2), i32(4)),
                 lambda: m.verify_tree(p, p, n, n, torch.zeros(2, 3))):
        with pytest.raises(TypeError):
            call()
