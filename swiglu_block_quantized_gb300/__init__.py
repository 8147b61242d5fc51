"""Python binding of libm4q.so: the block-quantized projection GEMM and the
fused gate/up SwiGLU projection for one GB300 (sm_103a).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libm4q.so (see include/m4q.h).  PyTorch supplies device memory and
streams.  There is no fallback: if the library is missing or the device is not
sm_103, calls raise.

Functions mirror the C ABI (same names without the ``m4q_`` prefix):
    gemm(x, w, codec, n, k, out=None, path=PATH_AUTO)
    gemm_heads(x, w, codec, n, k, head_dim, out=None)
    swiglu(x, wg, wu, codec, n, k, out=None, path=PATH_AUTO)
    geglu(x, wg, wu, codec, n, k, out=None, path=PATH_AUTO)
    glu(x, wg, wu, codec, n, k, act, out=None, path=PATH_AUTO)
    mlp(x, wg, wu, wd, codec_gu, codec_d, d, f, act=ACT_SILU, h=None, out=None)
    project_host(x_host, w, codec, n, k, wu=None, act=ACT_SILU, out=None, ...)
    dequant(w, codec, n, k, out=None)
    mlx4_pack(words, scales, biases, n, k, out=None)
    attention(q, k, v, kv_codec, hkv, t, q_offset=None, causal=True, scale=None, out=None)
    rope_freqs(rot, base=10000.0, ...), rope_axes(sections, ...), rope(x, pos, freqs, ..., axes=None)
    kv_write(k, v, kc, vc, kv_codec, slots, pos=None, freqs=None, ..., q=None, axes=None)
    kv_read(kc, vc, kv_codec, slots, ...)
    attention_tree(q, kc, vc, kv_codec, past, parents, ...)
    page_plan(past, new, table, held, free, n_free, page, tokens)
    attention_paged(q, kc, vc, kv_codec, table, lengths, ...)
    verify_tree(target, draft, tokens, parents, u)
    norm_residual(h, r, w_pre, w_post=None, gate=None, ...)
    weight_bytes(codec, n, k), check_finite(t), check_device_status(),
    selftest_wait_timeout(limit_ns), status_string(code), version()
Activations are read as M whole rows (their element count must be a multiple
of the row length) and a caller's ``out`` must hold exactly the result's
element count; both are checked before anything is launched.  M = 0 (an
empty batch) returns an empty result without a launch.

``QuantLinear`` is the layer wrapper (leading batch dimensions are
flattened into M; M <= 16 streams the weights, larger M uses tcgen05), the
analogue of the pages' M4QuantizedLinear ("Releases" v0.3.0); ``QuantGLU``
wraps the gated gate/up projection (SwiGLU or GeGLU), ``QuantMLP`` the
whole gated MLP block (gate/up then down, one stream) and ``QuantQKV`` the
fused Q/K/V projection with head-major outputs.
"""
from __future__ import annotations

import ctypes
import os
import threading

Q4_0, Q8_0, Q2_0, MLX4 = 0, 1, 2, 3
CODECS = (Q4_0, Q8_0, Q2_0, MLX4)
BLOCK = {Q4_0: 32, Q8_0: 32, Q2_0: 128, MLX4: 32}
BLOCK_BYTES = {Q4_0: 18, Q8_0: 34, Q2_0: 34, MLX4: 20}
KV_F16 = 16   # fp16 KV cache values (the quantized KV cache uses Q8_0)
PATH_AUTO, PATH_GEMV, PATH_TC = 0, 1, 2
ACT_SILU, ACT_GELU = 0, 1
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_BANDS, ROPE_YARN = 0, 1, 2, 3, 4
RES_F16, RES_F32 = 0, 1
PROB_F32, PROB_F16 = 0, 1

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED_CODEC = -2
ERR_BAD_SHAPE = -3
ERR_MISALIGNED = -4
ERR_CUDA = -5
ERR_NONFINITE = -6
ERR_TIMEOUT = -7
ERR_UNSUPPORTED_DEVICE = -8
ERR_SCRATCH_LIMIT = -9
ERR_BOUNDS = -10
BUILD_BOUNDS = 1

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libm4q.so")
LIB_BOUNDS_PATH = os.path.join(HERE, "_build", "libm4q_bounds.so")   # bounds-checked build

# Every symbol declared in include/m4q.h, with its ctypes signature.
_i64, _i32, _vp, _sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
SIGNATURES = {
    "m4q_gemm": (_i32, [_vp, _vp, _i32, _i64, _i64, _i64, _vp, _vp]),
    "m4q_swiglu": (_i32, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _vp]),
    "m4q_gemm_ex": (_i32, [_vp, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _vp]),
    "m4q_swiglu_ex": (_i32, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _vp]),
    "m4q_geglu": (_i32, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _vp]),
    "m4q_gemm_heads": (_i32, [_vp, _vp, _i32, _i64, _i64, _i64, _i64, _vp, _vp]),
    "m4q_glu_ex": (_i32, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _i32, _vp]),
    "m4q_mlp": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i64, _i64, _i64, _vp, _vp, _i32, _vp]),
    "m4q_mlp_noalloc": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i64, _i64, _i64, _vp, _i32, _vp]),
    "m4q_project_host": (_i32, [_vp, _vp, _vp, _i32, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _vp,
                                _vp]),
    "m4q_dequant": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp]),
    "m4q_mlx4_pack": (_i32, [_vp, _vp, _vp, _i64, _i64, _vp, _vp]),
    "m4q_repack": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp]),
    "m4q_attention": (_i32, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _i64, _i64, _i64, _i32,
                             ctypes.c_float, _vp, _vp, _sz, _vp]),
    "m4q_attention_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64, _i64]),
    "m4q_attention_workspace": (_sz, [_i32, _i64, _i64, _i64, _i64, _i64]),
    "m4q_rope_freqs": (_i32, [_i64, ctypes.c_double, _i32, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                              ctypes.c_double, _vp, _vp]),
    "m4q_rope": (_i32, [_vp, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _i32, ctypes.c_float, _vp, _i64, _i64,
                        _vp]),
    "m4q_kv_write": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _i32,
                            ctypes.c_float, _vp, _vp, _vp, _i32, _i64, _i64, _vp, _i64, _i64, _i64, _vp, _vp]),
    "m4q_kv_read": (_i32, [_vp, _vp, _i32, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp]),
    "m4q_attention_tree": (_i32, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _i64, _i64, _i64, _vp, _vp,
                                  ctypes.c_float, _vp, _vp, _sz, _vp]),
    "m4q_attention_tree_workspace": (_sz, [_i32, _i64, _i64, _i64, _i64, _i64, _i64]),
    "m4q_rope_axes": (_i32, [_vp, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _i32, ctypes.c_float, _vp,
                             _i64, _i64, _vp]),
    "m4q_kv_write_axes": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _i32,
                                 ctypes.c_float, _vp, _vp, _vp, _i32, _i64, _i64, _vp, _i64, _i64, _i64, _vp, _vp]),
    "m4q_page_plan": (_i32, [_vp, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp]),
    "m4q_attention_paged": (_i32, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _vp,
                                   ctypes.c_float, _vp, _vp, _sz, _vp]),
    "m4q_attention_paged_workspace": (_sz, [_i32, _i64, _i64, _i64, _i64, _i64, _i64, _i64]),
    "m4q_verify_tree": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                               _vp]),
    "m4q_norm_residual": (_i32, [_vp, _vp, _i32, _vp, _vp, _i32, _vp, _i64, _i64, ctypes.c_float, ctypes.c_float,
                                 ctypes.c_float, _vp, _vp, _vp]),
    "m4q_weight_bytes": (_sz, [_i32, _i64, _i64]),
    "m4q_check_finite": (_i32, [_vp, _i64, _vp]),
    "m4q_check_device_status": (_i32, [_vp]),
    "m4q_build_flags": (_i32, []),
    "m4q_bounds_site": (_i32, [_vp]),
    "m4q_selftest_wait_timeout": (_i32, [_i64, _vp]),
    "m4q_status_string": (ctypes.c_char_p, [_i32]),
    "m4q_version": (_i32, []),
}

_lock = threading.Lock()
_lib = None


class M4QError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__("%s failed: %s (%d)" % (what, status_string(code), code))


def load(path: str | None = None):
    """Load libm4q.so (raises if it has not been built)."""
    global _lib
    if path is None and _lib is not None:   # (set once, never back: no lock to read it)
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise ImportError("libm4q.so not built (run python -m swiglu_block_quantized_gb300.buildlib): %s" % p)
        lib = ctypes.CDLL(p)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path is None:
            _lib = lib
        return lib


def build(force: bool = False, bounds: bool = False) -> str:
    from . import buildlib
    return buildlib.build(force=force, bounds=bounds)


def status_string(code: int) -> str:
    try:
        return load().m4q_status_string(code).decode()
    except ImportError:
        return "status %d" % code


def version() -> int:
    return int(load().m4q_version())


def weight_bytes(codec: int, n: int, k: int) -> int:
    return int(load().m4q_weight_bytes(codec, n, k))


def _check(rc: int, what: str):
    if rc != OK:
        raise M4QError(rc, what)


def _stream_ptr(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _require(t, dtype, what):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % what)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)


def _rows(x, k: int, what: str = "x") -> int:
    """Rows M of an activation tensor read as [M, k]; its element count must
    be a whole number of rows (M = 0 is allowed: an empty batch)."""
    if k < 1 or x.numel() % k != 0:
        raise ValueError("%s holds %d elements, not a whole number of rows of %d"
                         % (what, x.numel(), k))
    return x.numel() // k


def _result(out, shape, device, what="out"):
    """The caller's output tensor, checked to hold exactly prod(shape) fp16
    values, or a new one of that shape.  A kernel writes every element of the
    result, so a smaller buffer would be overrun and a larger one only partly
    written: both are rejected before anything is launched."""
    import torch
    need = 1
    for s in shape:
        need *= int(s)
    if out is None:
        return torch.empty(tuple(int(s) for s in shape), dtype=torch.float16, device=device)
    _require(out, torch.float16, what)
    if out.numel() != need:
        raise ValueError("%s holds %d elements, expected %d for shape %s"
                         % (what, out.numel(), need, tuple(int(s) for s in shape)))
    return out


def _packed_check(w, codec, n, k, what):
    import torch
    _require(w, torch.uint8, what)
    need = weight_bytes(codec, n, k)
    if need == 0 or w.numel() != need:
        raise ValueError("%s holds %d bytes, expected %d for %s [%d, %d]"
                         % (what, w.numel(), need, codec, n, k))


def gemm(x, w, codec: int, n: int, k: int, out=None, path: int = PATH_AUTO, stream=None):
    """Y[M, n] = X[M, k] . W^T with W packed [n, k] (uint8 blocks).  X holds
    M whole rows of k values; out, if given, exactly M * n values."""
    import torch
    _require(x, torch.float16, "x")
    _packed_check(w, codec, n, k, "w")
    m = _rows(x, k)
    out = _result(out, (m, n), x.device)
    if m == 0:
        return out
    _check(load().m4q_gemm_ex(x.data_ptr(), w.data_ptr(), codec, m, n, k, out.data_ptr(),
                              path, _stream_ptr(stream)), "m4q_gemm")
    return out


def gemm_heads(x, w, codec: int, n: int, k: int, head_dim: int, out=None, stream=None):
    """Y[n / head_dim, M, head_dim] with Y[h, m, d] = (X . W^T)[m, h * head_dim + d]."""
    import torch
    _require(x, torch.float16, "x")
    _packed_check(w, codec, n, k, "w")
    if head_dim < 1 or n % head_dim != 0:
        raise ValueError("head_dim %d must divide n = %d" % (head_dim, n))
    m = _rows(x, k)
    out = _result(out, (n // head_dim, m, head_dim), x.device)
    if m == 0:
        return out
    _check(load().m4q_gemm_heads(x.data_ptr(), w.data_ptr(), codec, m, n, k, head_dim, out.data_ptr(),
                                 _stream_ptr(stream)), "m4q_gemm_heads")
    return out


def glu(x, wg, wu, codec: int, n: int, k: int, act: int, out=None, path: int = PATH_AUTO, stream=None):
    """Y[M, n] = act(X . Wg^T) * (X . Wu^T), act = ACT_SILU or ACT_GELU."""
    import torch
    _require(x, torch.float16, "x")
    _packed_check(wg, codec, n, k, "wg")
    _packed_check(wu, codec, n, k, "wu")
    m = _rows(x, k)
    out = _result(out, (m, n), x.device)
    if m == 0:
        return out
    _check(load().m4q_glu_ex(x.data_ptr(), wg.data_ptr(), wu.data_ptr(), codec, m, n, k,
                             out.data_ptr(), act, path, _stream_ptr(stream)), "m4q_glu_ex")
    return out


def swiglu(x, wg, wu, codec: int, n: int, k: int, out=None, path: int = PATH_AUTO, stream=None):
    """Y[M, n] = SiLU(X . Wg^T) * (X . Wu^T)."""
    return glu(x, wg, wu, codec, n, k, ACT_SILU, out=out, path=path, stream=stream)


def geglu(x, wg, wu, codec: int, n: int, k: int, out=None, path: int = PATH_AUTO, stream=None):
    """Y[M, n] = GELU(X . Wg^T) * (X . Wu^T)."""
    return glu(x, wg, wu, codec, n, k, ACT_GELU, out=out, path=path, stream=stream)


def mlp(x, wg, wu, wd, codec_gu: int, codec_d: int, d: int, f: int, act: int = ACT_SILU,
        h=None, out=None, stream=None):
    """Y[M, d] = (act(X Wg^T) * (X Wu^T)) Wd^T; Wg, Wu packed [f, d], Wd packed
    [d, f].  h (fp16 [M, f]) receives the intermediate; allocated if None."""
    import torch
    _require(x, torch.float16, "x")
    _packed_check(wg, codec_gu, f, d, "wg")
    _packed_check(wu, codec_gu, f, d, "wu")
    _packed_check(wd, codec_d, d, f, "wd")
    m = _rows(x, d)
    out = _result(out, (m, d), x.device)
    if h is None:
        h = torch.empty((m, f), dtype=torch.float16, device=x.device)
    _require(h, torch.float16, "h")
    if h.numel() < m * f:
        raise ValueError("h holds %d elements, needs %d" % (h.numel(), m * f))
    if m == 0:
        return out
    _check(load().m4q_mlp(x.data_ptr(), wg.data_ptr(), wu.data_ptr(), wd.data_ptr(), codec_gu, codec_d,
                          m, d, f, h.data_ptr(), out.data_ptr(), act, _stream_ptr(stream)), "m4q_mlp")
    return out


_host_streams_by_device = {}


def _host_streams(device):
    """Two copy streams per device, created once, for project_host."""
    import torch
    key = torch.device(device).index
    if key not in _host_streams_by_device:
        _host_streams_by_device[key] = (torch.cuda.Stream(device=device), torch.cuda.Stream(device=device))
    return _host_streams_by_device[key]


def project_host(x, w, codec: int, n: int, k: int, wu=None, act: int = ACT_SILU, out=None, x_dev=None,
                 y_dev=None, chunk_rows: int = 0, stream=None):
    """Y = X W^T (wu None) or act(X W^T) * (X Wu^T) with X and Y in host
    memory: chunks of rows are copied in, projected and copied back with the
    copies overlapping the kernels (m4q_project_host).  x: CPU fp16 [..., k]
    (page-locked for overlap); out: CPU fp16 [M, n], page-locked when
    allocated here.  x_dev / y_dev: device staging [M, k] / [M, n], allocated
    if not given.  The result is complete once the current stream (or
    `stream`) has reached this point: synchronize it before reading out."""
    import torch
    if not isinstance(x, torch.Tensor) or x.is_cuda or x.dtype != torch.float16 or not x.is_contiguous():
        raise TypeError("x must be a contiguous fp16 host tensor")
    _packed_check(w, codec, n, k, "w")
    if wu is not None:
        _packed_check(wu, codec, n, k, "wu")
    m = _rows(x, k)
    if out is None:
        out = torch.empty((m, n), dtype=torch.float16, pin_memory=True)
    elif (not isinstance(out, torch.Tensor) or out.is_cuda or out.dtype != torch.float16
          or not out.is_contiguous() or out.numel() != m * n):
        raise ValueError("out must be a contiguous fp16 host tensor of %d elements" % (m * n))
    x_dev = _result(x_dev, (m, k), w.device, "x_dev")
    y_dev = _result(y_dev, (m, n), w.device, "y_dev")
    if m == 0:
        return out
    s_in, s_out = _host_streams(w.device)
    _check(load().m4q_project_host(x.data_ptr(), w.data_ptr(), wu.data_ptr() if wu is not None else None, codec,
                                   act, m, n, k, out.data_ptr(), x_dev.data_ptr(), y_dev.data_ptr(), chunk_rows,
                                   _stream_ptr(stream), ctypes.c_void_p(s_in.cuda_stream),
                                   ctypes.c_void_p(s_out.cuda_stream)), "m4q_project_host")
    return out


def dequant(w, codec: int, n: int, k: int, out=None, stream=None):
    """fp16 [n, k] decode of the packed weights (bit-exact test hook)."""
    import torch
    _packed_check(w, codec, n, k, "w")
    out = _result(out, (n, k), w.device)
    _check(load().m4q_dequant(w.data_ptr(), codec, n, k, out.data_ptr(), _stream_ptr(stream)),
           "m4q_dequant")
    return out


def mlx4_pack(words, scales, biases, n: int, k: int, out=None, stream=None):
    """MLX planar arrays -> MLX4 blocks uint8 [n, (k/32) * 20].  words holds
    the [n, k/8] little-endian uint32 code words (any contiguous CUDA tensor
    of n * k / 2 bytes, e.g. int32 [n, k/8]); scales and biases are fp16
    [n, k/32]."""
    import torch
    if not isinstance(words, torch.Tensor) or not words.is_cuda or not words.is_contiguous():
        raise TypeError("words must be a contiguous CUDA tensor")
    if k % 32 or words.numel() * words.element_size() != n * k // 2:
        raise ValueError("words must hold n * k / 2 bytes with k % 32 == 0")
    for t, what in ((scales, "scales"), (biases, "biases")):
        _require(t, torch.float16, what)
        if t.numel() != n * (k // 32):
            raise ValueError("%s must hold n * k / 32 values" % what)
    if out is None:
        out = torch.empty((n, (k // 32) * 20), dtype=torch.uint8, device=words.device)
    _packed_check(out, MLX4, n, k, "out")
    _check(load().m4q_mlx4_pack(words.data_ptr(), scales.data_ptr(), biases.data_ptr(), n, k,
                                out.data_ptr(), _stream_ptr(stream)), "m4q_mlx4_pack")
    return out


def repack(w, codec: int, n: int, k: int, out=None, stream=None):
    """Packed blocks [n, k] -> planes, uint8 [weight_bytes(codec, n, k)]: the
    code bytes of every block in row-major block order, then the fp16 scales
    [n, k/B], then (MLX4) the fp16 biases [n, k/B]."""
    import torch
    _packed_check(w, codec, n, k, "w")
    if out is None:
        out = torch.empty(weight_bytes(codec, n, k), dtype=torch.uint8, device=w.device)
    _require(out, torch.uint8, "out")
    if out.numel() != weight_bytes(codec, n, k):
        raise ValueError("out must hold %d bytes" % weight_bytes(codec, n, k))
    _check(load().m4q_repack(w.data_ptr(), codec, n, k, out.data_ptr(), _stream_ptr(stream)), "m4q_repack")
    return out


def attention(q, k, v, kv_codec: int, hkv: int, t: int, q_offset: int | None = None,
              causal: bool = True, scale: float | None = None, out=None, workspace=None, stream=None):
    """O fp16 [M, H * D] = attention of q fp16 [H, M, D] over the KV cache k,
    v [hkv, t, D] (fp16 for KV_F16; uint8 Q8_0 blocks [hkv, t, D / 32 * 34]
    for Q8_0).  q_offset defaults to t - M (the queries are the last M
    positions); scale to 1 / sqrt(D).  The workspace (the key split's
    partial results, or the Q8_0 caches decoded to fp16 for a prefill-sized
    call) is allocated here when not given; workspace=False runs without
    one."""
    import torch
    _require(q, torch.float16, "q")
    if q.dim() != 3:
        raise ValueError("q must be [H, M, D]")
    h, m_, d = q.shape
    row = 2 * d if kv_codec == KV_F16 else (d // 32) * 34
    for x, what in ((k, "k"), (v, "v")):
        _require(x, torch.float16 if kv_codec == KV_F16 else torch.uint8, what)
        if x.numel() * x.element_size() != hkv * t * row:
            raise ValueError("%s must hold [%d, %d] rows of %d bytes" % (what, hkv, t, row))
    if q_offset is None:
        q_offset = t - m_
    if scale is None:
        scale = float(d) ** -0.5
    if out is None:
        out = torch.empty((m_, h * d), dtype=torch.float16, device=q.device)
    _require(out, torch.float16, "out")
    if out.numel() != m_ * h * d:
        raise ValueError("out must hold M * H * D values")
    lib = load()
    if workspace is None:
        need = int(lib.m4q_attention_workspace(kv_codec, h, hkv, m_, t, d))
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    elif workspace is False:
        workspace = None
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.m4q_attention(q.data_ptr(), k.data_ptr(), v.data_ptr(), kv_codec, h, hkv, m_, t, d,
                             q_offset, int(bool(causal)), float(scale), out.data_ptr(), ws_ptr, ws_bytes,
                             _stream_ptr(stream)), "m4q_attention")
    return out


# The serving calls below run once or several times a layer for a few tokens,
# where the binding's own time counts: checks take the short way where they
# pass and the long one (which raises) where they do not.
_torch = None


def _t():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _need(t, dtype, what):
    """_require, short where it passes."""
    try:
        if t.dtype is dtype and t.is_cuda and t.is_contiguous():
            return
    except AttributeError:
        pass
    _require(t, dtype, what)


def _one_device(first, *others):
    """All tensors live on the current device (the library launches there);
    returns its index."""
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors are on %s and %s" % (first.device, t.device))
    if dev != _torch._C._cuda_getDevice():
        raise ValueError("tensors are on %s, but cuda:%d is the current device"
                         % (first.device, _torch.cuda.current_device()))
    return dev


def _allocate(shape, dtype, like, stream):
    """A new tensor on `like`'s device that belongs to `stream` (the current
    one if None)."""
    if stream is None:
        return _t().empty(shape, dtype=dtype, device=like.device)
    with _t().cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=like.device)


def _raw_stream(stream, dev):
    """The stream's handle (device dev's current stream's if None, without a
    Stream object in between)."""
    if stream is not None:
        return stream.cuda_stream
    return _torch._C._cuda_getCurrentRawStream(dev)


def _plain(t, dtype, shape):
    """A contiguous CUDA tensor of this type and shape: nothing more to check."""
    return t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous()


def _ints(t, dtype, n, what):
    _need(t, dtype, what)
    if t.numel() != n:
        raise ValueError("%s holds %d values, expected %d" % (what, t.numel(), n))


def _halfs(t, n, what):
    """A caller's contiguous fp16 tensor of exactly n values."""
    _need(t, _t().float16, what)
    if t.numel() != n:
        raise ValueError("%s holds %d elements, expected %d" % (what, t.numel(), n))
    return t


def _head_rows(x, what):
    """fp16 rows [heads, M, D] with unit-stride values, any head and row
    strides; returns (heads, M, D, head stride, row stride)."""
    if not isinstance(x, _t().Tensor) or x.dtype is not _torch.float16:
        raise TypeError("%s must be a torch.float16 tensor" % what)
    if x.dim() != 3:
        raise ValueError("%s must be [heads, M, D]" % what)
    (h, n, d), (hs, rs, one) = x.shape, x.stride()
    if one != 1 and d > 1:
        raise ValueError("%s must be [heads, M, D] with unit-stride rows" % what)
    if not x.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % what)
    return h, n, d, hs if h > 1 else 0, rs if n > 1 else 0


def _cache_shape(kc, vc, kv_codec):
    """(B, Hkv, C, D) of a pair of caches [B, Hkv, C, row] (or [Hkv, C, row]:
    one sequence)."""
    if kv_codec == KV_F16:
        dtype = _t().float16
    elif kv_codec == Q8_0:
        dtype = _t().uint8
    else:
        raise M4QError(ERR_UNSUPPORTED_CODEC, "KV cache")
    shape = None
    if kc is not None:
        _need(kc, dtype, "kc")
        shape = kc.shape
    if vc is not None:
        _need(vc, dtype, "vc")
        if shape is not None and vc.shape != shape:
            raise ValueError("kc and vc must have one shape")
        shape = vc.shape
    if len(shape) == 4:
        b, hkv, c, row = shape
    elif len(shape) == 3:
        b, (hkv, c, row) = 1, shape
    else:
        raise ValueError("a cache must be [B, Hkv, C, row] or [Hkv, C, row]")
    d = row if kv_codec == KV_F16 else row // 34 * 32
    if d not in (64, 128) or (kv_codec != KV_F16 and row % 34):
        raise ValueError("cache rows of %d are not fp16 or Q8_0 rows of 64 or 128 values" % row)
    return b, hkv, c, d


def rope_freqs(rot: int, base: float = 10000.0, scaling: int = ROPE_PLAIN, factor: float = 1.0,
               original: float = 0.0, low: float = 1.0, high: float = 32.0, device="cuda"):
    """(freqs, mscale): the table of rotary frequencies for rope and kv_write,
    int64 [rot / 2] on `device` (turns per position in units of 2^-64), and the
    magnitude factor of the scaling (m4q_rope_freqs).  ROPE_BANDS and ROPE_YARN
    mix by the turns of a pair over the original length; a model trained with a
    ramp over pair indices needs a table of its own."""
    import torch
    host = (ctypes.c_int64 * max(1, rot // 2))()
    mscale = ctypes.c_float()
    _check(load().m4q_rope_freqs(rot, base, scaling, factor, original, low, high, host, ctypes.byref(mscale)),
           "m4q_rope_freqs")
    return torch.tensor(list(host), dtype=torch.int64).to(device), float(mscale.value)


def rope_axes(sections, dealt: bool = False, device="cuda"):
    """The table of axes for rope and kv_write, int32 [sum(sections)] on
    `device`: sections[a] pairs turn by the positions of axis a, one section
    after the other; dealt: pair i belongs to axis i % len(sections) while that
    axis has pairs left, and to axis 0 otherwise (sections[0] is the rest)."""
    import torch
    n = [int(v) for v in sections]
    if not n or len(n) > 8 or min(n) < 0 or sum(n) < 1:
        raise ValueError("sections must be up to 8 counts of pairs")
    if not dealt:
        table = [a for a, c in enumerate(n) for _ in range(c)]
    else:
        table = [i % len(n) if i < len(n) * n[i % len(n)] else 0 for i in range(sum(n))]
        if [table.count(a) for a in range(len(n))] != n:
            raise ValueError("%s pairs cannot be dealt out in turn" % (n,))
    return torch.tensor(table, dtype=torch.int32).to(device)


def _turn_args(pos, freqs, m_, axes):
    """(rot, axes, their pointer): one axis (0, None) without a table."""
    pairs = freqs.numel()
    if axes is None:
        _ints(pos, _t().int32, m_, "pos")
        _need(freqs, _torch.int64, "freqs")
        return 2 * pairs, 0, None
    _need(pos, _t().int32, "pos")
    if pos.dim() != 2 or pos.shape[1] != m_:
        raise ValueError("pos must be [axes, %d]" % m_)
    _need(freqs, _torch.int64, "freqs")
    _ints(axes, _torch.int32, pairs, "axes")
    return 2 * pairs, pos.shape[0], axes.data_ptr()


def rope(x, pos, freqs, layout: int = ROPE_HALF, mscale: float = 1.0, out=None, stream=None, axes=None):
    """Rotary positions: the first 2 * len(freqs) values of each row of x fp16
    [H, M, D] turned by pos int32 [M].  x may have any head and row strides
    that are multiples of 8.  out (fp16 [H, M, D], rows that do not overlap)
    may be x itself.  With axes int32 [len(freqs)] (rope_axes) pos is [A, M],
    and pair i turns by pos[axes[i]]."""
    h, m_, d, hs, rs = _head_rows(x, "x")
    rot, n_axes, p_axes = _turn_args(pos, freqs, m_, axes)
    if out is None:
        out = _allocate((h, m_, d), _torch.float16, x, stream)
        ohs, ors = m_ * d, d
    else:
        oh, om, od, ohs, ors = _head_rows(out, "out")
        if (oh, om, od) != (h, m_, d):
            raise ValueError("out must be [%d, %d, %d]" % (h, m_, d))
        reach = d   # rows in order of their step: each starts past the end of the ones before
        for step, count in sorted(((ohs, oh), (ors, om))):
            if count > 1:
                if step < reach:
                    raise ValueError("out's rows overlap")
                reach += step * (count - 1)
        if out.data_ptr() == x.data_ptr() and (hs, rs) != (ohs, ors):
            raise ValueError("out starts where x does, with other strides")
    dev = _one_device(x, pos, freqs, out, axes)
    if h == 0 or m_ == 0:
        return out
    if p_axes is not None:
        rc = load().m4q_rope_axes(x.data_ptr(), hs, rs, h, m_, d, pos.data_ptr(), n_axes, freqs.data_ptr(), p_axes,
                                  rot, layout, mscale, out.data_ptr(), ohs, ors, _raw_stream(stream, dev))
        if rc:
            raise M4QError(rc, "m4q_rope_axes")
        return out
    rc = load().m4q_rope(x.data_ptr(), hs, rs, h, m_, d, pos.data_ptr(), freqs.data_ptr(), rot, layout, mscale,
                         out.data_ptr(), ohs, ors, _raw_stream(stream, dev))
    if rc:
        raise M4QError(rc, "m4q_rope")
    return out


def kv_write(k, v, kc, vc, kv_codec: int, slots, pos=None, freqs=None, layout: int = ROPE_HALF,
             mscale: float = 1.0, q=None, q_out=None, stream=None, axes=None):
    """Write the rows k, v fp16 [Hkv, M, D] of M tokens to the caches kc, vc
    [B, Hkv, C, row] at slots int32 [M] (b * C + j; outside the cache: not
    written), k turned by pos and freqs when given.  With q fp16 [H, M, D] the
    queries are turned in the same launch and returned as q_out [H, M, D].  With
    axes (rope) pos is [A, M].  Pages [P, Hkv, page, row] are written by the slots
    of page_plan."""
    hkv, m_, d, khs, krs = _head_rows(k, "k")
    vh, vm, vd, vhs, vrs = _head_rows(v, "v")
    b, ch, c, cd = _cache_shape(kc, vc, kv_codec)
    if kc is None or vc is None:
        raise ValueError("both caches are written")
    if vh != hkv or vm != m_ or vd != d or ch != hkv or cd != d:
        raise ValueError("k, v and the caches must agree on heads, rows and D")
    _ints(slots, _torch.int32, m_, "slots")
    rot, h, qhs, qrs, p_pos, p_freqs, p_q, p_qo, p_axes = 0, 0, 0, 0, None, None, None, None, None
    if freqs is not None:
        if pos is None:
            raise ValueError("freqs needs pos")
        rot, n_axes, p_axes = _turn_args(pos, freqs, m_, axes)
        p_pos, p_freqs = pos.data_ptr(), freqs.data_ptr()
    elif axes is not None:
        raise ValueError("axes needs freqs")
    if q is not None:
        if freqs is None:
            raise ValueError("q needs freqs")
        h, qm, qd, qhs, qrs = _head_rows(q, "q")
        if qm != m_ or qd != d or h == 0:
            raise ValueError("q must be [H, %d, %d]" % (m_, d))
        p_q = q.data_ptr()
        if q_out is None:
            q_out = _allocate((h, m_, d), _torch.float16, q, stream)
            p_qo = q_out.data_ptr()
        else:
            _halfs(q_out, h * m_ * d, "q_out")
            p_qo = q_out.data_ptr()
            if p_qo == p_q and not q.is_contiguous():
                raise ValueError("q_out starts where q does, with other strides")
        dev = _one_device(k, v, kc, vc, slots, pos, freqs, q, q_out, axes)
    else:
        q_out = None
        dev = _one_device(k, v, kc, vc, slots, pos if rot else None, freqs, axes if rot else None)
    if m_ == 0:
        return q_out
    if p_axes is not None:
        rc = load().m4q_kv_write_axes(k.data_ptr(), khs, krs, v.data_ptr(), vhs, vrs, hkv, m_, d, p_pos, n_axes,
                                      p_freqs, p_axes, rot, layout, mscale, slots.data_ptr(), kc.data_ptr(),
                                      vc.data_ptr(), kv_codec, b, c, p_q, qhs, qrs, h, p_qo, _raw_stream(stream, dev))
        if rc:
            raise M4QError(rc, "m4q_kv_write_axes")
        return q_out
    rc = load().m4q_kv_write(k.data_ptr(), khs, krs, v.data_ptr(), vhs, vrs, hkv, m_, d, p_pos, p_freqs, rot, layout,
                             mscale, slots.data_ptr(), kc.data_ptr(), vc.data_ptr(), kv_codec, b, c, p_q, qhs, qrs, h,
                             p_qo, _raw_stream(stream, dev))
    if rc:
        raise M4QError(rc, "m4q_kv_write")
    return q_out


def kv_read(kc, vc, kv_codec: int, slots, k_out=None, v_out=None, stream=None):
    """(k, v): the cache rows slots int32 [n] of every KV head as fp16 [Hkv, n,
    D] (a slot outside the cache: zeros).  kc or vc may be None (and so its
    result)."""
    if kc is None and vc is None:
        raise ValueError("kc or vc is needed")
    b, hkv, c, d = _cache_shape(kc, vc, kv_codec)
    n = slots.numel()
    _ints(slots, _torch.int32, n, "slots")
    shape, total = (hkv, n, d), hkv * n * d
    pk = pv = pko = pvo = None
    if kc is None:
        k_out = None
    else:
        k_out = _allocate(shape, _torch.float16, kc, stream) if k_out is None else _halfs(k_out, total, "k_out")
        pk, pko = kc.data_ptr(), k_out.data_ptr()
    if vc is None:
        v_out = None
    else:
        v_out = _allocate(shape, _torch.float16, vc, stream) if v_out is None else _halfs(v_out, total, "v_out")
        pv, pvo = vc.data_ptr(), v_out.data_ptr()
    dev = _one_device(slots, kc, vc, k_out, v_out)
    if n:
        rc = load().m4q_kv_read(pk, pv, kv_codec, b, hkv, c, d, slots.data_ptr(), n, pko, pvo,
                                _raw_stream(stream, dev))
        if rc:
            raise M4QError(rc, "m4q_kv_read")
    return k_out, v_out


def attention_tree(q, kc, vc, kv_codec: int, past, parents, scale: float | None = None, out=None, workspace=None,
                   stream=None):
    """O fp16 [B * N, H * D]: attention of the drafted nodes q fp16 [H, B * N,
    D] (node i of sequence b is row b * N + i) over the caches kc, vc [B, Hkv,
    C, row].  A node sees the rows below past int32 [B], its ancestors by
    parents int32 [B, N] or [B * N] (-1: the context; anything else that is not
    an earlier used node: unused, a zero row) and itself, at rows past + node.
    N = 1 is one new token a sequence.  The workspace is allocated here when not given;
    workspace=False runs without one (no key split)."""
    _need(q, _t().float16, "q")
    if kc is None or vc is None:
        raise ValueError("both caches are read")
    b, hkv, c, d = _cache_shape(kc, vc, kv_codec)
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError("q must be [H, B * N, %d]" % d)
    h, rows, _ = q.shape
    if b == 0 or rows % b:
        raise ValueError("q holds %d rows, not a whole number for %d sequences" % (rows, b))
    n = rows // b
    _ints(past, _torch.int32, b, "past")
    _ints(parents, _torch.int32, rows, "parents")
    if parents.dim() > 1 and tuple(parents.shape) != (b, n):   # [N, B] holds as many
        raise ValueError("parents must be [%d, %d]" % (b, n))
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _allocate((rows, h * d), _torch.float16, q, stream)
    else:
        _halfs(out, rows * h * d, "out")
    if rows == 0 or h == 0:
        return out
    lib = load()
    p_ws, n_ws = None, 0
    if workspace is None:
        n_ws = lib.m4q_attention_tree_workspace(kv_codec, b, h, hkv, n, c, d)
        if n_ws:
            workspace = _allocate((n_ws,), _torch.uint8, q, stream)
            p_ws = workspace.data_ptr()
    elif workspace is False:
        workspace = None
    else:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        p_ws, n_ws = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    dev = _one_device(q, kc, vc, past, parents, out, workspace)
    rc = lib.m4q_attention_tree(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), kv_codec, b, h, hkv, n, c, d,
                                past.data_ptr(), parents.data_ptr(), scale, out.data_ptr(), p_ws, n_ws,
                                _raw_stream(stream, dev))
    if rc:
        raise M4QError(rc, "m4q_attention_tree")
    return out


def page_plan(past, new, table, held, free, n_free, page: int, tokens: int, out=None, stream=None):
    """(slots, pos, lengths, starts): the cache rows of a step's tokens, planned on
    the GPU.  Sequence b has past int32 [B] rows and gets new int32 [B] tokens
    (below 0: it has ended).  table int32 [B, W], held int32 [B], free int32 [P]
    and n_free int32 [1] are the pages' state and are updated: pages of `page`
    rows that b lacks come from the end of free[:n_free], those of an ended
    sequence go back on top (a page is held by one sequence only: m4q_page_plan says
    how a shared prefix is given back).  slots and pos int32 [tokens] are those of all
    sequences' tokens one after the other, from starts int32 [B + 1] on (behind
    them -1 and 0; -1 too where the pages ran out); lengths int32 [B] counts the
    rows after the step.  out: the four tensors of the results."""
    i32 = _t().int32
    if not isinstance(table, _torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be [B, W]")
    b, w = table.shape
    _need(table, i32, "table")
    _ints(past, i32, b, "past")
    _ints(new, i32, b, "new")
    _ints(held, i32, b, "held")
    _ints(n_free, i32, 1, "n_free")
    _need(free, i32, "free")
    tokens = int(tokens)
    if tokens < 1:
        raise ValueError("tokens must be at least 1")
    if out is None:   # (four small tensors cost less of the host's time than views of one)
        slots, pos = _allocate((tokens,), i32, table, stream), _allocate((tokens,), i32, table, stream)
        lengths, starts = _allocate((b,), i32, table, stream), _allocate((b + 1,), i32, table, stream)
    else:
        slots, pos, lengths, starts = out
        for t, n, what in ((slots, tokens, "slots"), (pos, tokens, "pos"), (lengths, b, "lengths"),
                           (starts, b + 1, "starts")):
            _ints(t, i32, n, what)
    dev = _one_device(table, past, new, held, free, n_free, slots, pos, lengths, starts)
    rc = load().m4q_page_plan(past.data_ptr(), new.data_ptr(), b, page, table.data_ptr(), w, held.data_ptr(),
                              free.data_ptr(), free.numel(), n_free.data_ptr(), tokens, slots.data_ptr(),
                              pos.data_ptr(), lengths.data_ptr(), starts.data_ptr(), _raw_stream(stream, dev))
    if rc:
        raise M4QError(rc, "m4q_page_plan")
    return slots, pos, lengths, starts


def attention_paged(q, kc, vc, kv_codec: int, table, lengths, scale: float | None = None, out=None, workspace=None,
                    stream=None):
    """O fp16 [B, H * D]: attention of one new token of each of B sequences, q
    fp16 [H, B, D], over the pages kc, vc [P, Hkv, page, row].  Sequence b sees
    its rows j < lengths int32 [B], row j at place j % page of page
    table[b, j // page] (table int32 [B, W]); none: a zero row.  Several tokens of a
    sequence (a prompt's, a drafted chain's) are rows of their own: q [H, T, D], the
    table's row for each and lengths up to itself; each reads its keys again.  The
    workspace is allocated here when not given; workspace=False runs without one (no
    key split)."""
    _need(q, _t().float16, "q")
    if kc is None or vc is None:
        raise ValueError("both pools are read")
    pages, hkv, page, d = _cache_shape(kc, vc, kv_codec)
    if kc.dim() != 4:
        raise ValueError("a page pool must be [P, Hkv, page, row]")
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError("q must be [H, B, %d]" % d)
    h, b, _ = q.shape
    _need(table, _torch.int32, "table")
    if table.dim() != 2 or table.shape[0] != b:
        raise ValueError("table must be [%d, W]" % b)
    w = table.shape[1]
    _ints(lengths, _torch.int32, b, "lengths")
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _allocate((b, h * d), _torch.float16, q, stream)
    else:
        _halfs(out, b * h * d, "out")
    if b == 0 or h == 0:
        return out
    lib = load()
    p_ws, n_ws = None, 0
    if workspace is None:
        n_ws = lib.m4q_attention_paged_workspace(kv_codec, b, h, hkv, pages, page, w, d)
        if n_ws:
            workspace = _allocate((n_ws,), _torch.uint8, q, stream)
            p_ws = workspace.data_ptr()
    elif workspace is False:
        workspace = None
    else:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        p_ws, n_ws = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    dev = _one_device(q, kc, vc, table, lengths, out, workspace)
    rc = lib.m4q_attention_paged(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), kv_codec, b, h, hkv, pages, page, d,
                                 table.data_ptr(), w, lengths.data_ptr(), scale, out.data_ptr(), p_ws, n_ws,
                                 _raw_stream(stream, dev))
    if rc:
        raise M4QError(rc, "m4q_attention_paged")
    return out


def _prob_rows(x, what):
    """fp32 or fp16 probabilities [B, N, V] with unit-stride rows; returns the
    sequence and row strides."""
    if not isinstance(x, _t().Tensor) or not (x.dtype is _torch.float32 or x.dtype is _torch.float16):
        raise TypeError("%s must be an fp32 or fp16 tensor" % what)
    if x.dim() != 3:
        raise ValueError("%s must be [B, N, V]" % what)
    if not x.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % what)
    b, n, v = x.shape
    bs, rs, one = x.stride()
    if one != 1 and v > 1:
        raise ValueError("%s must be [B, N, V] with unit-stride rows" % what)
    return bs if b > 1 else 0, rs if n > 1 else 0


def verify_tree(target, draft, tokens, parents, u, out=None, stream=None):
    """(path, count, token): drafted trees verified against the target's
    probabilities.  target and draft [B, N, V] (both fp32 or both fp16, any
    sequence and row strides) are the distributions behind node i of sequence b;
    node 0 is its last known token (parents -1), node i > 0 the drafted token
    tokens int32 [B, N] behind node parents int32 [B, N] in [0, i).  u fp32 [B, N]
    in [0, 1): u[b, i] decides on node i, u[b, 0] draws the next token.  path
    int32 [B, N] holds the nodes kept (0 first, -1 behind them), count int32 [B]
    their number, token int32 [B] the next token.  draft may be None with N = 1.
    out: the three tensors of the results."""
    tbs, trs = _prob_rows(target, "target")
    b, n, v = target.shape
    p_draft, dbs, drs = None, 0, 0
    if draft is not None:
        if draft.dtype is not target.dtype:
            raise TypeError("draft must be of target's type")
        if draft.shape != target.shape:
            raise ValueError("draft must be [%d, %d, %d]" % (b, n, v))
        dbs, drs = _prob_rows(draft, "draft")
        p_draft = draft.data_ptr()
    elif n > 1:
        raise ValueError("draft is needed with drafted nodes")
    shape = target.shape[:2]
    if not (_plain(tokens, _torch.int32, shape) and _plain(parents, _torch.int32, shape) and
            _plain(u, _torch.float32, shape)):
        for t, dtype, what in ((tokens, _torch.int32, "tokens"), (parents, _torch.int32, "parents"),
                               (u, _torch.float32, "u")):
            _ints(t, dtype, b * n, what)
            if t.dim() > 1 and tuple(t.shape) != (b, n):
                raise ValueError("%s must be [%d, %d]" % (what, b, n))
    if out is None:
        path, count = _allocate((b, n), _torch.int32, target, stream), _allocate((b,), _torch.int32, target, stream)
        token = _allocate((b,), _torch.int32, target, stream)
    else:
        path, count, token = out
        for t, size, what in ((path, b * n, "path"), (count, b, "count"), (token, b, "token")):
            _ints(t, _torch.int32, size, what)
    dev = _one_device(target, draft, tokens, parents, u, path, count, token)
    if b:
        rc = load().m4q_verify_tree(target.data_ptr(), tbs, trs, p_draft, dbs, drs,
                                    PROB_F16 if target.dtype is _torch.float16 else PROB_F32, b, n, v,
                                    tokens.data_ptr(), parents.data_ptr(), u.data_ptr(), path.data_ptr(),
                                    count.data_ptr(), token.data_ptr(), _raw_stream(stream, dev))
        if rc:
            raise M4QError(rc, "m4q_verify_tree")
    return path, count, token


def norm_residual(h, r, w_pre, w_post=None, gate=None, res_scale: float = 1.0, branch_scale: float = 1.0,
                  eps: float = 1e-6, out=None, r_out=None, stream=None):
    """(y, r_new): r_new = res_scale * r + branch_scale * gate * rmsnorm(h) *
    w_post, y = rmsnorm(r_new) * w_pre, over the last dimension.  r is fp16 or
    fp32; h, y and the weights fp16; gate [D] or one value for each of h.
    Without w_post the branch is not normalised; with h None r is only
    normalised (r_new is r); with w_pre None there is no y.  r_out may be r,
    out may be h."""
    f16 = _t().float16
    res32 = getattr(r, "dtype", None) is _torch.float32
    if not isinstance(r, _torch.Tensor) or not (res32 or r.dtype is f16):
        raise TypeError("r must be an fp16 or fp32 CUDA tensor")
    _need(r, r.dtype, "r")
    shape = r.shape
    if len(shape) < 1:
        raise ValueError("r needs a last dimension")
    d, total = shape[-1], r.numel()
    m_ = total // d if d else 0
    if h is None and (w_post is not None or gate is not None or r_out is not None):
        raise ValueError("w_post, gate and r_out need h")
    if h is None and w_pre is None:
        raise ValueError("nothing to compute")
    p_h = p_wpost = p_wpre = p_gate = p_y = p_ro = y = None
    gate_rows = 0
    if h is not None:
        p_h = _halfs(h, total, "h").data_ptr()
    if w_post is not None:
        p_wpost = _halfs(w_post, d, "w_post").data_ptr()
    if gate is not None:
        gate_rows = int(gate.numel() != d)
        p_gate = _halfs(gate, total if gate_rows else d, "gate").data_ptr()
        if gate.shape[-1] != d and not (gate_rows and gate.dim() == 1):   # a value for each row, say
            raise ValueError("gate must be [%d] or hold one value for each of h" % d)
    if w_pre is not None:
        p_wpre = _halfs(w_pre, d, "w_pre").data_ptr()
        y = _allocate(shape, f16, r, stream) if out is None else _halfs(out, total, "out")
        p_y = y.data_ptr()
    if h is not None:
        if r_out is None:
            r_out = _allocate(shape, r.dtype, r, stream)
        else:
            _need(r_out, r.dtype, "r_out")
            if r_out.numel() != total:
                raise ValueError("r_out must hold %d values" % total)
        p_ro = r_out.data_ptr()
    dev = _one_device(r, h, w_pre, w_post, gate, y, r_out)
    if m_:
        rc = load().m4q_norm_residual(p_h, r.data_ptr(), RES_F32 if res32 else RES_F16, p_wpost, p_gate, gate_rows,
                                      p_wpre, m_, d, res_scale, branch_scale, eps, p_ro, p_y,
                                      _raw_stream(stream, dev))
        if rc:
            raise M4QError(rc, "m4q_norm_residual")
    return y, r_out if h is not None else r


def check_finite(t, stream=None) -> bool:
    """True if every element of the fp16 tensor is finite (synchronizes)."""
    import torch
    _require(t, torch.float16, "t")
    rc = load().m4q_check_finite(t.data_ptr(), t.numel(), _stream_ptr(stream))
    if rc == ERR_NONFINITE:
        return False
    _check(rc, "m4q_check_finite")
    return True


def check_device_status(stream=None) -> int:
    """Synchronize and return (and clear) the device status: OK, ERR_BOUNDS or ERR_TIMEOUT."""
    return int(load().m4q_check_device_status(_stream_ptr(stream)))


def build_flags() -> int:
    """BUILD_BOUNDS for the bounds-checked build, else 0."""
    return int(load().m4q_build_flags())


def bounds_site(stream=None) -> int:
    """Synchronize and return (and clear) the site of the first failed bounds
    check (0: none; bounds-checked build only)."""
    rc = int(load().m4q_bounds_site(_stream_ptr(stream)))
    if rc < 0:
        _check(rc, "m4q_bounds_site")
    return rc


def selftest_wait_timeout(limit_ns: int, stream=None):
    _check(load().m4q_selftest_wait_timeout(int(limit_ns), _stream_ptr(stream)),
           "m4q_selftest_wait_timeout")


class QuantLinear:
    """A linear layer over block-quantized weights [out_features, in_features]
    (GEMV for M <= 16, tcgen05 otherwise); leading dims of x are flattened."""

    def __init__(self, weight, codec: int, out_features: int, in_features: int):
        _packed_check(weight, codec, out_features, in_features, "weight")
        self.weight, self.codec = weight, codec
        self.out_features, self.in_features = out_features, in_features

    def __call__(self, x):
        lead = x.shape[:-1]
        if x.shape[-1] != self.in_features:
            raise ValueError("last dim of x must be %d" % self.in_features)
        x2 = x.reshape(-1, self.in_features)
        y = gemm(x2, self.weight, self.codec, self.out_features, self.in_features)
        return y.reshape(*lead, self.out_features)


class QuantGLU:
    """The fused gate/up projection act(x Wg^T) * (x Wu^T) (SwiGLU or GeGLU);
    leading dims of x are flattened."""

    def __init__(self, wg, wu, codec: int, out_features: int, in_features: int, act: int = ACT_SILU):
        _packed_check(wg, codec, out_features, in_features, "wg")
        _packed_check(wu, codec, out_features, in_features, "wu")
        self.wg, self.wu, self.codec, self.act = wg, wu, codec, act
        self.out_features, self.in_features = out_features, in_features

    def __call__(self, x):
        lead = x.shape[:-1]
        x2 = x.reshape(-1, self.in_features)
        y = glu(x2, self.wg, self.wu, self.codec, self.out_features, self.in_features, self.act)
        return y.reshape(*lead, self.out_features)


class QuantSwiGLU(QuantGLU):
    """The fused gate/up projection SiLU(x Wg^T) * (x Wu^T)."""

    def __init__(self, wg, wu, codec: int, out_features: int, in_features: int):
        super().__init__(wg, wu, codec, out_features, in_features, ACT_SILU)


class QuantMLP:
    """The gated MLP block: down(act(x Wg^T) * (x Wu^T)).  Wg, Wu: packed
    [hidden_ff, hidden]; Wd: packed [hidden, hidden_ff].  The fp16
    intermediate buffer is kept and reused across calls of the same M."""

    def __init__(self, wg, wu, wd, codec_gu: int, codec_d: int, hidden: int, hidden_ff: int,
                 act: int = ACT_SILU):
        _packed_check(wg, codec_gu, hidden_ff, hidden, "wg")
        _packed_check(wu, codec_gu, hidden_ff, hidden, "wu")
        _packed_check(wd, codec_d, hidden, hidden_ff, "wd")
        self.wg, self.wu, self.wd = wg, wu, wd
        self.codec_gu, self.codec_d, self.act = codec_gu, codec_d, act
        self.hidden, self.hidden_ff = hidden, hidden_ff
        self._h = None

    def __call__(self, x):
        import torch
        lead = x.shape[:-1]
        x2 = x.reshape(-1, self.hidden)
        m = x2.shape[0]
        if self._h is None or self._h.shape[0] != m or self._h.device != x2.device:
            self._h = torch.empty((m, self.hidden_ff), dtype=torch.float16, device=x2.device)
        y = mlp(x2, self.wg, self.wu, self.wd, self.codec_gu, self.codec_d, self.hidden, self.hidden_ff,
                act=self.act, h=self._h)
        return y.reshape(*lead, self.hidden)


class QuantQKV:
    """Fused Q/K/V projection: one GEMM on the row concatenation of Wq [hq * hd,
    hidden], Wk and Wv [hkv * hd, hidden], written head-major, returning the
    views q [hq, M, hd], k [hkv, M, hd], v [hkv, M, hd] (no transposes)."""

    def __init__(self, wq, wk, wv, codec: int, hidden: int, head_dim: int, q_heads: int, kv_heads: int):
        import torch
        _packed_check(wq, codec, q_heads * head_dim, hidden, "wq")
        _packed_check(wk, codec, kv_heads * head_dim, hidden, "wk")
        _packed_check(wv, codec, kv_heads * head_dim, hidden, "wv")
        self.w = torch.cat([wq, wk, wv]).contiguous()
        self.codec, self.hidden, self.head_dim = codec, hidden, head_dim
        self.q_heads, self.kv_heads = q_heads, kv_heads

    def __call__(self, x):
        x2 = x.reshape(-1, self.hidden)
        n = (self.q_heads + 2 * self.kv_heads) * self.head_dim
        y = gemm_heads(x2, self.w, self.codec, n, self.hidden, self.head_dim)
        hq, hk = self.q_heads, self.kv_heads
        return y[:hq], y[hq:hq + hk], y[hq + hk:]
