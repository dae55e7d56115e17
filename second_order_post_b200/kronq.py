"""Python binding of libkronq.so (include/kronq.h): argument marshalling only.

Every function keeps the C name and argument order; tensors are passed as
device pointers of torch CUDA tensors and the call is enqueued on the current
torch CUDA stream (or ``stream=``). A non-OK status raises ``KronqError``.
There is no fallback: without the compiled library this module raises at
import time.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkronq.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "kronq.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with "
        "`python -m second_order_post_b200.build` (nvcc, sm_100a)")
_lib = ctypes.CDLL(LIB_PATH)

# ---------------------------------------------------------------- constants
KRONQ_OK = 0
KRONQ_ERR_INVALID_ARG = 1
KRONQ_ERR_UNSUPPORTED = 2
KRONQ_ERR_NOT_PD = 3
KRONQ_ERR_NONFINITE = 4
KRONQ_ERR_TIMEOUT = 5
KRONQ_ERR_CUDA = 6
KRONQ_F32 = 0
KRONQ_BF16 = 1
KRONQ_ACT_NONE, KRONQ_ACT_RELU, KRONQ_ACT_SILU, KRONQ_ACT_GELU, KRONQ_ACT_GELU_TANH = range(5)
KRONQ_ACTS = {"none": KRONQ_ACT_NONE, "relu": KRONQ_ACT_RELU, "silu": KRONQ_ACT_SILU,
              "gelu": KRONQ_ACT_GELU, "gelu_tanh": KRONQ_ACT_GELU_TANH}
KRONQ_FLAG_NO_ROT_IN = 0x1
KRONQ_FLAG_NO_ROT_OUT = 0x2
KRONQ_FLAG_NO_SCALE = 0x4
KRONQ_WS_BIIP, KRONQ_WS_CHOL, KRONQ_WS_QUANT, KRONQ_WS_LOSS, KRONQ_WS_QUANT_SPLIT = 0, 1, 2, 3, 4


class kronq_rot(ctypes.Structure):
    _fields_ = [("had", ctypes.c_int64), ("m", ctypes.c_int64)]


class kronq_opts(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("group", ctypes.c_int32),
                ("block", ctypes.c_int32), ("damp_rel", ctypes.c_float),
                ("scale_exp", ctypes.c_float), ("seed", ctypes.c_uint64),
                ("rot_in", kronq_rot), ("rot_out", kronq_rot),
                ("flags", ctypes.c_uint32)]


def make_opts(bits=4, group=128, block=128, damp_rel=0.01, scale_exp=0.25,
              seed=0, rot_in=(1, 1), rot_out=(1, 1), flags=0) -> kronq_opts:
    return kronq_opts(bits, group, block, damp_rel, scale_exp, seed,
                      kronq_rot(*rot_in), kronq_rot(*rot_out), flags)


class KronqError(RuntimeError):
    def __init__(self, fn, status):
        msg = _lib.kronq_status_string(status).decode()
        if status == KRONQ_ERR_CUDA:
            msg += ": " + _lib.kronq_last_cuda_error().decode()
        super().__init__(f"{fn}: {msg} (status {status})")
        self.status = status


_p, _i64, _f, _d, _sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_float,
                         ctypes.c_double, ctypes.c_size_t)
_OPTS = ctypes.POINTER(kronq_opts)
_SIGS = {
    "kronq_accum_cov": [_p, _p, ctypes.c_int, _i64, _i64, _i64, _f, _f, _p, _p],
    "kronq_sensitivity": [_p, _p, _i64, _p, _i64, _p],
    "kronq_biip": [_p, _OPTS, _p, ctypes.c_int, _i64, _i64, _p, _p, _p, _p, _p,
                   _p, _sz, _p],
    "kronq_biip_noalloc": [_p, _OPTS, _p, ctypes.c_int, _i64, _i64, _p, _p, _p,
                           _p, _p, _p],
    "kronq_chol_inv": [_p, _p, _i64, _f, _p, _sz, _p],
    "kronq_quantize_sublayer": [_p, _OPTS, _p, _p, _i64, _i64, _p, _p, _p, _p,
                                _sz, _p],
    "kronq_layer_loss": [_p, _p, _p, _p, _p, _i64, _i64, _p, _p, _sz, _p],
    "kronq_selftest_timeout": [_p, ctypes.c_uint64, _p],
    "kronq_matvec_desc_bytes": [_OPTS, _i64, _i64],
    "kronq_matvec_workspace_bytes": [_i64, _i64, _i64],
    "kronq_matvec_prepare": [_p, _OPTS, _p, _p, _i64, _i64, _p, _sz],
    "kronq_dequant_matvec": [_p, _OPTS, _p, _p, _p, _p, _i64, _i64, _p, _i64, _p, _p, _sz, _p],
    "kronq_chol_split": [_p, _p, _i64, _f, _p, _sz, _p],
    "kronq_chol_split_point": [_i64],
    "kronq_quantize_split": [_p, _OPTS, _p, _p, _i64, _i64, _p, _p, _p, _p, _sz, _p],
    "kronq_gemm_f32": [_p, _i64, _i64, _i64, _f, _p, _i64, ctypes.c_int, _p,
                       _i64, ctypes.c_int, _f, _p, _i64, _p, _sz, _p],
    "kronq_gemm_f32_workspace_bytes": [_i64, _i64, _i64],
    "kronq_linear": [_p, _p, _i64, _i64, _i64, _p, _i64, _i64, _p, ctypes.c_int, _p, _i64, _p,
                     _i64, _p, _i64, _p],
    "kronq_linear_bwd": [_p, _p, _i64, _p, _i64, ctypes.c_int, _p, _i64, _p, _i64, _i64, _i64,
                         _i64, _p, _i64, _p, _p, _i64, _p, _i64, _p, _i64, _p],
    "kronq_gated": [_p, _p, _i64, _i64, _i64, _p, _p, _i64, _i64, ctypes.c_int, _p, _p, _i64, _p,
                    _i64, _p],
    "kronq_gated_bwd": [_p, _p, _i64, _p, _p, _i64, ctypes.c_int, _p, _i64, _p, _p, _i64, _i64,
                        _i64, _i64, _p, _p, _i64, _p, _i64, _p, _i64, _p, _p, _i64, _p],
    "kronq_distill_fwd": [_p, _p, ctypes.c_int, _i64, _i64, _i64, _p, ctypes.c_int, _p, _i64,
                          _i64, _f, _p, _p, _p, _p],
    "kronq_distill_bwd": [_p, _p, ctypes.c_int, _i64, _i64, _i64, _p, ctypes.c_int, _p, _i64,
                          _i64, _f, _p, _p, _p, _i64, _p],
    "kronq_distill_step": [_p, _p, ctypes.c_int, _i64, _i64, _i64, _p, ctypes.c_int, _p, _i64,
                           _i64, _f, _p, _p, _p, _p, _i64, _p],
    "kronq_workspace_bytes": [ctypes.c_int, _i64, _i64, _OPTS],
    "kronq_allocate_bits": [_p, _p, ctypes.c_int, _d, _p],
    "kronq_status_string": [ctypes.c_int],
    "kronq_kernel_launches": [],
    "kronq_last_cuda_error": [],
}
for _name, _args in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = ctypes.c_int
_lib.kronq_workspace_bytes.restype = ctypes.c_size_t
_lib.kronq_matvec_desc_bytes.restype = ctypes.c_size_t
_lib.kronq_matvec_workspace_bytes.restype = ctypes.c_size_t
_lib.kronq_gemm_f32_workspace_bytes.restype = ctypes.c_size_t
_lib.kronq_chol_split_point.restype = ctypes.c_int64
_lib.kronq_status_string.restype = ctypes.c_char_p
_lib.kronq_kernel_launches.restype = ctypes.c_uint64
_lib.kronq_last_cuda_error.restype = ctypes.c_char_p


def _check(fn, st):
    if st != KRONQ_OK:
        raise KronqError(fn, st)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _dtype(t):
    if t.dtype == torch.bfloat16:
        return KRONQ_BF16
    if t.dtype == torch.float32:
        return KRONQ_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


# ---------------------------------------------------------------- entry points
def kronq_accum_cov(A, H, alpha, beta, info, stream=None):
    """H = alpha * AᵀA + beta * H for A (n x d, bf16/fp32, row-major); info is
    a device int32 word (TIMEOUT when a pipeline wait ran out)."""
    n, d = A.shape
    lda = A.stride(0) if n > 1 else d + 7 & -8   # (a single row's stride may be any)
    _check("kronq_accum_cov", _lib.kronq_accum_cov(
        _stream(stream), _ptr(A), _dtype(A), n, d, lda, alpha, beta, _ptr(H), _ptr(info)))


def kronq_sensitivity(H_X, H_G, out, stream=None):
    """out (float64[3], device) = (tr H_X, tr H_G, product)."""
    _check("kronq_sensitivity", _lib.kronq_sensitivity(
        _stream(stream), _ptr(H_X), H_X.shape[0], _ptr(H_G), H_G.shape[0],
        _ptr(out)))


def kronq_workspace_bytes(kind, d_out, d_in, opts=None):
    return int(_lib.kronq_workspace_bytes(
        kind, d_out, d_in, ctypes.byref(opts) if opts is not None else None))


def kronq_biip(opts, W, W_rot, H_X, H_G, s_x, s_g, ws, info, stream=None):
    d_out, d_in = W.shape
    _check("kronq_biip", _lib.kronq_biip(
        _stream(stream), ctypes.byref(opts), _ptr(W), _dtype(W), d_out, d_in,
        _ptr(W_rot), _ptr(H_X), _ptr(H_G), _ptr(s_x), _ptr(s_g), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(info)))


def kronq_biip_noalloc(opts, W, W_rot, H_X, H_G, s_x, s_g, info, stream=None):
    """kronq_biip without a workspace, for callers that cannot allocate device
    memory; the library's own fixed device array serves as scratch (calls
    that overlap on the GPU race on it)."""
    d_out, d_in = W.shape
    _check("kronq_biip_noalloc", _lib.kronq_biip_noalloc(
        _stream(stream), ctypes.byref(opts), _ptr(W), _dtype(W), d_out, d_in,
        _ptr(W_rot), _ptr(H_X), _ptr(H_G), _ptr(s_x), _ptr(s_g), _ptr(info)))


def kronq_chol_inv(H, damp_rel, ws, info, stream=None):
    _check("kronq_chol_inv", _lib.kronq_chol_inv(
        _stream(stream), _ptr(H), H.shape[0], damp_rel, _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(info)))


def kronq_quantize_sublayer(opts, W_rot, U, codes, scales, zeros, ws, info,
                            stream=None):
    d_out, d_in = W_rot.shape
    _check("kronq_quantize_sublayer", _lib.kronq_quantize_sublayer(
        _stream(stream), ctypes.byref(opts), _ptr(W_rot), _ptr(U), d_out, d_in,
        _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(info)))


def kronq_chol_split(H, damp_rel, ws, info, stream=None):
    _check("kronq_chol_split", _lib.kronq_chol_split(
        _stream(stream), _ptr(H), H.shape[0], damp_rel, _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(info)))


def kronq_chol_split_point(d):
    return _lib.kronq_chol_split_point(d)


def kronq_quantize_split(opts, W_rot, F, codes, scales, zeros, ws, info,
                         stream=None):
    d_out, d_in = W_rot.shape
    _check("kronq_quantize_split", _lib.kronq_quantize_split(
        _stream(stream), ctypes.byref(opts), _ptr(W_rot), _ptr(F), d_out, d_in,
        _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(info)))


def kronq_layer_loss(W_ref, W_hat, H_X, H_G, loss, ws, info, stream=None):
    d_out, d_in = W_ref.shape
    _check("kronq_layer_loss", _lib.kronq_layer_loss(
        _stream(stream), _ptr(W_ref), _ptr(W_hat), _ptr(H_X), _ptr(H_G), d_out,
        d_in, _ptr(loss), _ptr(ws), ws.numel() * ws.element_size(), _ptr(info)))


def kronq_matvec_desc_bytes(opts, d_out, d_in):
    return int(_lib.kronq_matvec_desc_bytes(ctypes.byref(opts), d_out, d_in))


def kronq_matvec_workspace_bytes(d_out, d_in, n_tokens):
    return int(_lib.kronq_matvec_workspace_bytes(d_out, d_in, n_tokens))


def kronq_matvec_prepare(opts, s_x, s_g, desc, stream=None):
    """Fills desc (a uint8 CUDA tensor) with the factors of both sides."""
    _check("kronq_matvec_prepare", _lib.kronq_matvec_prepare(
        _stream(stream), ctypes.byref(opts), _ptr(s_x), _ptr(s_g), s_g.numel(),
        s_x.numel(), _ptr(desc), desc.numel()))


def kronq_dequant_matvec(opts, desc, codes, scales, zeros, x, y, ws, info, stream=None):
    """y (n_tokens x d_out) = the quantized sublayer applied to x (n_tokens x d_in)."""
    n_tokens, d_in = x.shape
    d_out = y.shape[1]
    _check("kronq_dequant_matvec", _lib.kronq_dequant_matvec(
        _stream(stream), ctypes.byref(opts), _ptr(desc), _ptr(codes), _ptr(scales),
        _ptr(zeros), d_out, d_in, _ptr(x), n_tokens, _ptr(y), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(info)))


def kronq_selftest_timeout(limit_ns, info, stream=None):
    """Runs the library's bounded device wait on a barrier nothing completes;
    *info becomes KRONQ_ERR_TIMEOUT after about limit_ns (<= 1e9)."""
    _check("kronq_selftest_timeout", _lib.kronq_selftest_timeout(
        _stream(stream), int(limit_ns), _ptr(info)))


def kronq_gemm_f32(A, B, C, info, alpha=1.0, beta=0.0, a_mn=False, b_mn=False,
                   ws=None, stream=None):
    """C = alpha * A Bᵀ + beta * C; A is M x K (or K x M with a_mn), B is
    N x K (or K x N with b_mn); all 2-D fp32 CUDA tensors, rows contiguous.
    ws (a uint8 CUDA tensor) lets large products take the fp16-split path."""
    M, N = C.shape
    K = A.shape[0] if a_mn else A.shape[1]
    _check("kronq_gemm_f32", _lib.kronq_gemm_f32(
        _stream(stream), M, N, K, alpha, _ptr(A), A.stride(0), int(a_mn),
        _ptr(B), B.stride(0), int(b_mn), beta, _ptr(C), C.stride(0),
        None if ws is None else _ptr(ws), 0 if ws is None else ws.numel(),
        _ptr(info)))


def kronq_gemm_f32_workspace_bytes(M, N, K):
    return _lib.kronq_gemm_f32_workspace_bytes(M, N, K)


def kronq_allocate_bits(scores, numel, avg_budget):
    """Host call: greedy 2/3/4-bit allocation (returns a list of ints)."""
    n = len(scores)
    s = (ctypes.c_double * n)(*[float(x) for x in scores])
    m = (ctypes.c_int64 * n)(*[int(x) for x in numel])
    out = (ctypes.c_int * n)()
    _check("kronq_allocate_bits", _lib.kronq_allocate_bits(
        ctypes.cast(s, _p), ctypes.cast(m, _p), n, float(avg_budget),
        ctypes.cast(out, _p)))
    return list(out)


# ---------------------------------------------------------------- calibration pass
# Matrices are 2-D CUDA tensors with contiguous rows (stride(1) == 1); their
# row strides are the library's leading dimensions. All tensors of a call lie
# on one device, which need not be the current one; without ``stream`` the
# call goes to that device's current stream.
def _view(name, t, rows, cols, dev, dtype=torch.bfloat16):
    """(pointer, row stride) of an optional matrix, checked."""
    if t is None:
        return None, cols + 7 & -8
    if t.dtype is dtype and t.shape == (rows, cols) and t.device == dev:
        s0, s1 = t.stride()
        if s1 == 1 or cols <= 1:
            return t.data_ptr(), (s0 if rows > 1 else cols + 7 & -8)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be {rows} x {cols}, not {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not on {dev}")
    raise ValueError(f"{name} must have contiguous rows, not strides {t.stride()}")


def _vector(name, t, n, dev, dtype=torch.float32):
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be {n} contiguous values, not {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not on {dev}")
    return t.data_ptr()


def _info(info, dev):
    if info.dtype is not torch.int32 or info.device != dev or info.numel() < 1:
        raise ValueError(f"info must be an int32 word on {dev}")
    return info.data_ptr()


def _device(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    return t.device


def _enqueue(fn, dev, stream, *args):
    """Calls the library with `dev` current, on `stream` or dev's current one."""
    index = dev.index
    if index != _current_device():
        with torch.cuda.device(dev):
            return _enqueue(fn, dev, stream, *args)
    if stream is None:
        raw = _current_stream(index)
    elif stream.device == dev:
        raw = stream.cuda_stream
    else:
        raise ValueError(f"the stream is on {stream.device}, not on {dev}")
    status = fn(raw, *args)
    if status != KRONQ_OK:
        raise KronqError(fn.__name__, status)


# the current device and the handle of its current stream, without building a
# Stream object per call (a token's call takes less time than that)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)


def kronq_linear(X, W, Y, info, bias=None, act=KRONQ_ACT_NONE, Z=None, R=None, stream=None):
    """Y = act(X Wᵀ + bias) + R for bf16 X (n x d_in), W (d_out x d_in), R and
    Y (n x d_out; R may be Y), fp32 bias (d_out). Z (n x d_out), if given,
    receives the pre-activations. info, an int32 word, is written on failure
    only."""
    dev = _device(X, "X")
    n, d_in = X.shape
    d_out = W.shape[0]
    x, w = _view("X", X, n, d_in, dev), _view("W", W, d_out, d_in, dev)
    z, r = _view("Z", Z, n, d_out, dev), _view("R", R, n, d_out, dev)
    y = _view("Y", Y, n, d_out, dev)
    _enqueue(_lib.kronq_linear, dev, stream, x[0], n, d_in, x[1], w[0], d_out, w[1],
             _vector("bias", bias, d_out, dev), act, z[0], z[1], r[0], r[1], y[0], y[1],
             _info(info, dev))


def kronq_linear_bwd(dY, X, W, info, act=KRONQ_ACT_NONE, Z=None, dZ=None, db=None, dX=None,
                     dXr=None, dW=None, stream=None):
    """dZ = dY * act'(Z) (the sublayer's G), db = sum of dZ's rows (fp32),
    dX = dZ W + dXr, dW = dZᵀ X; each output but dZ is optional, and so are
    dZ and Z with KRONQ_ACT_NONE, X without dW, W without dX (one of X and dX,
    or W, gives d_in)."""
    dev = _device(dY, "dY")
    n, d_out = dY.shape
    d_in = next((t.shape[1] for t in (X, W, dX, dW) if t is not None), None)
    if d_in is None:
        raise ValueError("one of X, W, dX and dW has to give d_in")
    dy, z = _view("dY", dY, n, d_out, dev), _view("Z", Z, n, d_out, dev)
    x, w = _view("X", X, n, d_in, dev), _view("W", W, d_out, d_in, dev)
    dz, dxr = _view("dZ", dZ, n, d_out, dev), _view("dXr", dXr, n, d_in, dev)
    dx, dw = _view("dX", dX, n, d_in, dev), _view("dW", dW, d_out, d_in, dev)
    _enqueue(_lib.kronq_linear_bwd, dev, stream, dy[0], dy[1], z[0], z[1], act, x[0], x[1], w[0],
             w[1], n, d_in, d_out, dz[0], dz[1], _vector("db", db, d_out, dev), dxr[0], dxr[1],
             dx[0], dx[1], dw[0], dw[1], _info(info, dev))


def _pair(name, a, b):
    """The common row stride of two matrices that are given together."""
    if (a[0] is None) != (b[0] is None):
        raise ValueError(f"{name} are given together or not at all")
    if a[1] != b[1]:
        raise ValueError(f"{name} must have the same row stride")
    return a[1]


def kronq_gated(X, Wg, Wu, H, info, act=KRONQ_ACT_SILU, A=None, U=None, stream=None):
    """H = act(X Wgᵀ) * (X Wuᵀ) for bf16 X (n x d), Wg and Wu (f x d, the same
    row stride), H (n x f). A and U (n x f), if given, receive the two products
    for kronq_gated_bwd."""
    dev = _device(X, "X")
    n, d = X.shape
    f = Wg.shape[0]
    x, h = _view("X", X, n, d, dev), _view("H", H, n, f, dev)
    wg, wu = _view("Wg", Wg, f, d, dev), _view("Wu", Wu, f, d, dev)
    a, u = _view("A", A, n, f, dev), _view("U", U, n, f, dev)
    _enqueue(_lib.kronq_gated, dev, stream, x[0], n, d, x[1], wg[0], wu[0], f,
             _pair("Wg and Wu", wg, wu), act, a[0], u[0], _pair("A and U", a, u), h[0], h[1],
             _info(info, dev))


def kronq_gated_bwd(dH, A, U, X, Wg, Wu, Gg, Gu, info, act=KRONQ_ACT_SILU, dX=None, dXr=None,
                    dWg=None, dWu=None, stream=None):
    """Gg = dH * U * act'(A) and Gu = dH * act(A) (the G of gate and up),
    dX = Gg Wg + Gu Wu + dXr, dWg = Ggᵀ X, dWu = Guᵀ X; dX and the weight
    gradients are optional (X may be None without the latter, Wg and Wu
    without dX)."""
    dev = _device(dH, "dH")
    n, f = dH.shape
    d = next((t.shape[1] for t in (X, Wg, dX, dWg) if t is not None), 1)
    dh, a, u = (_view(m, t, n, f, dev) for m, t in (("dH", dH), ("A", A), ("U", U)))
    x, wg, wu = _view("X", X, n, d, dev), _view("Wg", Wg, f, d, dev), _view("Wu", Wu, f, d, dev)
    gg, gu = _view("Gg", Gg, n, f, dev), _view("Gu", Gu, n, f, dev)
    dx, dxr = _view("dX", dX, n, d, dev), _view("dXr", dXr, n, d, dev)
    dwg, dwu = _view("dWg", dWg, f, d, dev), _view("dWu", dWu, f, d, dev)
    _enqueue(_lib.kronq_gated_bwd, dev, stream, dh[0], dh[1], a[0], u[0], _pair("A and U", a, u),
             act, x[0], x[1], wg[0], wu[0], _pair("Wg and Wu", wg, wu), n, d, f, gg[0], gu[0],
             _pair("Gg and Gu", gg, gu), dxr[0], dxr[1], dx[0], dx[1], dwg[0], dwu[0],
             _pair("dWg and dWu", dwg, dwu), _info(info, dev))


def _distill_args(Z, T, idx, tau, weight, dev):
    n, vocab = Z.shape
    k = T.shape[1]
    z, t = _view("Z", Z, n, vocab, dev, Z.dtype), _view("T", T, n, k, dev, T.dtype)
    i = _view("idx", idx, n, k, dev, torch.int32)
    if n > 1 and t[1] != i[1]:
        raise ValueError("T and idx must have the same row stride")
    return (z[0], _dtype(Z), n, vocab, max(z[1], vocab), t[0], _dtype(T), i[0], k, t[1], tau,
            _vector("weight", weight, n, dev))


def kronq_distill_fwd(Z, T, idx, loss, lse, info, tau=1.0, weight=None, stream=None):
    """loss and lse (n fp32 values) of student logits Z (n x vocab, fp32 or
    bf16) against a teacher's top logits T (n x k, fp32 or bf16) at the places
    idx (n x k int32, negative: padding). Rows of weight 0 do not count."""
    dev = _device(Z, "Z")
    n = Z.shape[0]
    _enqueue(_lib.kronq_distill_fwd, dev, stream, *_distill_args(Z, T, idx, tau, weight, dev),
             _vector("loss", loss, n, dev), _vector("lse", lse, n, dev), _info(info, dev))


def kronq_distill_bwd(Z, T, idx, lse, dZ, info, tau=1.0, weight=None, stream=None):
    """dZ (like Z; may be Z) = the gradient of sum(weight * loss), from
    kronq_distill_fwd's lse."""
    dev = _device(Z, "Z")
    n, vocab = Z.shape
    dz = _view("dZ", dZ, n, vocab, dev, Z.dtype)
    _enqueue(_lib.kronq_distill_bwd, dev, stream, *_distill_args(Z, T, idx, tau, weight, dev),
             _vector("lse", lse, n, dev), dz[0], max(dz[1], vocab), _info(info, dev))


def kronq_distill_step(Z, T, idx, loss, lse, dZ, info, tau=1.0, weight=None, stream=None):
    """kronq_distill_fwd and kronq_distill_bwd in one pass over the logits;
    lse may be None."""
    dev = _device(Z, "Z")
    n, vocab = Z.shape
    dz = _view("dZ", dZ, n, vocab, dev, Z.dtype)
    _enqueue(_lib.kronq_distill_step, dev, stream, *_distill_args(Z, T, idx, tau, weight, dev),
             _vector("loss", loss, n, dev), _vector("lse", lse, n, dev), dz[0],
             max(dz[1], vocab), _info(info, dev))


def kronq_status_string(status):
    return _lib.kronq_status_string(status).decode()


def kronq_kernel_launches():
    """Kernels this process has launched through the library so far."""
    return int(_lib.kronq_kernel_launches())


def exported_symbols():
    """Names of the C entry points this binding wraps."""
    return list(_SIGS)
