"""Operators over channels-last frames on the C ABI of include/mh3a.h (argument marshalling only).

``group_norm_act`` / ``group_norm_act_backward``: group norm with an activation and its gradient.
``fp8_quantize`` / ``fp8_matmul`` / ``fp8_linear``: matrices in 8-bit floating point with one scale for each
block of 128 values, their product, and the linear layer (a pointwise convolution) built of both.

Tensors are CUDA tensors of one device; calls run on that device, on ``stream`` (a torch stream or a
cudaStream_t; the device's current stream when None).  Results and scratch are allocated on that
stream; ordering the caller's own tensors with it stays the caller's business, as everywhere in
CUDA, but tensors that are still in use there are kept from the allocator until the call is done.
Bad arguments raise ``MH3AError`` before anything is launched.
"""
from __future__ import annotations

import ctypes as C

import torch

from .binding import MH3AError, _check, load

DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
ACTS = {"none": 0, "silu": 1, "snake_beta": 2}
INVALID, SHAPE = 1, 3


class mh3a_norm(C.Structure):
    _fields_ = [("dtype", C.c_int), ("act", C.c_int), ("B", C.c_int), ("T", C.c_int), ("C", C.c_int),
                ("groups", C.c_int), ("eps", C.c_float), ("weight", C.c_void_p), ("bias", C.c_void_p),
                ("alpha", C.c_void_p), ("beta", C.c_void_p), ("lengths", C.c_void_p)]


_lib = None


def _load():
    global _lib
    if _lib is None:
        L = load()
        vp, ll, i, sz = C.c_void_p, C.c_longlong, C.c_int, C.c_size_t
        norm = C.POINTER(mh3a_norm)
        L.mh3a_group_norm_act_workspace.argtypes = [norm, i]
        L.mh3a_group_norm_act_workspace.restype = sz
        L.mh3a_group_norm_act.argtypes = [norm, vp, ll, ll, vp, vp, vp, vp, sz, vp]
        L.mh3a_group_norm_act.restype = i
        L.mh3a_group_norm_act_backward.argtypes = [norm, vp, ll, ll, vp, ll, ll, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.mh3a_group_norm_act_backward.restype = i
        L.mh3a_fp8_quantize.argtypes = [vp, i, i, i, ll, i, i, vp, ll, vp, vp]
        L.mh3a_fp8_quantize.restype = i
        L.mh3a_fp8_matmul.argtypes = [vp, ll, vp, vp, ll, vp, i, i, i, i, vp, i, vp, ll, vp]
        L.mh3a_fp8_matmul.restype = i
        L.mh3a_fp8_linear_workspace.argtypes = [i, i]
        L.mh3a_fp8_linear_workspace.restype = sz
        L.mh3a_fp8_linear.argtypes = [vp, i, ll, vp, ll, vp, i, i, i, i, vp, vp, ll, vp, sz, vp]
        L.mh3a_fp8_linear.restype = i
        _lib = L
    return _lib


def _bad(what, detail, status=INVALID):
    return MH3AError(status, what, detail)


_raw_stream = torch._C._cuda_getCurrentRawStream


def _launch(device, stream, call, inputs):
    """call(cudaStream_t) -> outputs, with the device current and torch allocating on the call's stream.
    Tensors that cross between that stream and the caller's are recorded with the allocator."""
    if stream is None and device.index == torch.cuda.current_device():
        return call(_raw_stream(device.index))
    with torch.cuda.device(device):
        current = torch.cuda.current_stream()
        if stream is None:
            stream = current
        elif not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(stream, device=device)
        if stream.cuda_stream == current.cuda_stream:
            return call(current.cuda_stream)
        with torch.cuda.stream(stream):
            outputs = call(stream.cuda_stream)
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
        for t in outputs:
            if t is not None:
                t.record_stream(current)
        return outputs


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_frames(what, name, x):
    if not (isinstance(x, torch.Tensor) and x.is_cuda):
        raise _bad(what, f"{name} is not a CUDA tensor")
    if x.dim() != 3:
        raise _bad(what, f"{name} is not [B, T, C]", SHAPE)
    if x.dtype not in DTYPES:
        raise _bad(what, f"{name} has type {x.dtype}")
    B, T, Cn = x.shape
    if not (1 <= B < 1 << 31 and 1 <= T < 1 << 31 and 1 <= Cn < 1 << 31):
        raise _bad(what, f"{name} is empty, or a size passes 2^31", SHAPE)
    if Cn > 1 and x.stride(2) != 1:
        raise _bad(what, f"the channels of {name} are not adjacent")
    return B, T, Cn


def _check_plain(what, name, t, device, dtype, shape):
    """A contiguous tensor of a type and shape on the call's device."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == device and t.is_contiguous()):
        raise _bad(what, f"{name} is not a contiguous {dtype} tensor on {device}")
    if t.shape != shape:
        raise _bad(what, f"{name} is not of shape {list(shape)}", SHAPE)


def _norm_args(what, x, groups, weight, bias, act, alpha, beta, eps, lengths):
    B, T, Cn = _check_frames(what, "x", x)
    if act not in ACTS:
        raise _bad(what, f"unknown activation {act!r}")
    if not (act == "snake_beta") == (alpha is not None) == (beta is not None):
        raise _bad(what, "alpha and beta belong to snake_beta, and it needs both")
    device, shape = x.device, (Cn,)
    if weight is not None:
        _check_plain(what, "weight", weight, device, torch.float32, shape)
    if bias is not None:
        _check_plain(what, "bias", bias, device, torch.float32, shape)
    if alpha is not None:
        _check_plain(what, "alpha", alpha, device, torch.float32, shape)
        _check_plain(what, "beta", beta, device, torch.float32, shape)
    if lengths is not None:
        _check_plain(what, "lengths", lengths, device, torch.int32, (B,))
    if not (isinstance(groups, int) and groups >= 1 and Cn % groups == 0):
        raise _bad(what, f"{groups} groups do not divide {Cn} channels", SHAPE)
    return mh3a_norm(DTYPES[x.dtype], ACTS[act], B, T, Cn, groups, eps, _ptr(weight), _ptr(bias), _ptr(alpha), _ptr(beta),
                     _ptr(lengths))


def group_norm_act(x, groups, weight=None, bias=None, act="none", alpha=None, beta=None, eps=1e-5, lengths=None,
                   out=None, stream=None):
    """Group norm with an activation over channels-last frames (mh3a_group_norm_act).

    x: [B, T, C] float32, float16 or bfloat16, channels adjacent, any other strides; ``groups`` divides
    C.  weight, bias: float32 [C] or None.  act: "none", "silu" or "snake_beta", the last with float32
    alpha and beta [C].  lengths: int32 [B], the valid rows of each item; rows behind them are not read
    and are zeros in y.  Returns (y, mean, rstd): y like x and contiguous (``out`` if given, which must
    not overlap x), mean and rstd float32 [B, groups], which group_norm_act_backward takes."""
    what = "mh3a_group_norm_act"
    p = _norm_args(what, x, groups, weight, bias, act, alpha, beta, eps, lengths)
    if out is not None:
        _check_plain(what, "out", out, x.device, x.dtype, x.shape)
    L = _load()

    def call(stream):
        y = x.new_empty(x.shape) if out is None else out
        mean = x.new_empty((p.B, groups), dtype=torch.float32)
        rstd = x.new_empty((p.B, groups), dtype=torch.float32)
        n = L.mh3a_group_norm_act_workspace(p, 0)
        ws = x.new_empty(n, dtype=torch.uint8)
        st = L.mh3a_group_norm_act(p, x.data_ptr(), x.stride(0), x.stride(1), y.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                   ws.data_ptr(), n, stream)
        if st:
            _check(st, what)
        return y, mean, rstd

    return _launch(x.device, stream, call, (x, weight, bias, alpha, beta, lengths, out))


def group_norm_act_backward(dy, x, mean, rstd, groups, weight=None, bias=None, act="none", alpha=None, beta=None,
                            lengths=None, stream=None):
    """Gradients of group_norm_act (mh3a_group_norm_act_backward) at x for the output gradient dy, both
    [B, T, C] of one type; mean and rstd from the forward pass, the rest as there.  Returns
    (dx, dweight, dbias, dalpha, dbeta): dx like x and contiguous, the others float32 [C], None for a
    parameter that is None."""
    what = "mh3a_group_norm_act_backward"
    p = _norm_args(what, x, groups, weight, bias, act, alpha, beta, 0.0, lengths)
    _check_frames(what, "dy", dy)
    if dy.device != x.device or dy.dtype != x.dtype:
        raise _bad(what, "dy is not of x's type and device")
    if dy.shape != x.shape:
        raise _bad(what, "dy is not of x's shape", SHAPE)
    _check_plain(what, "mean", mean, x.device, torch.float32, (p.B, groups))
    _check_plain(what, "rstd", rstd, x.device, torch.float32, (p.B, groups))
    L = _load()

    def call(stream):
        dx = x.new_empty(x.shape)
        dw, db, da, de = (None if t is None else torch.empty_like(t) for t in (weight, bias, alpha, beta))
        n = L.mh3a_group_norm_act_workspace(p, 1)
        ws = x.new_empty(n, dtype=torch.uint8)
        st = L.mh3a_group_norm_act_backward(p, x.data_ptr(), x.stride(0), x.stride(1), dy.data_ptr(), dy.stride(0),
                                            dy.stride(1), mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), _ptr(dw), _ptr(db),
                                            _ptr(da), _ptr(de), ws.data_ptr(), n, stream)
        if st:
            _check(st, what)
        return dx, dw, db, da, de

    return _launch(x.device, stream, call, (dy, x, mean, rstd, weight, bias, alpha, beta, lengths))


FP8 = torch.float8_e4m3fn
BLOCK = 128


def _check_matrix(what, name, x, types):
    if not (isinstance(x, torch.Tensor) and x.is_cuda):
        raise _bad(what, f"{name} is not a CUDA tensor")
    if x.dtype not in types:
        raise _bad(what, f"{name} has type {x.dtype}")
    if x.dim() != 2:
        raise _bad(what, f"{name} is not a matrix", SHAPE)
    rows, cols = x.shape
    if not (1 <= rows < 1 << 31 and 1 <= cols < 1 << 31):
        raise _bad(what, f"{name} is empty, or a size passes 2^31", SHAPE)
    if cols > 1 and x.stride(1) != 1:
        raise _bad(what, f"the columns of {name} are not adjacent")
    return rows, cols


def _check_stored(what, name, q, scale):
    """An fp8 matrix and its scales: (rows, cols, row stride in bytes, block rows)."""
    rows, cols = _check_matrix(what, name, q, (FP8,))
    stride = q.stride(0) if rows > 1 else (cols + 15) // 16 * 16
    if stride < cols or stride % 16 or q.data_ptr() % 16:
        raise _bad(what, f"the rows of {name} do not start on 16-byte boundaries")
    if not (isinstance(scale, torch.Tensor) and scale.dtype == torch.float32 and scale.device == q.device and scale.is_contiguous()):
        raise _bad(what, f"the scales of {name} are not a contiguous float32 tensor on {q.device}")
    kb = -(-cols // BLOCK)
    if scale.shape == (kb, rows):
        return rows, cols, stride, 1
    if scale.shape == (kb, -(-rows // BLOCK)):
        return rows, cols, stride, BLOCK
    raise _bad(what, f"the scales of {name} are {list(scale.shape)}: [{kb}, {rows}] or [{kb}, {-(-rows // BLOCK)}] are wanted", SHAPE)


def _check_bias_out(what, bias, out, device, shape, dtype):
    if bias is not None:
        _check_plain(what, "bias", bias, device, torch.float32, shape[1:])
    if out is not None:
        if not (isinstance(out, torch.Tensor) and out.dtype == dtype and out.device == device):
            raise _bad(what, f"out is not a {dtype} tensor on {device}")
        if out.shape != shape:
            raise _bad(what, f"out is not {list(shape)}", SHAPE)
        if (shape[1] > 1 and out.stride(1) != 1) or (shape[0] > 1 and out.stride(0) < shape[1]):
            raise _bad(what, "the columns of out are not adjacent, or its rows overlap")


def _row_stride(t, cols):
    return t.stride(0) if t.shape[0] > 1 else cols


def fp8_quantize(x, block_rows=1, transpose=False, stream=None):
    """x [rows, cols] (float32, float16 or bfloat16, columns adjacent) in fp8 with one scale for each block of
    128 columns and ``block_rows`` rows, 1 (activations, gradients) or 128 (weights); mh3a_fp8_quantize.
    With ``transpose`` the matrix that is blocked and returned is x transposed.  Returns (q, scale): q
    float8_e4m3fn, its rows on 16-byte boundaries, scale float32 [ceil(inner / 128), ceil(outer /
    block_rows)]; an element stands for q times its block's scale."""
    what = "mh3a_fp8_quantize"
    rows, cols = _check_matrix(what, "x", x, DTYPES)
    if block_rows not in (1, BLOCK):
        raise _bad(what, f"block_rows is {block_rows}: 1 or {BLOCK} are wanted")
    outer, inner = (cols, rows) if transpose else (rows, cols)
    L = _load()

    def call(stream):
        ld = (inner + 15) // 16 * 16
        buf = x.new_empty((outer, ld), dtype=FP8)
        scale = x.new_empty((-(-inner // BLOCK), -(-outer // block_rows)), dtype=torch.float32)
        st = L.mh3a_fp8_quantize(x.data_ptr(), DTYPES[x.dtype], rows, cols, _row_stride(x, cols), block_rows,
                                 1 if transpose else 0, buf.data_ptr(), ld, scale.data_ptr(), stream)
        if st:
            _check(st, what)
        return (buf if ld == inner else buf[:, :inner]), scale

    return _launch(x.device, stream, call, (x,))


def fp8_matmul(a, a_scale, b, b_scale, out_dtype=torch.bfloat16, bias=None, out=None, stream=None):
    """a [M, K] times b [N, K] transposed, plus bias [N] (float32), for fp8 matrices as fp8_quantize returns
    them: a with block_rows 1, b with 1 or 128 (mh3a_fp8_matmul).  Sums are fp32, rounded once to
    ``out_dtype``.  Returns [M, N] (``out`` if given)."""
    what = "mh3a_fp8_matmul"
    M, K, a_stride, a_rows = _check_stored(what, "a", a, a_scale)
    N, Kb, b_stride, b_rows = _check_stored(what, "b", b, b_scale)
    if a_rows != 1:
        raise _bad(what, "a has blocks of 128 rows: block_rows 1 is wanted")
    if K != Kb:
        raise _bad(what, f"a has {K} columns and b {Kb}", SHAPE)
    if a.device != b.device:
        raise _bad(what, "a and b are on different devices")
    if out_dtype not in DTYPES:
        raise _bad(what, f"out_dtype is {out_dtype}")
    _check_bias_out(what, bias, out, a.device, (M, N), out_dtype)
    L = _load()

    def call(stream):
        y = a.new_empty((M, N), dtype=out_dtype) if out is None else out
        st = L.mh3a_fp8_matmul(a.data_ptr(), a_stride, a_scale.data_ptr(), b.data_ptr(), b_stride, b_scale.data_ptr(), b_rows,
                               M, N, K, _ptr(bias), DTYPES[out_dtype], y.data_ptr(), _row_stride(y, N), stream)
        if st:
            _check(st, what)
        return (y,)

    return _launch(a.device, stream, call, (a, a_scale, b, b_scale, bias, out))[0]


def fp8_linear(x, w, w_scale, bias=None, out=None, stream=None):
    """x [M, K] times w [N, K] transposed, plus bias: x (float32, float16 or bfloat16) is quantised with
    block_rows 1, w and w_scale come from fp8_quantize (mh3a_fp8_linear).  For channels-last frames
    [B, T, C] pass x.view(B * T, C).  Returns [M, N] of x's type (``out`` if given)."""
    what = "mh3a_fp8_linear"
    M, K = _check_matrix(what, "x", x, DTYPES)
    N, Kw, w_stride, w_rows = _check_stored(what, "w", w, w_scale)
    if K != Kw:
        raise _bad(what, f"x has {K} columns and w {Kw}", SHAPE)
    if x.device != w.device:
        raise _bad(what, "x and w are on different devices")
    _check_bias_out(what, bias, out, x.device, (M, N), x.dtype)
    L = _load()

    def call(stream):
        y = x.new_empty((M, N)) if out is None else out
        n = L.mh3a_fp8_linear_workspace(M, K)
        ws = x.new_empty(n, dtype=torch.uint8) if n else None
        st = L.mh3a_fp8_linear(x.data_ptr(), DTYPES[x.dtype], _row_stride(x, K), w.data_ptr(), w_stride, w_scale.data_ptr(),
                               w_rows, M, N, K, _ptr(bias), y.data_ptr(), _row_stride(y, N), _ptr(ws), n, stream)
        if st:
            _check(st, what)
        return (y,)

    return _launch(x.device, stream, call, (x, w, w_scale, bias, out))[0]
