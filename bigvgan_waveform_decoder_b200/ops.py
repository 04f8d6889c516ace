"""Operators over channels-last frames on the C ABI of include/mh3a.h (argument marshalling only).

``group_norm_act`` / ``group_norm_act_backward``: group norm with an activation and its gradient.

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
