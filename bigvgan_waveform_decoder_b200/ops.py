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


def _require(ok, what, detail, status=INVALID):
    if not ok:
        raise MH3AError(status, what, detail)


class _Launch:
    """The device and stream of a call.  Inside the block the device is current and torch allocates
    on the call's stream; tensors that cross between that stream and the caller's are recorded."""

    def __init__(self, device, stream):
        self.device = device
        self.guard = None if device.index == torch.cuda.current_device() else torch.cuda.device(device)
        self.current = torch.cuda.current_stream(device)
        if stream is None:
            stream = self.current
        elif not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(stream, device=device)
        self.stream = stream
        self.ptr = stream.cuda_stream
        self.side = None if self.ptr == self.current.cuda_stream else torch.cuda.stream(stream)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        if self.side is not None:
            self.side.__enter__()
        return self

    def __exit__(self, *exc):
        if self.side is not None:
            self.side.__exit__(*exc)
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def crossing(self, inputs, outputs):
        if self.side is not None:
            for t in inputs:
                if t is not None:
                    t.record_stream(self.stream)
            for t in outputs:
                if t is not None:
                    t.record_stream(self.current)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _same_device(what, device, **tensors):
    for name, t in tensors.items():
        _require(t is None or (isinstance(t, torch.Tensor) and t.device == device), what, f"{name} is not on {device}")


def _frames(what, name, x):
    _require(isinstance(x, torch.Tensor) and x.is_cuda, what, f"{name} is not a CUDA tensor")
    _require(x.dim() == 3, what, f"{name} is not [B, T, C]", SHAPE)
    _require(x.dtype in DTYPES, what, f"{name} has type {x.dtype}")
    _require(x.shape[2] <= 1 or x.stride(2) == 1, what, f"the channels of {name} are not adjacent")
    _require(min(x.shape) >= 1, what, f"{name} is empty", SHAPE)


def _norm_args(what, x, groups, weight, bias, act, alpha, beta, eps, lengths):
    _frames(what, "x", x)
    B, T, Cn = x.shape
    _require(max(x.shape) < 1 << 31, what, "a size of x passes 2^31", SHAPE)
    _require(act in ACTS, what, f"unknown activation {act!r}")
    _require((act == "snake_beta") == (alpha is not None) == (beta is not None), what,
             "alpha and beta belong to snake_beta, and it needs both")
    for name, t in (("weight", weight), ("bias", bias), ("alpha", alpha), ("beta", beta)):
        if t is not None:
            _require(isinstance(t, torch.Tensor) and t.device == x.device and t.dtype == torch.float32 and t.is_contiguous(),
                     what, f"{name} is not a contiguous float32 tensor on {x.device}")
            _require(t.shape == (Cn,), what, f"{name} is not [{Cn}]", SHAPE)
    if lengths is not None:
        _require(isinstance(lengths, torch.Tensor) and lengths.device == x.device and lengths.dtype == torch.int32 and
                 lengths.is_contiguous(), what, f"lengths is not a contiguous int32 tensor on {x.device}")
        _require(lengths.shape == (B,), what, f"lengths is not [{B}]", SHAPE)
    _require(isinstance(groups, int) and groups >= 1 and Cn % groups == 0, what, f"{groups} groups do not divide {Cn} channels", SHAPE)
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
        _same_device(what, x.device, out=out)
        _require(out.dtype == x.dtype and out.is_contiguous(), what, "out is not contiguous or not of x's type")
        _require(out.shape == x.shape, what, "out is not of x's shape", SHAPE)
    L = _load()
    with _Launch(x.device, stream) as on:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device) if out is None else out
        stats = torch.empty((2, p.B, groups), dtype=torch.float32, device=x.device)
        mean, rstd = stats[0], stats[1]
        n = L.mh3a_group_norm_act_workspace(C.byref(p), 0)
        ws = torch.empty(n, dtype=torch.uint8, device=x.device)
        _check(L.mh3a_group_norm_act(C.byref(p), x.data_ptr(), x.stride(0), x.stride(1), y.data_ptr(), mean.data_ptr(),
                                     rstd.data_ptr(), ws.data_ptr(), n, on.ptr), what)
        on.crossing((x, weight, bias, alpha, beta, lengths, out), (y if out is None else None, mean, rstd))
    return y, mean, rstd


def group_norm_act_backward(dy, x, mean, rstd, groups, weight=None, bias=None, act="none", alpha=None, beta=None,
                            lengths=None, stream=None):
    """Gradients of group_norm_act (mh3a_group_norm_act_backward) at x for the output gradient dy, both
    [B, T, C] of one type; mean and rstd from the forward pass, the rest as there.  Returns
    (dx, dweight, dbias, dalpha, dbeta): dx like x and contiguous, the others float32 [C], None for a
    parameter that is None."""
    what = "mh3a_group_norm_act_backward"
    p = _norm_args(what, x, groups, weight, bias, act, alpha, beta, 0.0, lengths)
    _frames(what, "dy", dy)
    _require(dy.device == x.device and dy.dtype == x.dtype, what, "dy is not of x's type and device")
    _require(dy.shape == x.shape, what, "dy is not of x's shape", SHAPE)
    for name, t in (("mean", mean), ("rstd", rstd)):
        _require(isinstance(t, torch.Tensor) and t.device == x.device and t.dtype == torch.float32 and t.is_contiguous(), what,
                 f"{name} is not a contiguous float32 tensor on {x.device}")
        _require(t.shape == (p.B, groups), what, f"{name} is not [{p.B}, {groups}]", SHAPE)
    L = _load()
    with _Launch(x.device, stream) as on:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        grads = torch.empty((4, p.C), dtype=torch.float32, device=x.device)
        dw, db, da, de = (None if t is None else grads[k] for k, t in enumerate((weight, bias, alpha, beta)))
        n = L.mh3a_group_norm_act_workspace(C.byref(p), 1)
        ws = torch.empty(n, dtype=torch.uint8, device=x.device)
        _check(L.mh3a_group_norm_act_backward(C.byref(p), x.data_ptr(), x.stride(0), x.stride(1), dy.data_ptr(),
                                              dy.stride(0), dy.stride(1), mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(),
                                              _ptr(dw), _ptr(db), _ptr(da), _ptr(de), ws.data_ptr(), n, on.ptr), what)
        on.crossing((dy, x, mean, rstd, weight, bias, alpha, beta, lengths), (dx, grads))
    return dx, dw, db, da, de
