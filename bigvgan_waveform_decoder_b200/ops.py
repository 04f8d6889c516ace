"""Operators over channels-last frames, for torch tensors.

``group_norm_act`` / ``group_norm_act_backward``: group norm with an activation and its gradient.
``fp8_quantize`` / ``fp8_matmul`` / ``fp8_linear``: matrices in 8-bit floating point with one scale for each
block of 128 values, their product, and the linear layer (a pointwise convolution) built of both.

The kernels are libmh3a.so's (C ABI in include/mh3a.h); ``_ops.so`` checks the arguments and allocates the
results and the scratch memory.  Tensors are CUDA tensors of one device; a call runs on that device, on
``stream`` (a torch stream or a cudaStream_t; the device's current stream when None).  Results and
scratch are allocated on that stream; ordering the caller's own tensors with it stays the caller's
business, as everywhere in CUDA, but tensors that are still in use there are kept from the allocator
until the call is done.  Bad arguments raise ``MH3AError`` before anything is launched.  The calls
record no gradient: it is a call of its own, for a ``torch.autograd.Function`` to make.  Where autograd is
recording and an input requires a gradient, the results lead back to a node that raises when a backward pass
reaches it, and ``out`` is refused; under ``torch.no_grad()`` or with detached inputs nothing is recorded.
"""
from __future__ import annotations

import torch

from .binding import load

load()  # libmh3a.so, with its own message where it is missing
try:
    from . import _ops
except ImportError as e:  # no fallback
    raise RuntimeError("operators not built: _ops.so is missing or was built for another torch "
                       f"(run python -m bigvgan_waveform_decoder_b200.build): {e}") from e


def _stream(stream):
    return getattr(stream, "cuda_stream", stream)


def group_norm_act(x, groups, weight=None, bias=None, act="none", alpha=None, beta=None, eps=1e-5, lengths=None,
                   out=None, stream=None):
    """Group norm with an activation over channels-last frames (mh3a_group_norm_act).

    x: [B, T, C] float32, float16 or bfloat16, channels adjacent, any other strides; ``groups`` divides
    C.  weight, bias: float32 [C] or None.  act: "none", "silu" or "snake_beta", the last with float32
    alpha and beta [C].  lengths: int32 [B], the valid rows of each item; rows behind them are not read
    and are zeros in y.  Returns (y, mean, rstd): y like x and contiguous (``out`` if given, which must
    not overlap an input), mean and rstd float32 [B, groups], which group_norm_act_backward takes."""
    return _ops.group_norm_act(x, groups, weight, bias, act, alpha, beta, eps, lengths, out, _stream(stream))


def group_norm_act_backward(dy, x, mean, rstd, groups, weight=None, bias=None, act="none", alpha=None, beta=None,
                            lengths=None, stream=None):
    """Gradients of group_norm_act (mh3a_group_norm_act_backward) at x for the output gradient dy, both
    [B, T, C] of one type; mean and rstd from the forward pass, the rest as there.  Returns
    (dx, dweight, dbias, dalpha, dbeta): dx like x and contiguous, the others float32 [C], None for a
    parameter that is None."""
    return _ops.group_norm_act_backward(dy, x, mean, rstd, groups, weight, bias, act, alpha, beta, lengths,
                                        _stream(stream))


def fp8_quantize(x, block_rows=1, transpose=False, stream=None):
    """x [rows, cols] (float32, float16 or bfloat16, columns adjacent) in fp8 with one scale for each block of
    128 columns and ``block_rows`` rows, 1 (activations, gradients) or 128 (weights); mh3a_fp8_quantize.
    With ``transpose`` the matrix that is blocked and returned is x transposed.  Returns (q, scale): q
    float8_e4m3fn, its rows on 16-byte boundaries, scale float32 [ceil(inner / 128), ceil(outer /
    block_rows)]; an element stands for q times its block's scale."""
    return _ops.fp8_quantize(x, block_rows, transpose, _stream(stream))


def fp8_matmul(a, a_scale, b, b_scale, out_dtype=torch.bfloat16, bias=None, out=None, stream=None):
    """a [M, K] times b [N, K] transposed, plus bias [N] (float32), for fp8 matrices as fp8_quantize returns
    them: a with block_rows 1, b with 1 or 128 (mh3a_fp8_matmul).  Sums are fp32, rounded once to
    ``out_dtype``.  Returns [M, N] (``out`` if given, which must not overlap an input)."""
    return _ops.fp8_matmul(a, a_scale, b, b_scale, out_dtype, bias, out, _stream(stream))


def fp8_linear(x, w, w_scale, bias=None, out=None, stream=None):
    """x [M, K] times w [N, K] transposed, plus bias: x (float32, float16 or bfloat16) is quantised with
    block_rows 1, w and w_scale come from fp8_quantize (mh3a_fp8_linear).  For channels-last frames
    [B, T, C] pass x.view(B * T, C).  Returns [M, N] of x's type (``out`` if given, which must not overlap
    an input)."""
    return _ops.fp8_linear(x, w, w_scale, bias, out, _stream(stream))
