"""Group norm with an activation over channels-last frames, against its formulas in 64 bits."""
import ctypes as C
import random
import time

import pytest
import torch

import bigvgan_waveform_decoder_b200 as pkg
from bigvgan_waveform_decoder_b200 import binding as Bd

from . import ops_ref as R

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("none", "silu", "snake_beta")


def case(B, T, Cn, act, dtype, seed, offset=1.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, T, Cn, generator=g) * (0.3 + 2 * torch.rand(Cn, generator=g)) + offset * torch.randn(Cn, generator=g)
    w, b = 1 + 0.3 * torch.randn(Cn, generator=g), 0.3 * torch.randn(Cn, generator=g)
    al, be = 0.7 + 0.6 * torch.rand(Cn, generator=g), 0.7 + 0.6 * torch.rand(Cn, generator=g)
    if act != "snake_beta":
        al = be = None
    return [None if t is None else t.to(device) for t in (x.to(TYPES[dtype]), w, b, al, be)]


def check_forward(x, groups, w, b, act, al, be, eps=1e-5, lengths=None, got=None, **kw):
    y, mean, rstd = got or pkg.group_norm_act(x, groups, w, b, act=act, alpha=al, beta=be, eps=eps, lengths=lengths, **kw)
    ry, rm, rr, mag = R.norm_forward(x, groups, w, b, act, al, be, eps, lengths)
    assert y.shape == x.shape and y.dtype == x.dtype and y.is_contiguous()
    # mean: rounded partial means put together in fp64; errors are relative to the values' size.  A batch
    # of 8 and at most a few merges in 32 bits: under 16 roundings.
    dev = 1 / rr
    assert torch.all((mean.double() - rm).abs() <= 16 * R.F24 * (rm.abs() + 4 * dev))
    # var: sums of squares of at most the same depth, two roundings a term more; rstd takes half of
    # the variance's relative error; the shift of the mean enters squared.
    assert torch.all((rstd.double() / rr - 1).abs() <= 32 * R.F24 * (1 + (R.F24 * rm.abs() / dev) ** 2))
    # y: u carries the errors of mean and rstd and three roundings, at most 64 half units of its parts;
    # the activation's slope is below 1 + alpha / beta < 3 and its own error below 2^-19 for the 16-bit
    # hardware sine and exponential (sin^2 / beta, 2 x 2^-21 / 0.7; sigmoid times u), 2^-22 otherwise
    own = 2.0 ** -19 if x.dtype != torch.float32 else 2.0 ** -22
    tol = torch.finfo(x.dtype).eps / 2 * ry.abs() + 3 * 64 * R.F24 * mag + own * (1 + mag) * (act != "none")
    tol = tol + torch.finfo(x.dtype).smallest_normal  # results below the normal range
    bad = (y.double() - ry).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((y.double() - ry).abs() / tol).max()))
    return y, mean, rstd


def check_backward(dy, x, mean, rstd, groups, w, b, act, al, be, lengths=None, got=None, **kw):
    got = got or pkg.group_norm_act_backward(dy, x, mean, rstd, groups, w, b, act=act, alpha=al, beta=be, lengths=lengths, **kw)
    ref, mag = R.norm_backward(dy, x, groups, w, b, act, al, be, mean, rstd, lengths)
    assert got[0].shape == x.shape and got[0].dtype == x.dtype and got[0].is_contiguous()
    # Every term has a few roundings and the activation's own error (2^-18 of the size of its parts for
    # 16-bit tensors, 2^-21 for fp32: two factors of sin and cos, or u times two of the sigmoid, and u's
    # own error times the slope's slope); a sum adds at most the depth of its longest chain, under 128
    # values in 32 bits before the chunks are put together, of its terms' magnitudes.
    own = 2.0 ** -18 if x.dtype != torch.float32 else 2.0 ** -21
    d = torch.finfo(x.dtype).eps / 2 * ref["dx"].abs() + (own + 128 * R.F24) * mag["dx"] + torch.finfo(x.dtype).smallest_normal
    bad = (got[0].double() - ref["dx"]).abs() > d
    assert not bad.any(), (int(bad.sum()), float(((got[0].double() - ref["dx"]).abs() / d).max()))
    for k, (name, p) in enumerate((("dweight", w), ("dbias", b), ("dalpha", al), ("dbeta", be)), 1):
        if p is None:
            assert got[k] is None
            continue
        base = mag[name] + mag["dbias"] + mag["dweight"]  # the activation's error scales with dy and u
        off = (got[k].double() - ref[name]).abs()
        assert torch.all(off <= (own + 128 * R.F24) * base), (name, float((off / base).max()))
    return got


SHAPES = [
    # B, T, C, groups
    (1, 1, 8, 1),         # one frame, one group
    (1, 1, 512, 512),     # every value is a group of its own: var 0
    (2, 4, 512, 32),      # a few frames
    (3, 37, 24, 3),
    (1, 5, 2048, 32),
    (2, 33, 25, 5),       # odd width: no vector access
    (1, 300, 7, 7),
    (2, 90, 174, 3),      # even: pairs
    (2, 6000, 30, 2),
    (2, 500, 200, 8),     # groups that end inside a vector
    (2, 130, 12, 4),      # 16-bit rows that are no multiple of 16 bytes
    (2, 2000, 512, 32),
    (3, 4097, 64, 4),
    (1, 20011, 8, 2),     # long and narrow
    (1, 70001, 3, 1),
    (5, 777, 96, 1),      # one group: layer-wide statistics
    (1, 3, 4104, 27),     # wider than a block
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward(shape, act, dtype):
    B, T, Cn, G = shape
    x, w, b, al, be = case(B, T, Cn, act, dtype, seed=T + Cn)
    _, mean, rstd = check_forward(x, G, w, b, act, al, be)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(9)).to(x.dtype).cuda()
    check_backward(dy, x, mean, rstd, G, w, b, act, al, be)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(6, 50, 64, 4), (6, 900, 200, 8), (6, 4100, 32, 4), (6, 9, 25, 5), (6, 30000, 16, 2)], ids=str)
def test_ragged_batch(shape, dtype):
    """Rows behind an item's length take no part, whatever they hold, and come out as zeros; lengths of 0
    and 1, and lengths outside [0, T]."""
    B, T, Cn, G = shape
    x, w, b, al, be = case(B, T, Cn, "snake_beta", dtype, seed=5)
    n = torch.tensor([T, 0, 1, T // 2 + 1, -3, T + 7], dtype=torch.int32, device="cuda")
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(9)).to(x.dtype).cuda()
    for i in range(B):
        k = min(max(int(n[i]), 0), T)
        x[i, k:] = float("nan")
        dy[i, k:] = float("inf")
    y, mean, rstd = check_forward(x, G, w, b, "snake_beta", al, be, lengths=n)
    got = check_backward(dy, x, mean, rstd, G, w, b, "snake_beta", al, be, lengths=n)
    for i in range(B):
        k = min(max(int(n[i]), 0), T)
        assert torch.all(y[i, k:] == 0) and torch.all(got[0][i, k:] == 0)
    assert torch.all(mean[[1, 4]] == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("T", (40, 3000, 60000))
def test_strided_and_repeated_rows(T, dtype):
    """Inputs that are slices, transposed batches or repeated items; outputs are contiguous."""
    Cn, G = 32, 4
    x, w, b, al, be = case(1, 3 * T, 2 * Cn, "silu", dtype, seed=2)
    wide = x.view(3, T, 2 * Cn)
    w, b = w[:Cn].contiguous(), b[:Cn].contiguous()
    odd = torch.empty(3, T * Cn + 1, device="cuda", dtype=wide.dtype)  # an item of one row of a strided batch
    odd[:1, :T * Cn] = wide[:1, :, :Cn].reshape(1, -1)
    views = [odd[:1, :T * Cn].unflatten(1, (T, Cn)), wide[:1, :1, :Cn].expand(2, T, Cn), wide[:, :, Cn:], wide.view(T, 3, 2 * Cn).transpose(0, 1)[..., :Cn], wide[:1, :, :Cn].expand(3, T, Cn),
             wide[:, :, 1:Cn + 1]]
    for v in views:
        _, mean, rstd = check_forward(v, G, w, b, "silu", None, None)
        check_backward(v, v.flip(0) if v.stride(0) else v, mean, rstd, G, w, b, "silu", None, None)


@pytest.mark.gpu
@pytest.mark.parametrize("T", (7, 2500, 50000))
def test_far_offset_and_outliers(T):
    """Statistics of values that lie far from zero, or that one value outweighs."""
    Cn, G = 32, 4
    x, w, b, _, _ = case(2, T, Cn, "none", "fp32", seed=3)
    check_forward(x + 1000, G, w, b, "none", None, None)
    x[:, 0] = 3e4
    check_forward(x, G, w, b, "none", None, None)


@pytest.mark.gpu
@pytest.mark.parametrize("T", (7, 2500, 50000))
def test_not_finite_values_stay_in_their_group(T):
    Cn, G = 32, 4
    x, w, b, al, be = case(2, T, Cn, "snake_beta", "bf16", seed=4)
    y0, m0, r0 = pkg.group_norm_act(x, G, w, b, act="snake_beta", alpha=al, beta=be)
    x[0, T // 2, 3] = float("inf")
    x[1, T - 1, 31] = float("nan")
    y, m, r = pkg.group_norm_act(x, G, w, b, act="snake_beta", alpha=al, beta=be)
    hit = torch.zeros(2, G, dtype=torch.bool, device="cuda")
    hit[0, 0] = hit[1, 3] = True
    assert torch.all(torch.isnan(y.view(2, T, G, 8).float()).any(dim=3).all(dim=1) | ~hit)
    keep = ~hit[:, None, :, None].expand(2, T, G, 8)
    assert torch.equal(y.view(2, T, G, 8)[keep], y0.view(2, T, G, 8)[keep])
    assert torch.equal(m[~hit], m0[~hit]) and torch.equal(r[~hit], r0[~hit])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", (5, 1500, 60000))
def test_phases_beyond_the_period(T, dtype):
    """SnakeBeta of huge u: fp32 (and its product with alpha) leaves no fraction of a period, so the sine is
    arbitrary but stays one; y - u is within [0, 1 / beta], the slope within 1 +- alpha / beta."""
    Cn, G = 16, 2
    x, w, b, al, be = case(1, T, Cn, "snake_beta", "fp32", seed=13)
    x, w = x.to(TYPES[dtype]), w.sign() * 10.0 ** torch.linspace(1, 4 if dtype == "fp16" else 14, Cn, device="cuda")
    y, m, r = pkg.group_norm_act(x, G, w, b, act="snake_beta", alpha=al, beta=be)
    u = R.norm_forward(x, G, w, b, "none", None, None, 1e-5, None)[0]
    slack = torch.finfo(y.dtype).eps / 2 * (u.abs() + 2) + 64 * R.F24 * (u.abs() + 10 * w.double().abs())
    d = y.double() - u
    assert torch.all(d >= -slack) and torch.all(d <= 1.001 / be.double() + slack)
    dx, dw, db, da, dbe = pkg.group_norm_act_backward(torch.ones_like(x), x, m, r, G, w, b, act="snake_beta", alpha=al, beta=be)
    for t in (dx.float(), dw, db, da, dbe):
        assert bool(torch.isfinite(t).all()) or dtype == "fp16"
    assert torch.all(db.double().abs() <= 1.01 * T * (1 + al.double() / be.double()))
    assert torch.all((dbe <= 0) & (dbe.double() >= -1.01 * T / be.double() ** 2))


@pytest.mark.gpu
def test_without_parameters_and_with_some():
    x, w, b, al, be = case(2, 60, 48, "snake_beta", "fp32", seed=6)
    dy = torch.randn_like(x)
    for ww, bb in ((None, None), (w, None), (None, b)):
        _, mean, rstd = check_forward(x, 6, ww, bb, "snake_beta", al, be)
        check_backward(dy, x, mean, rstd, 6, ww, bb, "snake_beta", al, be)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", (6, 1100))
def test_gradient_against_differences(act, T):
    """Central differences of sum(y dy) along random directions, in fp32 with the reference's forward in
    64 bits: the analytic gradients have to give the same slopes."""
    G = 4
    x, w, b, al, be = case(2, T, 16, act, "fp32", seed=7)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(1)).cuda()
    _, mean, rstd = pkg.group_norm_act(x, G, w, b, act=act, alpha=al, beta=be)
    got = pkg.group_norm_act_backward(dy, x, mean, rstd, G, w, b, act=act, alpha=al, beta=be)
    params = [x, w, b, al, be]
    for k, (p, grad) in enumerate(zip(params, got)):
        if p is None:
            continue
        d = torch.randn(p.shape, generator=torch.Generator().manual_seed(k)).cuda().double()
        h = 1e-5

        def loss(sign):
            q = [None if t is None else t.double() for t in params]
            q[k] = q[k] + sign * h * d
            return float((R.norm_forward(q[0], G, q[1], q[2], act, q[3], q[4], 1e-5, None)[0] * dy.double()).sum())

        slope = (loss(1) - loss(-1)) / (2 * h)
        have = float((grad.double() * d).sum())
        size = float((grad.double() * d).abs().sum())
        # the difference is off by h^2 times a third derivative of order 10 (1e-9) and by rounding in 64
        # bits (1e-16 x sum |y dy| / h); the gradient by a few 2^-21 of its parts
        assert abs(slope - have) <= 2e-6 * size + 1e-6 * x.numel() ** 0.5, (k, slope, have, size)


@pytest.mark.gpu
def test_repeats_are_identical_and_streams_do_not_mix():
    x, w, b, al, be = case(3, 3001, 64, "snake_beta", "bf16", seed=8)
    x2 = x.flip(0).contiguous()
    dy = torch.randn(x.shape, device="cuda").to(x.dtype)
    kw = dict(act="snake_beta", alpha=al, beta=be)

    def both(x, stream=None):
        y, m, r = pkg.group_norm_act(x, 8, w, b, stream=stream, **kw)
        return (y, m, r) + pkg.group_norm_act_backward(dy, x, m, r, 8, w, b, stream=stream, **kw)

    first, second = both(x), both(x2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    runs = []
    for _ in range(5):
        runs.append((both(x, s1), both(x2, s2.cuda_stream)))
    torch.cuda.synchronize()
    for a, c in runs:
        assert all(torch.equal(p, q) for p, q in zip(a, first))
        assert all(torch.equal(p, q) for p, q in zip(c, second))


@pytest.mark.gpu
@pytest.mark.parametrize("T", (5, 3000))
def test_captured_and_replayed(T):
    x, w, b, al, be = case(2, T, 64, "snake_beta", "fp32", seed=10)
    dy = torch.randn_like(x)
    kw = dict(act="snake_beta", alpha=al, beta=be)
    graphs, outs = [], []
    for k in range(2):  # two graphs with scratch of their own, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y, m, r = pkg.group_norm_act(x, 8, w, b, **kw)
            outs.append((y, m, r) + pkg.group_norm_act_backward(dy, x, m, r, 8, w, b, **kw))
        graphs.append(g)
    x.copy_(x.flip(1).clone() * 1.5)
    for g in (graphs[0], graphs[1], graphs[0]):
        g.replay()
    torch.cuda.synchronize()
    y, m, r = pkg.group_norm_act(x, 8, w, b, **kw)
    ref = (y, m, r) + pkg.group_norm_act_backward(dy, x, m, r, 8, w, b, **kw)
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(o, ref))


@pytest.mark.gpu
def test_writes_nothing_outside_its_outputs():
    """Guard values around y, dx and the statistics stay; a caller's `out` is used."""
    B, T, Cn, G = 2, 301, 24, 3
    x, w, b, _, _ = case(B, T, Cn, "silu", "bf16", seed=11)
    buf = torch.full((x.numel() + 64,), 7.0, device="cuda", dtype=x.dtype)
    out = buf[32:32 + x.numel()].view(B, T, Cn)
    y, m, r = pkg.group_norm_act(x, G, w, b, act="silu", out=out)
    assert y.data_ptr() == out.data_ptr()
    check_forward(x, G, w, b, "silu", None, None, got=(y, m, r))
    assert torch.all(buf[:32] == 7) and torch.all(buf[-32:] == 7)


@pytest.mark.gpu
def test_python_refusals():
    x, w, b, al, be = case(2, 10, 24, "snake_beta", "fp32", seed=12)
    f, n = pkg.group_norm_act, pkg.MH3AError
    for bad in (lambda: f(x, 5, w, b), lambda: f(x, 0, w, b), lambda: f(x, 3, w[:8], b), lambda: f(x, 3, w.cpu(), b),
                lambda: f(x, 3, w.half(), b), lambda: f(x.cpu(), 3, w, b), lambda: f(x.double(), 3, w, b),
                lambda: f(x[0], 3, w, b), lambda: f(x[:, :, ::2], 3), lambda: f(x[:, :0], 3), lambda: f(x, 3, act="gelu"),
                lambda: f(x, 3, act="snake_beta"), lambda: f(x, 3, act="silu", alpha=al, beta=be),
                lambda: f(x, 3, act="snake_beta", alpha=al), lambda: f(x, 3, lengths=torch.tensor([1, 2])),
                lambda: f(x, 3, lengths=torch.tensor([1, 2], device="cuda")),
                lambda: f(x, 3, lengths=torch.tensor([1], device="cuda", dtype=torch.int32)),
                lambda: f(x, 3, out=torch.empty(2, 10, 12, device="cuda")), lambda: f(x, 3, out=x.half())):
        with pytest.raises(n):
            bad()
    y, m, r = f(x, 3)
    g = pkg.group_norm_act_backward
    for bad in (lambda: g(y[:1], x, m, r, 3), lambda: g(y.half(), x, m, r, 3), lambda: g(y, x, m[:1], r, 3),
                lambda: g(y, x, m, r.double(), 3), lambda: g(y, x, m, r, 4)):
        with pytest.raises(n):
            bad()


def norm(**kw):
    p = Bd.mh3a_norm(1, 1, 2, 10, 24, 3, 1e-5, None, None, None, None, None)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def test_abi_refusals():
    """Every refusal comes before any device work (the pointers here are no device memory)."""
    L = Bd.load()
    p0, ok = C.byref(norm()), 1 << 20
    size = L.mh3a_group_norm_act_workspace(p0, 0, 0)
    assert size > 0 and L.mh3a_group_norm_act_workspace(p0, 1, 0) > 0
    assert L.mh3a_group_norm_act_workspace(p0, 0, 1) == 0 and 0 < L.mh3a_group_norm_act_workspace(p0, 1, 1)
    large = C.byref(norm(B=16, T=20000, C=256, groups=32))
    for backward in (0, 1):
        some = L.mh3a_group_norm_act_workspace(large, backward, 1)
        assert 0 < some <= L.mh3a_group_norm_act_workspace(large, backward, 0)

    def fwd(p=None, x=ok + 2, xb=240, xr=24, y=ok, mean=ok, rstd=ok, ws=ok, n=size):
        return L.mh3a_group_norm_act(None if p is None else C.byref(p), x, xb, xr, y, mean, rstd, ws, n, None)

    good = norm()
    assert fwd(None) == 1
    for kw in (dict(x=None), dict(y=None), dict(mean=None), dict(rstd=None), dict(ws=None), dict(n=size - 1), dict(xb=-1),
               dict(xr=-1), dict(x=ok + 1), dict(y=ok + 1), dict(ws=ok + 8), dict(x=ok, xr=25, ws=None)):
        assert fwd(good, **kw) == 1, kw
    for kw in (dict(dtype=3), dict(dtype=-1), dict(act=3), dict(act=-1), dict(act=2), dict(act=2, alpha=ok)):
        assert fwd(norm(**kw)) == 1, kw
        assert L.mh3a_group_norm_act_workspace(C.byref(norm(**kw)), 0, 0) == 0
    for kw in (dict(B=0), dict(T=0), dict(C=0), dict(groups=0), dict(groups=5), dict(T=(1 << 30) + 1),
               dict(B=1 << 20, C=1 << 12, groups=1)):
        assert fwd(norm(**kw)) == 3, kw
    n1 = L.mh3a_group_norm_act_workspace(p0, 1, 0)

    def bwd(p=None, x=ok + 2, dy=ok, mean=ok, rstd=ok, dx=ok, da=None, ws=ok, n=n1, gb=240):
        return L.mh3a_group_norm_act_backward(None if p is None else C.byref(p), x, 240, 24, dy, gb, 24, mean, rstd, dx, ok, ok,
                                              da, None, ws, n, None)

    assert bwd(None) == 1
    for kw in (dict(x=None), dict(dy=None), dict(mean=None), dict(rstd=None), dict(dx=None), dict(da=ok), dict(ws=None),
               dict(n=n1 - 1), dict(gb=-1), dict(dy=ok + 1)):
        assert bwd(good, **kw) == 1, kw
    assert bwd(norm(groups=7)) == 3
    assert L.mh3a_group_norm_act_workspace(None, 0, 0) == 0


def test_tensors_that_are_not_on_a_gpu_are_refused():
    x = torch.zeros(1, 2, 4)
    for bad in (lambda: pkg.group_norm_act(x, 2), lambda: pkg.group_norm_act_backward(x, x, x[0, :, :2], x[0, :, :2], 2),
                lambda: pkg.fp8_quantize(x[0]), lambda: pkg.fp8_linear(x[0], x[0], x[0]), lambda: pkg.fp8_matmul(x[0], x[0], x[0], x[0])):
        with pytest.raises(pkg.MH3AError, match="not a CUDA tensor") as e:
            bad()
        assert e.value.status == 1


def test_exports():
    assert {"mh3a_group_norm_act", "mh3a_group_norm_act_backward", "mh3a_group_norm_act_workspace"} <= set(Bd.EXPORTS)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("shape", [(64, 4, 64, 4), (64, 161, 200, 8), (64, 1034, 200, 8), (64, 50, 25, 5), (2, 60000, 96, 3)], ids=str)
def test_equal_values_far_from_zero(shape, dtype):
    """Every value of an item alike and large: the variance is 0, and rounding must not take it below."""
    B, T, Cn, G = shape
    g = torch.Generator().manual_seed(T)
    x = (10 ** (4 + 6 * torch.rand(B, 1, 1, generator=g)) * torch.randn(B, 1, 1, generator=g).sign()).to(TYPES[dtype])
    x = x.repeat(1, T, Cn).cuda()
    y, mean, rstd = pkg.group_norm_act(x, G, eps=1e-12)
    assert torch.equal(mean, x[:, 0, :1].float().expand(B, G)) and torch.all(y == 0)
    # nothing but eps under the root, or what the squares of half units of the values leave
    assert torch.all(rstd > 0) and torch.all(rstd <= 1e6 * (1 + 4 * R.F24))


def test_planning_takes_no_time_for_any_width():
    """Channels whose count has no small divisor: the search for a slab is bounded."""
    L = Bd.load()
    p = norm(dtype=0, B=1, T=1, C=4 * 5999993, groups=4 * 5999993)
    t0 = time.perf_counter()
    for _ in range(20):
        assert L.mh3a_group_norm_act_workspace(C.byref(p), 0, 1) > 0
    assert time.perf_counter() - t0 < 0.2


def test_abi_refuses_misaligned_statistics_and_gradients():
    L, ok = Bd.load(), 1 << 20
    p = norm(act=2, alpha=ok, beta=ok)
    n = L.mh3a_group_norm_act_workspace(C.byref(p), 1, 0)
    for bad in range(6):
        f = [ok + 2 * (i == bad) for i in range(6)]
        assert L.mh3a_group_norm_act_backward(C.byref(p), ok, 240, 24, ok, 240, 24, f[0], f[1], ok, *f[2:], ok, n, None) == 1


@pytest.mark.gpu
def test_an_output_over_its_input_is_refused():
    x = torch.randn(3, 5, 64, device="cuda")
    buf = torch.zeros(2 * x.numel() + 32, device="cuda")
    part = buf[16:16 + x.numel()].view(x.shape)
    for bad in (lambda: pkg.group_norm_act(x, 4, out=x), lambda: pkg.group_norm_act(part, 4, out=buf[:x.numel()].view(x.shape))):
        with pytest.raises(pkg.MH3AError, match="overlaps") as e:
            bad()
        assert e.value.status == 1
    out = buf[x.numel() + 16:]
    with pytest.raises(pkg.MH3AError):
        pkg.group_norm_act(x, 4, out=out)
    y, *_ = pkg.group_norm_act(part, 4, out=buf[-x.numel():].view(x.shape))  # side by side in one storage
    assert torch.all(y == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", (9, 40000))
def test_parameters_off_16_bytes(T, dtype):
    x, *params = case(2, T, 64, "snake_beta", dtype, seed=T)
    params = [torch.cat((p[:1], p))[1:] for p in params]
    assert all(p.data_ptr() % 16 for p in params)
    w, b, al, be = params
    _, mean, rstd = check_forward(x, 4, w, b, "snake_beta", al, be)
    check_backward(torch.flip(x, (1,)), x, mean, rstd, 4, w, b, "snake_beta", al, be)


@pytest.mark.gpu
@pytest.mark.parametrize("T", (8, 1024))
def test_offsets_beyond_32_bits(T):
    """Items whose elements lie more than 2^31 from the tensor's start: 2^31 elements in a row, and far strides."""
    Cn, G, B = 1024, 32, 2100
    g = torch.Generator(device="cuda").manual_seed(1)
    if T == 1024:
        x = torch.empty(B, T, Cn, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    else:
        x = torch.empty((1 << 31) + 3 * T * Cn, device="cuda", dtype=torch.bfloat16).as_strided((3, T, Cn), ((1 << 30) + 8 * Cn, Cn, 1))
        x.normal_(generator=g)
    y, mean, rstd = pkg.group_norm_act(x, G, act="silu")
    dx, *_ = pkg.group_norm_act_backward(x, x, mean, rstd, G, act="silu")
    for i in (0, -1):
        one, m, r = x[i:][:1], mean[i:][:1], rstd[i:][:1]
        check_forward(one, G, None, None, "silu", None, None, got=(y[i:][:1], m, r))
        check_backward(one, one, m, r, G, None, None, "silu", None, None, got=(dx[i:][:1], None, None, None, None))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
def test_outliers_in_a_large_batch(dtype):
    """So many items that one block could take all rows of one: a thread's sums must not grow long."""
    x = torch.empty(300, 6000, 256, device="cuda", dtype=TYPES[dtype]).normal_(generator=torch.Generator(device="cuda").manual_seed(4))
    x[:, ::3000] *= 1e5
    y, mean, rstd = pkg.group_norm_act(x, 32, act="silu")
    dx, *_ = pkg.group_norm_act_backward(x, x, mean, rstd, 32, act="silu")
    for i in (0, 150, 299):
        one, m, r = x[i:i + 1], mean[i:i + 1], rstd[i:i + 1]
        check_forward(one, 32, None, None, "silu", None, None, got=(y[i:i + 1], m, r))
        check_backward(one, one, m, r, 32, None, None, "silu", None, None, got=(dx[i:i + 1], None, None, None, None))


def test_more_than_2_to_the_40_values_are_refused():
    L = Bd.load()
    for B, ok in ((1 << 10, False), ((1 << 10) - 1, True)):
        p = norm(B=B, T=1 << 20, C=1 << 10, groups=1)
        assert (L.mh3a_group_norm_act_workspace(C.byref(p), 0, 0) > 0) == ok


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp16", "bf16"))
@pytest.mark.parametrize("T", (40, 70000))
def test_silu_far_out(T, dtype):
    """Arguments from the exponential's overflow to its underflow, infinities and NaN, in both places of a pair."""
    Cn = 32
    x = case(1, T, Cn, "none", dtype, seed=3)[0]
    b = torch.linspace(-140, 140, Cn, device="cuda")
    for shift in (0, 1):
        b = b.roll(shift)
        y, mean, rstd = check_forward(x, 4, None, b, "silu", None, None)
        check_backward(x, x, mean, rstd, 4, None, b, "silu", None, None)
        far = b.clone()
        far[:3] = torch.tensor([float("inf"), -float("inf"), float("nan")])
        far[5], far[6] = float("nan"), -float("inf")
        got = pkg.group_norm_act(x, 4, None, far, act="silu")[0]
        odd = torch.tensor([0, 1, 2, 5, 6], device="cuda")
        rest = torch.tensor([i for i in range(Cn) if i not in (0, 1, 2, 5, 6)], device="cuda")
        assert torch.equal(got[..., rest], y[..., rest])
        assert torch.all(got[..., 0] == float("inf")) and torch.isnan(got[..., odd[2:4]]).all()
        # -inf times a sigmoid of 0, or of 2^-126 where it is clamped there: never a finite number
        assert not torch.isfinite(got[..., odd[[1, 4]]]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp16", "bf16"))
@pytest.mark.parametrize("T", (40, 70000))
def test_silu_far_out_in_both_channels_of_a_pair(T, dtype):
    """Neighbouring channels that hold the same values give the same results, also where the exponential
    overflows: 0 for finite arguments far below zero, NaN for -inf (0 times infinity), and no gradient."""
    far = [-84.0, -86.0, -86.5, -87.0, -87.5, -88.0, -89.0, -100.0, -200.0, -1e4, -1e10, -1e30, -3e38, float("-inf"), float("inf"), float("nan")]
    x = case(1, T, 16, "none", dtype, seed=3)[0].repeat_interleave(2, dim=2)
    b = torch.tensor(far, device="cuda").repeat_interleave(2)
    y, mean, rstd = pkg.group_norm_act(x, 4, None, b, act="silu")
    dx, _, db, _, _ = pkg.group_norm_act_backward(torch.ones_like(x), x, mean, rstd, 4, None, b, act="silu")
    even, odd = y[..., ::2].double(), y[..., 1::2].double()
    assert torch.equal(torch.isnan(even), torch.isnan(odd))
    # each is off by half a step of its type and a few units of 2^-24
    near = (even - odd).abs() <= 1.01 * torch.finfo(x.dtype).eps * even.abs() + torch.finfo(x.dtype).smallest_normal
    assert torch.all(near | torch.isnan(even) | (even == odd))
    assert torch.all(y[..., 16:26] == 0) and torch.isnan(y[..., 26:28]).all() and torch.isnan(y[..., 30:]).all()
    assert torch.all(y[..., 28:30] == float("inf"))
    assert torch.all(db[16:26] == 0)


def test_2_to_the_30_channels_are_refused():
    """Channel indices plus a tile, and groups plus channel tiles, have to fit 32 bits: near 2^31 channels the
    scratch size came out of a sum that had wrapped."""
    L, ok = Bd.load(), 1 << 20
    for B, Cn, groups in ((1, (1 << 31) - 1, (1 << 31) - 1), (1, 1 << 30, 1), (1 << 15, 1 << 15, 1 << 15), ((1 << 31) - 1, 1, 1)):
        p = norm(dtype=0, B=B, T=1, C=Cn, groups=groups)
        for backward in (0, 1):
            assert L.mh3a_group_norm_act_workspace(C.byref(p), backward, 0) == 0
        assert L.mh3a_group_norm_act(C.byref(p), ok, 0, 0, ok, ok, ok, ok, 1 << 40, None) == 3
    # below: an entry of 16 bytes for every group and channel tile, or the sums of every channel and two means a group
    most = (1 << 30) - 1
    p = norm(dtype=0, B=1, T=1, C=most, groups=most)
    assert L.mh3a_group_norm_act_workspace(C.byref(p), 0, 0) >= 16 * (most + most // 32)
    assert L.mh3a_group_norm_act_workspace(C.byref(p), 1, 0) >= 4 * most * (2 + 2 + 2)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ("weight", "bias", "alpha", "beta", "lengths"))
def test_an_output_over_a_parameter_is_refused(name):
    B, T, Cn = 2, 3, 16
    x, w, b, al, be = case(B, T, Cn, "snake_beta", "fp32", seed=1)
    buf = torch.ones(B * T * Cn + 2 * Cn, device="cuda")
    kw = dict(weight=w, bias=b, alpha=al, beta=be, lengths=None)
    size = B if name == "lengths" else Cn
    for at in (0, 7, B * T * Cn - 1):  # the first, one inside, across the end
        part = buf[Cn:][at:at + size]
        kw[name] = part.view(torch.int32) if name == "lengths" else part
        with pytest.raises(pkg.MH3AError, match="out overlaps " + name) as e:
            pkg.group_norm_act(x, 4, act="snake_beta", out=buf[Cn:-Cn].view(B, T, Cn), **kw)
        assert e.value.status == 1
    for at in (Cn - size, Cn + B * T * Cn):  # side by side
        part = buf[at:at + size]
        kw[name] = part.view(torch.int32) if name == "lengths" else part
        pkg.group_norm_act(x, 4, act="snake_beta", out=buf[Cn:-Cn].view(B, T, Cn), **kw)


def places(t):
    """The places of a view's elements in its storage."""
    at = torch.tensor(t.storage_offset())
    for n, s in zip(t.shape, t.stride()):
        at = at[..., None] + torch.arange(n) * s
    return set(at.flatten().tolist())


@pytest.mark.gpu
def test_views_of_one_buffer_are_refused_where_they_meet():
    """Random views with gaps, repeated and overlapping rows: refused if, and only if, they share an element."""
    rng = random.Random(5)
    buf = torch.randn(7000, device="cuda")
    met = 0
    for _ in range(400):
        B, T, Cn = rng.choice([(1, 5, 8), (3, 4, 8), (2, 1, 16), (4, 7, 4)])
        row = rng.choice([0, 3, Cn, Cn + 4, 5 * Cn, 96])
        item = rng.choice([0, Cn, row * T, row * T + 8, 2 * row * T + 1])
        out = buf[(at := rng.randrange(1500)):at + B * T * Cn].view(B, T, Cn)
        x = buf.as_strided((B, T, Cn), (item, row, 1), rng.randrange(1500))
        if places(x) & places(out):
            met += 1
            with pytest.raises(pkg.MH3AError, match="out overlaps x"):
                pkg.group_norm_act(x, 2, out=out)
        else:
            # (the way a call goes depends on the output's alignment, so bits may differ from a call without `out`)
            check_forward(x, 2, None, None, "none", None, None, got=pkg.group_norm_act(x, 2, out=out))
            buf.normal_()
    assert met > 40
    # the same view twice, and its neighbour's columns
    wide = torch.randn(2, 30, 64, device="cuda")
    some = wide[:1, :, :32]
    with pytest.raises(pkg.MH3AError, match="out overlaps x"):
        pkg.group_norm_act(wide[1:, ::2, 8:40], 2, out=wide.view(-1)[40 * 64:][:15 * 32].view(1, 15, 32))
    assert some.shape == pkg.group_norm_act(some, 2, out=wide.view(-1)[30 * 64:][:30 * 32].view(1, 30, 32))[0].shape


@pytest.mark.gpu
def test_gradients_are_not_lost_without_a_word():
    """Where autograd is recording, results lead back to a node that raises; elsewhere they are plain."""
    x, w, b, al, be = case(2, 5, 16, "snake_beta", "fp32", seed=2)
    args = dict(x=x, weight=w, bias=b, alpha=al, beta=be)
    for name in args:
        kw = {**args, name: args[name].clone().requires_grad_()}
        for k in range(3):
            r = pkg.group_norm_act(kw["x"], 4, kw["weight"], kw["bias"], act="snake_beta", alpha=kw["alpha"], beta=kw["beta"])[k]
            with pytest.raises(RuntimeError, match="mh3a_group_norm_act records no gradient: call group_norm_act_backward"):
                (3 * r).sum().backward()
            assert kw[name].grad is None
        with pytest.raises(pkg.MH3AError, match="out cannot be given"):
            pkg.group_norm_act(kw["x"], 4, kw["weight"], kw["bias"], act="snake_beta", alpha=kw["alpha"], beta=kw["beta"],
                               out=torch.empty_like(x))
        with torch.no_grad():
            got = pkg.group_norm_act(kw["x"], 4, kw["weight"], kw["bias"], act="snake_beta", alpha=kw["alpha"], beta=kw["beta"],
                                     out=torch.empty_like(x))
            assert not any(t.requires_grad for t in got)
    with pytest.raises(pkg.MH3AError, match="out cannot be given"):
        pkg.group_norm_act(x, 4, out=torch.empty_like(x).requires_grad_())
    y, m, r = pkg.group_norm_act(x, 4, w, b)
    assert not (y.requires_grad or m.requires_grad or r.requires_grad)
    for dx in pkg.group_norm_act_backward(y.clone().requires_grad_(), x, m, r, 4, w, b)[:3]:
        with pytest.raises(RuntimeError, match="records no gradient"):
            dx.sum().backward()


class NormAct(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, al, be):
        y, mean, rstd = pkg.group_norm_act(x, 4, w, b, act="snake_beta", alpha=al, beta=be)
        ctx.save_for_backward(x, mean, rstd, w, b, al, be)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, mean, rstd, w, b, al, be = ctx.saved_tensors
        return pkg.group_norm_act_backward(dy, x, mean, rstd, 4, w, b, act="snake_beta", alpha=al, beta=be)


@pytest.mark.gpu
def test_inside_an_autograd_function():
    x, w, b, al, be = case(2, 50, 16, "snake_beta", "fp32", seed=3)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(1)).cuda()
    leaves = [t.clone().requires_grad_() for t in (x, w, b, al, be)]
    y = NormAct.apply(*leaves)
    y.backward(dy)
    plain, mean, rstd = pkg.group_norm_act(x, 4, w, b, act="snake_beta", alpha=al, beta=be)
    want = pkg.group_norm_act_backward(dy, x, mean, rstd, 4, w, b, act="snake_beta", alpha=al, beta=be)
    assert torch.equal(y, plain) and all(torch.equal(t.grad, g) for t, g in zip(leaves, want))


class Guarded:
    """A buffer of exactly `shape` between guard values, on a 16-byte boundary."""

    def __init__(self, shape, dtype, lead=64):
        n = 1
        for s in shape:
            n *= s
        self.all = torch.full((n + 2 * lead,), 7, dtype=dtype, device="cuda")
        self.t = self.all[lead:lead + n].view(shape)
        self.lead = lead

    def ptr(self):
        return self.t.data_ptr()

    def whole(self):
        return bool((self.all[:self.lead] == 7).all() and (self.all[-self.lead:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", (False, True), ids=("full", "ragged"))
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("shape", [(3, 301, 24, 3), (3, 301, 25, 5), (3, 301, 30, 2), (3, 301, 12, 4), (1, 5, 8, 1), (2, 1, 7, 7),
                                   (3, 4001, 200, 8), (2, 700, 174, 3), (1, 3, 4104, 27)], ids=str)
def test_guards_around_every_output_and_the_scratch(shape, dtype, lengths):
    """Through the ABI, with scratch of exactly the size asked for: guard values around y, dx, the statistics, every
    gradient and the scratch stay.  Resident and general forms, vectors of 1 to 8 channels."""
    L = Bd.load()
    B, T, Cn, G = shape
    x, w, b, al, be = case(B, T, Cn, "snake_beta", dtype, seed=T)
    dy = x.flip(1).contiguous()
    n = torch.tensor([T, T // 2, 0][:B], dtype=torch.int32, device="cuda") if lengths else None
    p = norm(dtype=("fp32", "fp16", "bf16").index(dtype), act=2, B=B, T=T, C=Cn, groups=G)
    p.weight, p.bias, p.alpha, p.beta = (t.data_ptr() for t in (w, b, al, be))
    p.lengths = n.data_ptr() if lengths else None
    stream = torch.cuda.current_stream().cuda_stream
    for aligned in (1, 0):
        off = 1 - aligned  # an element off 16 bytes: narrower vectors
        size = [L.mh3a_group_norm_act_workspace(C.byref(p), k, aligned) for k in (0, 1)]
        ws = [Guarded((k,), torch.uint8) for k in size]
        y, mean, rstd = Guarded(x.shape, x.dtype, 64 + off), Guarded((B, G), torch.float32), Guarded((B, G), torch.float32)
        assert L.mh3a_group_norm_act(C.byref(p), x.data_ptr(), T * Cn, Cn, y.ptr(), mean.ptr(), rstd.ptr(), ws[0].ptr() if size[0] else None,
                                     size[0], stream) == 0
        dx, grads = Guarded(x.shape, x.dtype, 64 + off), [Guarded((Cn,), torch.float32) for _ in range(4)]
        assert L.mh3a_group_norm_act_backward(C.byref(p), x.data_ptr(), T * Cn, Cn, dy.data_ptr(), T * Cn, Cn, mean.ptr(), rstd.ptr(),
                                              dx.ptr(), *(g.ptr() for g in grads), ws[1].ptr() if size[1] else None, size[1], stream) == 0
        for g in (y, mean, rstd, dx, *grads, *ws):
            assert g.whole()
        check_forward(x, G, w, b, "snake_beta", al, be, lengths=n, got=(y.t, mean.t, rstd.t))
        check_backward(dy, x, mean.t, rstd.t, G, w, b, "snake_beta", al, be, lengths=n, got=(dx.t, *(g.t for g in grads)))


GENERAL = [(3, 3001, 25, 5, 0), (3, 3001, 64, 8, 1), (2, 40, 30, 2, 0)]  # odd and even widths; parameters off 16 bytes


def general_case(shape):
    B, T, Cn, G, off = shape
    x, *params = case(B, T, Cn, "snake_beta", "bf16", seed=T + Cn)
    if off:
        params = [torch.cat((p[:1], p))[1:] for p in params]
    w, b, al, be = params
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(2)).to(x.dtype).cuda()

    def both(x, stream=None):
        y, m, r = pkg.group_norm_act(x, G, w, b, act="snake_beta", alpha=al, beta=be, stream=stream)
        return (y, m, r) + pkg.group_norm_act_backward(dy, x, m, r, G, w, b, act="snake_beta", alpha=al, beta=be, stream=stream)

    return x, both


@pytest.mark.gpu
@pytest.mark.parametrize("shape", GENERAL, ids=str)
def test_general_form_on_two_streams(shape):
    """The launches of a call share scratch of their own, whatever another stream does."""
    x, both = general_case(shape)
    x2 = x.flip(0).contiguous()
    first, second = both(x), both(x2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    runs = [(both(x, s1), both(x2, s2.cuda_stream)) for _ in range(8)]
    torch.cuda.synchronize()
    for a, c in runs:
        assert all(torch.equal(p, q) for p, q in zip(a, first))
        assert all(torch.equal(p, q) for p, q in zip(c, second))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", GENERAL, ids=str)
def test_general_form_captured_and_replayed(shape):
    x, both = general_case(shape)
    graphs, outs = [], []
    for _ in range(2):  # two graphs with scratch of their own, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both(x))
        graphs.append(g)
    x.copy_(x.flip(1).clone() * 1.5)
    for k in (0, 1, 0):
        graphs[k].replay()
    torch.cuda.synchronize()
    want = both(x)
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(o, want))
