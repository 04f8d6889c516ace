"""Group norm with an activation over channels-last frames, and matrix products in 8-bit floating point
with one scale for each block of 128: cases, inputs, plain forms and 64-bit values.

``run`` makes the framework's calls where ``own`` is true, else the plain torch form.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "fp16": 2, "bf16": 2}
EPS = 1e-5
FP8_MAX = 448.0
FP8_TINY = 2.0 ** -100


# ----------------------------------------------------------------------------------- cases
def listed():
    return [
        # a few frames at 512 channels, as a streaming decoder gets them: latency
        dict(name="norm_frames", op="norm", B=1, T=4, C=512, G=32, act="snake_beta", dtype="bf16", ragged=False),
        # the length and width of the decoder's first stage on a 10 s stereo clip
        dict(name="norm_clip", op="norm", B=2, T=2000, C=512, G=32, act="snake_beta", dtype="bf16", ragged=False),
        # a padded batch of clips of unequal lengths, a width that is no power of two
        dict(name="norm_ragged", op="norm", B=7, T=3001, C=200, G=8, act="silu", dtype="fp16", ragged=True),
        # the second stage on sixteen 20 s items
        dict(name="norm_batch", op="norm", B=16, T=20000, C=256, G=32, act="silu", dtype="bf16", ragged=False),
        # gradients at the first stage's size, in the framework's own type
        dict(name="norm_grad_clip", op="norm_grad", B=2, T=2000, C=512, G=32, act="snake_beta", dtype="fp32",
             ragged=False),
        # gradients of a padded training batch
        dict(name="norm_grad_batch", op="norm_grad", B=16, T=10000, C=256, G=32, act="snake_beta", dtype="bf16",
             ragged=True),
        # one latent frame through a pointwise layer of the latent width: latency and the weights' bytes
        dict(name="linear_frame", op="linear", M=1, K=2048, N=2048, dtype="bf16", bias=True),
        # a 10 s stereo clip (2 x 400 frames), the decoder's input widths
        dict(name="linear_clip", op="linear", M=800, K=2048, N=1024, dtype="bf16", bias=True),
        # odd sizes: the last block of the inner axis is short, no size is a multiple of a tile
        dict(name="linear_odd", op="linear", M=517, K=1336, N=1000, dtype="fp32", bias=False),
        # sixteen 20 s items through an expanding layer
        dict(name="linear_batch", op="linear", M=12800, K=2048, N=8192, dtype="bf16", bias=True),
        # both gradients of a layer on a training batch of 16 clips of 10 s
        dict(name="linear_grad", op="linear_grad", M=6400, K=2048, N=2048, dtype="bf16"),
        # a layer's master weights laid out for the forward and the backward product after an update
        dict(name="weights", op="quantize", R=8192, K=2048, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "linear", "linear", "linear_grad", "quantize"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm_grad"):
        D = _log(rng, 1, 64)
        G = _log(rng, 1, 64)
        if rng.random() < 0.6:  # the usual widths: a multiple of 8
            D, G = max(1, D // 4 * 4), max(2, G // 2 * 2)
        B = _log(rng, 1, 16)
        most = (60_000_000 if op == "norm" else 30_000_000) // (B * D * G)
        T = _log(rng, 1, min(40000, max(1, most)))
        return dict(op=op, B=B, T=T, C=D * G, G=G, act=rng.choice(["none", "silu", "snake_beta"]), dtype=dtype,
                    ragged=rng.random() < 0.4)
    K, N = _log(rng, 32, 8192), _log(rng, 32, 8192)
    if rng.random() < 0.5:
        K, N = max(32, K // 128 * 128), max(32, N // 128 * 128)
    if op == "quantize":
        return dict(op=op, R=N, K=min(K, 2048), dtype=dtype)
    M = _log(rng, 1 if op == "linear" else 64, 12800)
    most = 200_000_000_000 if op == "linear" else 25_000_000_000
    M = max(1, min(M, most // (K * N)))
    c = dict(op=op, M=M, K=K, N=N, dtype=dtype)
    return dict(c, bias=rng.random() < 0.5) if op == "linear" else c


def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op in ("norm", "norm_grad"):
        n = case["B"] * case["T"] * case["C"]
        if op == "norm":
            return {"bytes": 2 * n * e + 16 * case["C"] + 8 * case["B"] * case["G"], "flops": 16 * n}
        return {"bytes": 3 * n * e + 32 * case["C"] + 8 * case["B"] * case["G"], "flops": 40 * n}
    if op == "quantize":
        n = case["R"] * case["K"]
        return {"bytes": n * e + 2 * n + 8 * (n // 16384 + 1), "flops": 4 * n}
    M, K, N = case["M"], case["K"], case["N"]
    if op == "linear":
        return {"bytes": M * K * e + N * K + M * N * e, "flops": 2 * M * K * N}
    return {"bytes": M * K * e + M * N * e + N * K + M * K * e + 4 * N * K, "flops": 4 * M * K * N}


# ---------------------------------------------------------------------------------- inputs
def _pad16(n):
    return (n + 15) // 16 * 16


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=g, device="cuda")

    dt = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] in ("norm", "norm_grad"):
        B, T, C, G = case["B"], case["T"], case["C"], case["G"]
        # channels with levels and offsets of their own
        s["x"] = (randn(B, T, C) * uniform(0.3, 3.0, C) + randn(C)).to(dt)
        s["weight"], s["bias"] = 1 + 0.2 * randn(C), 0.2 * randn(C)
        snake = case["act"] == "snake_beta"
        s["alpha"] = uniform(0.8, 1.2, C) if snake else None
        s["beta"] = uniform(0.8, 1.2, C) if snake else None
        s["lengths"] = None
        if case["ragged"]:
            n = torch.randint(T // 2, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            n[0] = T
            s["lengths"] = n
        if case["op"] == "norm_grad":
            s["dy"] = randn(B, T, C).to(dt)
            # what the forward pass keeps for the backward pass
            mean, rstd = _norm_stats(s["x"].float(), G, s["lengths"])
            s["mean"], s["rstd"] = mean.contiguous(), rstd.contiguous()
        return s
    if case["op"] == "quantize":
        s["x"] = (randn(case["R"], case["K"]) / math.sqrt(case["K"])).to(dt)
        return s
    M, K, N = case["M"], case["K"], case["N"]
    # activations: channels of unequal level
    s["x"] = (randn(M, K) * torch.exp(0.7 * randn(K))).to(dt)
    w = randn(N, K) / math.sqrt(K)
    if case["op"] == "linear":
        s["w"], s["w_scale"] = _stored(*_quantize(w, 128))
        s["bias"] = 0.1 * randn(N) if case["bias"] else None
    else:
        s["dy"] = randn(M, N).to(dt)
        s["wt"], s["wt_scale"] = _stored(*_quantize(w.t(), 128))
    return s


def _stored(q, scale):
    """The fp8 matrix as a user's program keeps it: rows start on 16-byte boundaries."""
    rows, k = q.shape
    buf = torch.zeros(rows, _pad16(k), device=q.device, dtype=torch.uint8)
    buf[:, :k] = q.contiguous().view(torch.uint8)
    return buf.view(torch.float8_e4m3fn)[:, :k], scale.contiguous()


# ------------------------------------------------------------------------------ plain forms
def _norm_stats(x, G, lengths):
    B, T, C = x.shape
    D = C // G
    if lengths is None:
        xg = x.view(B, T, G, D)
        mean = xg.mean(dim=(1, 3))
        var = (xg - mean[:, None, :, None]).square().mean(dim=(1, 3))
    else:
        valid = _valid(x, lengths)
        n = (lengths.clamp(1, T).float() * D)[:, None]
        mean = torch.where(valid, x, 0).view(B, T, G, D).sum(dim=(1, 3)) / n
        d = torch.where(valid, x - mean.repeat_interleave(D, 1)[:, None], 0)
        var = d.square().view(B, T, G, D).sum(dim=(1, 3)) / n
    return mean, torch.rsqrt(var + EPS)


def _valid(x, lengths):
    return (torch.arange(x.shape[1], device=x.device)[None] < lengths[:, None])[:, :, None]


def _plain_norm(s):
    x, G, D = s["x"].float(), s["G"], s["C"] // s["G"]
    mean, rstd = _norm_stats(x, G, s["lengths"])
    u = (x - mean.repeat_interleave(D, 1)[:, None]) * rstd.repeat_interleave(D, 1)[:, None]
    u = u * s["weight"] + s["bias"]
    if s["act"] == "silu":
        y = u / (1 + torch.exp(-u))
    elif s["act"] == "snake_beta":
        y = u + torch.sin(s["alpha"] * u).square() / (s["beta"] + 1e-9)
    else:
        y = u
    if s["lengths"] is not None:
        y = torch.where(_valid(x, s["lengths"]), y, 0)
    return y.to(s["x"].dtype), mean, rstd


def _plain_norm_grad(s):
    x, dy, D = s["x"].float(), s["dy"].float(), s["C"] // s["G"]
    B, T, C = x.shape
    rstd = s["rstd"].repeat_interleave(D, 1)[:, None]
    xh = (x - s["mean"].repeat_interleave(D, 1)[:, None]) * rstd
    n = float(T)
    if s["lengths"] is not None:
        valid = _valid(x, s["lengths"])
        xh, dy = torch.where(valid, xh, 0), torch.where(valid, dy, 0)
        n = s["lengths"].clamp(1, T).float()[:, None]
    u = xh * s["weight"] + s["bias"]
    dalpha = dbeta = None
    if s["act"] == "silu":
        sig = 1 / (1 + torch.exp(-u))
        du = dy * (sig * (1 + u * (1 - sig)))
    elif s["act"] == "snake_beta":
        inv = 1 / (s["beta"] + 1e-9)
        sin2 = torch.sin(2 * s["alpha"] * u) * inv
        du = dy * (1 + s["alpha"] * sin2)
        dalpha = (dy * u * sin2).sum(dim=(0, 1))
        dbeta = -(dy * torch.sin(s["alpha"] * u).square()).sum(dim=(0, 1)) * inv * inv
    else:
        du = dy
    dbias = du.sum(dim=(0, 1))
    dweight = (du * xh).sum(dim=(0, 1))
    dxh = du * s["weight"]
    s1 = dxh.sum(dim=1).view(B, -1, D).sum(dim=2) / (n * D)
    s2 = (dxh * xh).sum(dim=1).view(B, -1, D).sum(dim=2) / (n * D)
    dx = rstd * (dxh - s1.repeat_interleave(D, 1)[:, None] - xh * s2.repeat_interleave(D, 1)[:, None])
    if s["lengths"] is not None:
        dx = torch.where(valid, dx, 0)
    return dx.to(s["x"].dtype), dweight, dbias, dalpha, dbeta


def _quantize(x, block_rows):
    """q [R, K] e4m3 and scale [ceil(K/128), ceil(R/block_rows)]: the block's largest magnitude becomes 448."""
    R, K = x.shape
    x = x.float()
    rb, kb = -(-R // block_rows), -(-K // 128)
    p = torch.nn.functional.pad(x, (0, kb * 128 - K, 0, rb * block_rows - R))
    p = p.view(rb, block_rows, kb, 128)
    amax = p.abs().amax(dim=(1, 3), keepdim=True).clamp(min=FP8_TINY)
    top = torch.full_like(amax, FP8_MAX)  # tensor by tensor: a quotient with a number is formed by its reciprocal
    q = (p * (top / amax)).to(torch.float8_e4m3fn).view(rb * block_rows, kb * 128)[:R, :K]
    return q, (amax / top)[:, 0, :, 0].t()


def _values(q, scale):
    """The numbers that q and its block scales stand for."""
    R, K = q.shape
    block_rows = 1 if scale.shape[1] == R else 128
    full = scale.repeat_interleave(128, 0)[:K].repeat_interleave(block_rows, 1)[:, :R]
    return q.float() * full.t()


def _plain_linear(s):
    y = _values(*_quantize(s["x"], 1)) @ _values(s["w"], s["w_scale"]).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["x"].dtype)


def _plain_linear_grad(s):
    dx = _values(*_quantize(s["dy"], 1)) @ _values(s["wt"], s["wt_scale"]).t()
    dyt, xt = _quantize(s["dy"].t(), 1), _quantize(s["x"].t(), 1)
    return dx.to(s["x"].dtype), _values(*dyt) @ _values(*xt).t()


# -------------------------------------------------------------------------------------- run
def run(s):
    op = s["op"]
    if own:
        import bigvgan_waveform_decoder_b200 as pkg

        if op == "norm":
            return pkg.group_norm_act(s["x"], s["G"], s["weight"], s["bias"], act=s["act"], alpha=s["alpha"],
                                      beta=s["beta"], eps=EPS, lengths=s["lengths"])
        if op == "norm_grad":
            return pkg.group_norm_act_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["G"], s["weight"], s["bias"],
                                               act=s["act"], alpha=s["alpha"], beta=s["beta"],
                                               lengths=s["lengths"])
        if op == "linear":
            return pkg.fp8_linear(s["x"], s["w"], s["w_scale"], s["bias"])
        if op == "linear_grad":
            dx = pkg.fp8_linear(s["dy"], s["wt"], s["wt_scale"])
            dyt, dyt_scale = pkg.fp8_quantize(s["dy"], transpose=True)
            xt, xt_scale = pkg.fp8_quantize(s["x"], transpose=True)
            return dx, pkg.fp8_matmul(dyt, dyt_scale, xt, xt_scale, torch.float32)
        return (*pkg.fp8_quantize(s["x"], block_rows=128), *pkg.fp8_quantize(s["x"], block_rows=128, transpose=True))
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_grad":
        return _plain_norm_grad(s)
    if op == "linear":
        return _plain_linear(s)
    if op == "linear_grad":
        return _plain_linear_grad(s)
    return (*_quantize(s["x"], 128), *_quantize(s["x"].t(), 128))


# ------------------------------------------------------------------------------------ exact
def _exact_fp8(x, rows, cols):
    """64-bit values of x in e4m3 under one scale for each rows x cols block.  The scale and the product that is
    rounded are 32-bit numbers by definition."""
    R, K = x.shape
    x = x.double()
    i = (torch.arange(R, device=x.device) // rows)[:, None]
    j = (torch.arange(K, device=x.device) // cols)[None]
    nj = -(-K // cols)
    block = (i * nj + j).reshape(-1)
    top = torch.zeros(-(-R // rows) * nj, device=x.device, dtype=torch.float64)
    top = top.scatter_reduce(0, block, x.abs().reshape(-1), "amax").clamp(min=FP8_TINY)
    scale = (top / FP8_MAX).float().double()
    factor = (FP8_MAX / top).float().double()
    v = (x * factor[block].view(R, K)).float().double()
    # e4m3: three fraction bits down to 2^-6, steps of 2^-9 below, nearest with ties to even
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.pow(2.0, e - 3)
    q = torch.clamp(torch.round(v / step) * step, -FP8_MAX, FP8_MAX)
    return q, scale.view(-1, nj), q * scale[block].view(R, K)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        q, scale, _ = _exact_fp8(s["x"], 128, 128)
        return q, scale.t(), q.t(), scale
    if op in ("linear", "linear_grad"):
        def held(q, scale):
            at = torch.arange(q.shape[0], device=q.device) // 128
            kt = torch.arange(q.shape[1], device=q.device) // 128
            return q.to(torch.float64) * scale.double()[kt][:, at].t()

        if op == "linear":
            y = torch.einsum("mk,nk->mn", _exact_fp8(s["x"], 1, 128)[2], held(s["w"], s["w_scale"]))
            return y if s["bias"] is None else y + s["bias"].double()
        dx = torch.einsum("mn,kn->mk", _exact_fp8(s["dy"], 1, 128)[2], held(s["wt"], s["wt_scale"]))
        dw = torch.einsum("mn,mk->nk", _exact_fp8(s["dy"], 128, 1)[2], _exact_fp8(s["x"], 128, 1)[2])
        return dx, dw
    B, T, C, G = case["B"], case["T"], case["C"], case["G"]
    D = C // G
    n = s["lengths"].double() if s["lengths"] is not None else torch.full((B,), float(T), device="cuda").double()
    keep = (torch.arange(T, device="cuda")[None] < n[:, None]).double()[:, :, None, None]
    x = s["x"].double().view(B, T, G, D) * keep
    count = (n.clamp(min=1) * D).view(B, 1, 1, 1)

    def per_channel(t):
        return t.double().view(1, 1, G, D)

    w, b = per_channel(s["weight"]), per_channel(s["bias"])
    if op == "norm":
        mean = x.sum(dim=(1, 3), keepdim=True) / count
        var = (keep * (x - mean) ** 2).sum(dim=(1, 3), keepdim=True) / count
        rstd = (var + EPS) ** -0.5
    else:
        mean, rstd = (s[k].double().view(B, 1, G, 1) for k in ("mean", "rstd"))
    xh = (x - mean) * rstd
    u = xh * w + b
    if op == "norm":
        if case["act"] == "silu":
            y = u * torch.sigmoid(u)
        elif case["act"] == "snake_beta":
            y = u + (1 - torch.cos(2 * per_channel(s["alpha"]) * u)) / (2 * (per_channel(s["beta"]) + 1e-9))
        else:
            y = u
        return (y * keep).view(B, T, C), mean.view(B, G), rstd.view(B, G)
    dy = s["dy"].double().view(B, T, G, D) * keep
    dalpha = dbeta = None
    slope = torch.ones_like(u)
    if case["act"] == "silu":
        sig = torch.sigmoid(u)
        slope = sig + u * sig * (1 - sig)
    elif case["act"] == "snake_beta":
        al, be = per_channel(s["alpha"]), per_channel(s["beta"]) + 1e-9
        sn, cs = torch.sin(al * u), torch.cos(al * u)
        slope = 1 + 2 * al * sn * cs / be
        dalpha = (dy * 2 * u * sn * cs / be).sum(dim=(0, 1)).view(C)
        dbeta = -(dy * sn * sn / be ** 2).sum(dim=(0, 1)).view(C)
    du = dy * slope
    dweight, dbias = (du * xh).sum(dim=(0, 1)).view(C), du.sum(dim=(0, 1)).view(C)
    h = du * w
    m1 = h.sum(dim=(1, 3), keepdim=True) / count
    m2 = (h * xh).sum(dim=(1, 3), keepdim=True) / count
    return (rstd * (h - m1 - xh * m2) * keep).view(B, T, C), dweight, dbias, dalpha, dbeta
