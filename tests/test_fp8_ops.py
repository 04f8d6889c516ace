"""fp8 matrices with one scale for each block of 128 values: quantisation, product, linear layer."""
import ctypes as C
import random

import pytest
import torch

import bigvgan_waveform_decoder_b200 as pkg
from bigvgan_waveform_decoder_b200 import binding as Bd

from . import ops_ref as R
from .test_norm_ops import places

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def rand(*shape, seed=0, dtype="fp32", spread=0.7):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp(spread * torch.randn(shape[-1], generator=g))
    return x.to(TYPES[dtype]).cuda()


def check_quantized(x, block_rows, transpose, got=None):
    q, scale = got or pkg.fp8_quantize(x, block_rows=block_rows, transpose=transpose)
    rq, rs, _ = R.quantize(x.t() if transpose else x, block_rows)
    assert q.dtype == torch.float8_e4m3fn and q.shape == rq.shape and scale.shape == rs.shape
    assert q.data_ptr() % 16 == 0 and (q.shape[0] == 1 or q.stride(0) % 16 == 0)
    assert torch.equal(scale.double(), rs)          # fp32 quotients, correctly rounded
    assert torch.equal(q.float().double(), rq)      # and what they give, exactly


def check_product(out, a, a_scale, b, b_scale, bias=None):
    va, vb = R.dequantize(a, a_scale), R.dequantize(b, b_scale)
    ref = va @ vb.t()
    mag = va.abs() @ vb.abs().t()
    if bias is not None:
        ref, mag = ref + bias.double(), mag + bias.double().abs()
    # Products of two e4m3 numbers are exact.  The tensor core adds a block's 128 of them in fp32, at worst
    # cutting instead of rounding (2^-23 of the running size a step, 4 steps of 32 with a tree below:
    # under 16 x 2^-23); a scale times a sum and its addition are two roundings a block, over K / 128
    # blocks; then one rounding to the output's type.
    kb = -(-a.shape[1] // 128)
    tol = (16 * 2 + 2 * kb) * R.F24 * mag + torch.finfo(out.dtype).eps / 2 * ref.abs() + torch.finfo(out.dtype).smallest_normal
    off = (out.double() - ref).abs()
    assert torch.all(off <= tol), float((off / tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mode", [(1, False), (1, True), (128, False), (128, True)], ids=str)
@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (3, 130), (128, 128), (129, 127), (5, 2048), (300, 36), (257, 513), (1000, 1336)],
                         ids=str)
def test_quantize(shape, mode, dtype):
    check_quantized(rand(*shape, seed=sum(shape), dtype=dtype), *mode)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [(1, False), (1, True), (128, False), (128, True)], ids=str)
def test_quantize_every_16_bit_value_and_ties(mode):
    """All finite bf16 and fp16 numbers, and powers of two times every tie between e4m3 numbers."""
    every = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16)
    for dt in (torch.bfloat16, torch.float16):
        v = every.view(dt)
        v = v[torch.isfinite(v.float())]
        n = v.numel() // 128 * 128
        check_quantized(v[:n].view(-1, 128).cuda(), *mode)
        check_quantized(v[torch.randperm(n, generator=torch.Generator().manual_seed(1))].view(-1, 256).cuda(), *mode)
    ties = torch.cat([torch.arange(1, 129) / 16.0 * 2.0 ** e for e in (-9, -4, 0, 3)])
    check_quantized(torch.cat([ties, torch.full((512,), 448.0)]).view(-1, 128).cuda(), *mode)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [(1, False), (1, True), (128, False), (128, True)], ids=str)
def test_quantize_extreme_blocks(mode):
    block_rows, transpose = mode
    x = torch.zeros(256, 256, device="cuda")
    check_quantized(x, *mode)                                  # nothing but zeros
    x[:128, :128] = 1e-44                                      # far below the smallest scale
    x[128:, :128] = 3.4e38
    x[:128, 128:] = torch.where(torch.rand(128, 128, device="cuda") < 0.5, -1e-37, 2e-38)
    check_quantized(x, *mode)
    x = rand(256, 256, seed=3)
    q0, s0 = pkg.fp8_quantize(x, block_rows=block_rows, transpose=transpose)
    x[130, 7] = float("nan")
    q, s = pkg.fp8_quantize(x, block_rows=block_rows, transpose=transpose)
    bad = torch.isnan(s)
    r, k = (7, 130) if transpose else (130, 7)
    want = torch.zeros_like(bad)
    want[k // 128, r if block_rows == 1 else r // 128] = True
    assert torch.equal(bad, want)
    whole = want.repeat_interleave(128, 0).repeat_interleave(block_rows, 1).t()
    assert torch.equal(torch.isnan(q.float()), whole)
    assert torch.equal(q.float()[~whole], q0.float()[~whole]) and torch.equal(s[~want], s0[~want])
    x[130, 7] = float("inf")
    q, s = pkg.fp8_quantize(x, block_rows=block_rows, transpose=transpose)
    assert torch.equal(torch.isinf(s), want) and bool(torch.isnan(q.float()[r, k]))
    assert torch.equal(q.float()[~whole], q0.float()[~whole])


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [(1, False), (1, True), (128, False), (128, True)], ids=str)
def test_quantize_strided(mode):
    x = rand(140, 700, seed=4, dtype="bf16")
    for v in (x[:, 3:400], x[::2, :256], x[:1].expand(140, 700), x[5:6, 1:2]):
        check_quantized(v, *mode)


@pytest.mark.gpu
def test_quantize_writes_nothing_behind_its_rows():
    """Through the ABI with guard bytes: between the rows, and behind the last one."""
    L = Bd.load()
    x = rand(37, 141, seed=5)
    for transpose in (0, 1):
        outer, inner = (141, 37) if transpose else (37, 141)
        for block_rows in (1, 128):
            buf = torch.full((outer + 1, 160), 0x5A, dtype=torch.uint8, device="cuda")
            scale = torch.full((-(-inner // 128) * -(-outer // block_rows) + 4,), 7.0, device="cuda")
            st = L.mh3a_fp8_quantize(x.data_ptr(), 0, 37, 141, 141, block_rows, transpose, buf.data_ptr(), 160, scale.data_ptr(),
                                     torch.cuda.current_stream().cuda_stream)
            assert st == 0
            torch.cuda.synchronize()
            assert torch.all(buf[:outer, inner:] == 0x5A) and torch.all(buf[outer] == 0x5A) and torch.all(scale[-4:] == 7)
            q = buf.view(torch.float8_e4m3fn)[:outer, :inner]
            check_quantized(x, block_rows, bool(transpose), got=(q, scale[:-4].view(-(-inner // 128), -1)))


PRODUCTS = [
    # M, N, K
    (1, 1, 1), (1, 16, 128), (9, 33, 32), (16, 2048, 2048), (128, 256, 128), (129, 257, 129), (77, 1000, 1336),
    (517, 1000, 300), (800, 1024, 2048), (1300, 2050, 640), (2304, 4224, 144),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("b_rows", (1, 128))
@pytest.mark.parametrize("shape", PRODUCTS, ids=str)
def test_matmul(shape, b_rows, dtype):
    M, N, K = shape
    a = pkg.fp8_quantize(rand(M, K, seed=M + K))
    b = pkg.fp8_quantize(rand(N, K, seed=N), block_rows=b_rows)
    bias = rand(N, seed=1) if N % 2 else None
    out = pkg.fp8_matmul(*a, *b, TYPES[dtype], bias=bias)
    assert out.shape == (M, N) and out.dtype == TYPES[dtype]
    check_product(out, *a, *b, bias)


@pytest.mark.gpu
def test_matmul_of_small_integers_is_exact():
    """Integers and scales that fp32 adds without rounding: every lane and column in its place."""
    for M, N, K, b_rows in ((300, 520, 384, 1), (140, 200, 256, 128), (2000, 4100, 128, 128)):
        g = torch.Generator().manual_seed(M)
        a = torch.randint(-8, 9, (M, K), generator=g).float().to(torch.float8_e4m3fn).cuda()
        b = torch.randint(-8, 9, (N, K), generator=g).float().to(torch.float8_e4m3fn).cuda()
        sa = torch.pow(2.0, torch.randint(-2, 3, (K // 128, M), generator=g).float()).cuda()
        sb = torch.pow(2.0, torch.randint(-2, 3, (K // 128, -(-N // b_rows)), generator=g).float()).cuda()
        out = pkg.fp8_matmul(a, sa, b, sb, torch.float32)
        assert torch.equal(out.double(), R.dequantize(a, sa) @ R.dequantize(b, sb).t())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
def test_matmul_padded_operands_and_strided_output(dtype):
    """Garbage (NaN bytes) behind the operands' rows is not read; bytes around the output stay."""
    M, N, K = 200, 140, 200
    qa, sa = pkg.fp8_quantize(rand(M, K, seed=1))
    qb, sb = pkg.fp8_quantize(rand(N, K, seed=2), block_rows=128)
    stored = []
    for q in (qa, qb):
        buf = torch.full((q.shape[0], 272), 0x7F, dtype=torch.uint8, device="cuda")
        buf[:, :K] = q.view(torch.uint8)
        stored.append(buf.view(torch.float8_e4m3fn)[:, :K])
    for extra in (0, 3, 20):
        wide = torch.full((M + 2, N + extra + 8), 5.0, device="cuda", dtype=TYPES[dtype])
        out = wide[1:-1, extra:extra + N]
        got = pkg.fp8_matmul(stored[0], sa, stored[1], sb, TYPES[dtype], out=out)
        assert got.data_ptr() == out.data_ptr()
        check_product(out, qa, sa, qb, sb)
        assert torch.all(wide[0] == 5) and torch.all(wide[-1] == 5)
        assert torch.all(wide[:, :extra] == 5) and torch.all(wide[:, extra + N:] == 5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 2048, 2048), (1, 8, 32), (2, 100, 130), (3, 1000, 2049), (4, 17, 5000), (5, 64, 256),
                                   (8, 2048, 1336), (9, 300, 500), (64, 2048, 2048), (1, 4100, 12300), (3, 8200, 4096), (517, 1000, 1336)], ids=str)
@pytest.mark.parametrize("w_rows", (1, 128))
def test_linear(shape, w_rows, dtype):
    M, N, K = shape
    x = rand(M, K, seed=M, dtype=dtype)
    w = pkg.fp8_quantize(rand(N, K, seed=N), block_rows=w_rows)
    bias = rand(N, seed=2)
    y = pkg.fp8_linear(x, *w, bias)
    assert y.shape == (M, N) and y.dtype == x.dtype
    xq, xs, _ = R.quantize(x, 1)
    check_product(y, xq.float(), xs.float(), *w, bias)


@pytest.mark.gpu
@pytest.mark.parametrize("M", (1, 3, 40))
def test_linear_strided_rows(M):
    K, N = 300, 130
    wide = rand(2 * M, K + 50, seed=6, dtype="bf16")
    w = pkg.fp8_quantize(rand(N, K, seed=7), block_rows=128)
    for x in (wide[:M, 1:K + 1], wide[::2, 8:K + 8], wide[:1, :K].expand(M, K)):
        xq, xs, _ = R.quantize(x, 1)
        out = torch.full((M, N + 7), 3.0, device="cuda", dtype=x.dtype)
        check_product(pkg.fp8_linear(x, *w, out=out[:, 2:N + 2]), xq.float(), xs.float(), *w)
        assert torch.all(out[:, :2] == 3) and torch.all(out[:, N + 2:] == 3)


@pytest.mark.gpu
@pytest.mark.parametrize("M", (1, 8, 100))
def test_not_finite_rows_stay_alone(M):
    K, N = 512, 256
    x = rand(M + 1, K, seed=8, dtype="bf16")
    w = pkg.fp8_quantize(rand(N, K, seed=9), block_rows=128)
    y0 = pkg.fp8_linear(x, *w)
    x[M, 200] = float("nan")
    y = pkg.fp8_linear(x, *w)
    assert bool(torch.isnan(y[M].float()).all()) and torch.equal(y[:M], y0[:M])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(200, 130, 300), (640, 512, 384)], ids=str)
def test_gradients_of_the_linear_layer(shape):
    """dx = dy w and dw = dy^T x with every operand in fp8, against 64 bits of the same operands, and
    against the gradients without fp8: each operand is off by at most 2^-4 of its values (half a step of
    e4m3) or, below 2^-6 of 448, by 2^-10 of the block's scale."""
    M, N, K = shape
    x, w, dy = rand(M, K, seed=1, dtype="bf16"), rand(N, K, seed=2, spread=0.0), rand(M, N, seed=3, dtype="bf16", spread=0.0)
    wt = pkg.fp8_quantize(w, block_rows=128, transpose=True)
    wq = pkg.fp8_quantize(w, block_rows=128)
    assert torch.equal(wt[0].float(), wq[0].float().t()) and torch.equal(wt[1], wq[1].t())
    dx = pkg.fp8_linear(dy, *wt)
    gq, gs, gv = R.quantize(dy, 1)
    check_product(dx, gq.float(), gs.float(), *wt)
    a, b = pkg.fp8_quantize(dy, transpose=True), pkg.fp8_quantize(x, transpose=True)
    dw = pkg.fp8_matmul(*a, *b, torch.float32)
    check_product(dw, *a, *b)

    def step(v, block_rows):
        s = R.quantize(v, block_rows)[1]
        r = torch.arange(v.shape[0], device=v.device) // block_rows
        k = torch.arange(v.shape[1], device=v.device) // 128
        return torch.maximum(v.double().abs() * 2.0 ** -4, s[k][:, r].t() * 2.0 ** -10)

    w64, x64, g64 = w.double(), x.double(), dy.double()
    ew, eg = step(w, 128), step(dy, 1)
    bound = g64.abs() @ ew + eg @ w64.abs() + eg @ ew
    slack = 1.01 * bound + 2.0 ** -8 * (g64 @ w64).abs() + 1e-6
    assert torch.all((dx.double() - g64 @ w64).abs() <= slack)
    et, ex = step(dy.t(), 1), step(x.t(), 1)
    bound = g64.t().abs() @ ex.t() + et @ x64.abs() + et @ ex.t()
    assert torch.all((dw.double() - g64.t() @ x64).abs() <= 1.01 * bound + 1e-6)


@pytest.mark.gpu
def test_streams_graphs_and_repeats():
    w = pkg.fp8_quantize(rand(1000, 640, seed=1), block_rows=128)
    xs = [rand(m, 640, seed=m, dtype="bf16") for m in (1, 6, 300)]
    first = [pkg.fp8_linear(x, *w) for x in xs]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        runs = [[pkg.fp8_linear(x, *w, stream=s) for x in xs] for s in (s1, s2.cuda_stream)]
        torch.cuda.synchronize()
        for r in runs:
            assert all(torch.equal(p, q) for p, q in zip(r, first))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = [pkg.fp8_linear(x, *w) for x in xs] + list(pkg.fp8_quantize(xs[2], transpose=True))
        graphs.append((g, outs))
    for x in xs:
        x.copy_(x.flip(1).clone())
    for k in (0, 1, 0):
        graphs[k][0].replay()
    torch.cuda.synchronize()
    want = [pkg.fp8_linear(x, *w) for x in xs] + list(pkg.fp8_quantize(xs[2], transpose=True))
    for _, outs in graphs:
        assert all(torch.equal(p.float(), q.float()) for p, q in zip(outs, want))


@pytest.mark.gpu
def test_norm_then_linear_then_decode(small_arch):
    """The layers as they are used: a residual unit over channels-last frames (norm, SnakeBeta, pointwise
    convolution), a projection to latents, and the decoder on them."""
    from bigvgan_waveform_decoder_b200 import synthetic as S

    B, T, Cn = 2, 6, 256
    x = rand(B, T, Cn, seed=1, dtype="bf16", spread=0.0)
    nw, nb = 1 + 0.1 * rand(Cn, seed=2, spread=0.0), 0.1 * rand(Cn, seed=3, spread=0.0)
    al, be = torch.rand(Cn, device="cuda") + 0.5, torch.rand(Cn, device="cuda") + 0.5
    w1 = pkg.fp8_quantize(rand(Cn, Cn, seed=4, spread=0.0) / 16, block_rows=128)
    w2 = pkg.fp8_quantize(rand(small_arch.latent_channels, Cn, seed=5, spread=0.0) / 16, block_rows=128)
    h, mean, rstd = pkg.group_norm_act(x, 32, nw, nb, act="snake_beta", alpha=al, beta=be)
    x2 = x + pkg.fp8_linear(h.view(B * T, Cn), *w1).view(B, T, Cn)
    z = pkg.fp8_linear(x2.view(B * T, Cn).float(), *w2).view(B, T, -1).transpose(1, 2).contiguous()
    d = pkg.Decoder(small_arch, S.make_weights(small_arch, 1), max_batch=B, max_frames=T)
    y = d.decode(z)
    torch.cuda.synchronize()
    d.check_device_error()
    d.close()
    assert y.shape == (B, 1, 800 * T) and bool(torch.isfinite(y).all())
    # the same layers from their formulas, each on the output that the library gave the one before
    rh = R.norm_forward(x, 32, nw, nb, "snake_beta", al, be, 1e-5, None)[0]
    assert torch.all((h.double() - rh).abs() <= 2.0 ** -8 * rh.abs() + 1e-3)
    xq, xs, _ = R.quantize(x2.view(B * T, Cn).float(), 1)
    check_product(z.transpose(1, 2).reshape(B * T, -1), xq.float(), xs.float(), *w2)
    # and back: gradients of the projection and of the norm
    dz = rand(B * T, small_arch.latent_channels, seed=6, spread=0.0)
    w1t = pkg.fp8_quantize(R.dequantize(*w1).float(), block_rows=128, transpose=True)
    w2t = pkg.fp8_quantize(R.dequantize(*w2).float(), block_rows=128, transpose=True)
    dx2 = pkg.fp8_linear(dz, *w2t)
    dh = pkg.fp8_linear(dx2.to(torch.bfloat16), *w1t).view(B, T, Cn)
    dx, dw, db, da, dbe = pkg.group_norm_act_backward(dh, x, mean, rstd, 32, nw, nb, act="snake_beta", alpha=al, beta=be)
    ref, mag = R.norm_backward(dh, x, 32, nw, nb, "snake_beta", al, be, mean, rstd, None)
    assert torch.all((dx.double() - ref["dx"]).abs() <= 2.0 ** -8 * ref["dx"].abs() + 2.0 ** -17 * mag["dx"])
    for g, k in ((dw, "dweight"), (db, "dbias"), (da, "dalpha"), (dbe, "dbeta")):
        assert torch.all((g.double() - ref[k]).abs() <= 2.0 ** -17 * mag[k])


@pytest.mark.gpu
def test_python_refusals():
    x = rand(10, 256, seed=1)
    q, s = pkg.fp8_quantize(x)
    w, ws = pkg.fp8_quantize(rand(300, 256, seed=2), block_rows=128)
    n = pkg.MH3AError
    for bad in (lambda: pkg.fp8_quantize(x, block_rows=2), lambda: pkg.fp8_quantize(x.double()), lambda: pkg.fp8_quantize(x.cpu()),
                lambda: pkg.fp8_quantize(x[0]), lambda: pkg.fp8_quantize(x[:, ::2]), lambda: pkg.fp8_quantize(x[:0]),
                lambda: pkg.fp8_matmul(w, ws, w, ws), lambda: pkg.fp8_matmul(q, s, w[:, :128], ws[:1].contiguous()),
                lambda: pkg.fp8_matmul(q, s.t().contiguous(), w, ws), lambda: pkg.fp8_matmul(q, s, w, ws.half()),
                lambda: pkg.fp8_matmul(q, s, w, ws, torch.float64), lambda: pkg.fp8_matmul(q.float(), s, w, ws),
                lambda: pkg.fp8_matmul(q[:, 1:129], s[:1].contiguous(), w[:, :128], ws[:1].contiguous()),
                lambda: pkg.fp8_matmul(q, s, w, ws, bias=torch.zeros(299, device="cuda")),
                lambda: pkg.fp8_matmul(q, s, w, ws, out=torch.empty(10, 300, device="cuda")),
                lambda: pkg.fp8_matmul(q, s, w, ws, torch.float32, out=torch.empty(300, 10, device="cuda").t()),
                lambda: pkg.fp8_linear(x[:, :128], w, ws), lambda: pkg.fp8_linear(x, w.cpu(), ws.cpu()),
                lambda: pkg.fp8_linear(x, w, ws, out=torch.empty(10, 299, device="cuda"))):
        with pytest.raises(n):
            bad()


def test_abi_refusals():
    """Every refusal comes before any device work (the pointers here are no device memory)."""
    L, ok = Bd.load(), 1 << 20

    def quant(x=ok, dtype=0, rows=10, cols=256, xs=256, br=1, tr=0, q=ok, qs=256, scale=ok):
        return L.mh3a_fp8_quantize(x, dtype, rows, cols, xs, br, tr, q, qs, scale, None)

    for kw in (dict(x=None), dict(q=None), dict(scale=None), dict(dtype=3), dict(dtype=-1), dict(br=2), dict(br=0), dict(tr=2),
               dict(xs=-1), dict(qs=255), dict(qs=240), dict(q=ok + 8), dict(x=ok + 2), dict(scale=ok + 2), dict(tr=1, rows=300)):
        assert quant(**kw) == 1, kw
    for kw in (dict(rows=0), dict(cols=0), dict(rows=(1 << 30) + 1), dict(rows=1 << 30, cols=1 << 20, qs=1 << 20)):
        assert quant(**kw) == 3, kw

    def mm(a=ok, as_=256, sa=ok, b=ok, bs=256, sb=ok, br=128, M=10, N=300, K=256, bias=None, dt=0, out=ok, os=300):
        return L.mh3a_fp8_matmul(a, as_, sa, b, bs, sb, br, M, N, K, bias, dt, out, os, None)

    for kw in (dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(out=None), dict(as_=255), dict(as_=272 + 8), dict(bs=128),
               dict(a=ok + 1), dict(b=ok + 8), dict(br=64), dict(dt=3), dict(os=299), dict(out=ok + 2), dict(bias=ok + 2),
               dict(as_=1 << 40), dict(sa=ok + 1)):
        assert mm(**kw) == 1, kw
    for kw in (dict(M=0), dict(N=0), dict(K=0), dict(M=1 << 30, N=1 << 30, os=1 << 30), dict(M=(1 << 30) + 1)):
        assert mm(**kw) == 3, kw

    def lin(x=ok, dt=2, xs=256, w=ok, ws=256, sw=ok, br=128, M=10, N=300, K=256, bias=None, y=ok, ys=300, wk=ok,
            n=L.mh3a_fp8_linear_workspace(10, 300, 256)):
        return L.mh3a_fp8_linear(x, dt, xs, w, ws, sw, br, M, N, K, bias, y, ys, wk, n, None)

    for kw in (dict(x=None), dict(w=None), dict(sw=None), dict(y=None), dict(wk=None), dict(wk=ok + 8), dict(n=10), dict(xs=-1),
               dict(x=ok + 1), dict(dt=7), dict(ws=128), dict(ys=10), dict(br=3)):
        assert lin(**kw) == 1, kw
    assert lin(M=0) == 3 and lin(K=0) == 3
    size = L.mh3a_fp8_linear_workspace
    assert size(4, 300, 256) == 0 and size(5, 300, 256) >= 5 * (256 + 8) and size(1, 8192, 8192) >= 8192 + 64 * 4
    assert size(0, 300, 256) == 0 and size(9, 300, -1) == 0 and size(9, 0, 256) == 0


def test_exports():
    assert {"mh3a_fp8_quantize", "mh3a_fp8_matmul", "mh3a_fp8_linear", "mh3a_fp8_linear_workspace"} <= set(Bd.EXPORTS)
    assert C.sizeof(Bd.mh3a_norm) == 72


@pytest.mark.gpu
@pytest.mark.parametrize("M", (2, 300))
def test_an_output_over_an_operand_is_refused(M):
    x = rand(M, 256)
    w, sw = pkg.fp8_quantize(rand(256, 256), block_rows=128)
    q, s = pkg.fp8_quantize(x)
    over = q.view(torch.float32).as_strided((M, 64), (64, 1))
    wn, swn = w[:64], sw[:, :1].contiguous()
    for bad in (lambda: pkg.fp8_linear(x, w, sw, out=x), lambda: pkg.fp8_matmul(q, s, wn, swn, torch.float32, out=over)):
        with pytest.raises(pkg.MH3AError, match="overlaps") as e:
            bad()
        assert e.value.status == 1
    # columns of one buffer side by side
    buf = torch.cat((x, torch.zeros_like(x)), 1)
    assert torch.equal(pkg.fp8_linear(buf[:, :256], w, sw, out=buf[:, 256:]), pkg.fp8_linear(x, w, sw))


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """Matrices of more than 2^31 elements, and rows far apart: the last rows are where they belong."""
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = (1 << 21) + 5
    x = torch.empty(rows, 1024, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    for block_rows in (1, 128):
        q, s = pkg.fp8_quantize(x, block_rows=block_rows)
        last = x[rows - 133:]  # from a block's first row
        rq, rs, _ = R.quantize(last, block_rows)
        assert torch.equal(q[rows - 133:].float().double(), rq)
        assert torch.equal((s[:, rows - 133:] if block_rows == 1 else s[:, -2:]).double(), rs)
        q, s = pkg.fp8_quantize(x, block_rows=block_rows, transpose=True)
        rq, rs, _ = R.quantize(last.t(), block_rows)
        assert torch.equal(q[:, rows - 133:].float().double(), rq) and torch.equal(s[-2:].double(), rs)
    del q, s, rq
    M, N, K = (1 << 20) + 3, 2056, 136
    a, sa = pkg.fp8_quantize(x.view(-1)[:M * K].view(M, K))
    b, sb = pkg.fp8_quantize(x[:N, :K], block_rows=128)
    out = pkg.fp8_matmul(a, sa, b, sb)
    for k in (0, M - 131):
        check_product(out[k:][:131], a[k:][:131], sa[:, k:][:, :131].contiguous(), b, sb)
    del out
    # 3 rows 2^30 and more elements apart: one layer of few rows, one of more
    wide = x.view(-1).as_strided((3, 1024), ((1 << 30) + 16, 1))
    w, sw = pkg.fp8_quantize(x[:200, :1024], block_rows=1)
    assert torch.equal(pkg.fp8_linear(wide, w, sw), pkg.fp8_linear(wide.contiguous(), w, sw))
    store = torch.empty(3 * (1 << 30), device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    far = store.as_strided((3, 1024), ((1 << 30) + 16, 1))
    far.copy_(w[:3])
    sf = sw[:, :3].contiguous()
    assert torch.equal(pkg.fp8_matmul(w, sw, far, sf), pkg.fp8_matmul(w, sw, w[:3], sf))
    assert torch.equal(pkg.fp8_matmul(far, sf, w, sw), pkg.fp8_matmul(w[:3], sf, w, sw))
    assert torch.equal(pkg.fp8_linear(x[:2], far, sf), pkg.fp8_linear(x[:2], w[:3], sf))


@pytest.mark.gpu
@pytest.mark.parametrize("name", ("w_scale", "bias", "a_scale"))
def test_an_output_over_scales_or_bias_is_refused(name):
    M, N, K = 20, 256, 256
    x = rand(M, K)
    w, sw = pkg.fp8_quantize(rand(N, K, seed=1), block_rows=128)
    q, s = pkg.fp8_quantize(x)
    bias = rand(N, seed=2)
    buf = torch.zeros(M * N + 2 * N, device="cuda")
    out = buf[N:-N].view(M, N)

    def calls(at):
        like = dict(w_scale=sw, bias=bias, a_scale=s)[name]
        part = buf[N + at:][:like.numel()].view(like.shape)
        part.copy_(like)
        kw = {"w_scale": sw, "bias": bias, "a_scale": s, name: part}
        if name != "a_scale":
            yield lambda: pkg.fp8_linear(x, w, kw["w_scale"], kw["bias"], out=out)
        yield lambda: pkg.fp8_matmul(q, kw["a_scale"], w, kw["w_scale"], torch.float32, bias=kw["bias"], out=out)

    names = dict(w_scale="(w|b)_scale", bias="bias", a_scale="a_scale")
    for at in (0, 1000, M * N - 1):
        for call in calls(at):
            with pytest.raises(pkg.MH3AError, match="out overlaps " + names[name]) as e:
                call()
            assert e.value.status == 1
    want = pkg.fp8_linear(x, w, sw, bias)
    for call in calls(M * N):  # side by side
        assert torch.equal(call(), want)


@pytest.mark.gpu
def test_views_of_one_buffer_are_refused_where_they_meet():
    """Random rows with gaps of one buffer as input and output: refused if, and only if, they share an element."""
    rng = random.Random(6)
    buf = torch.randn(6000, device="cuda")
    met = 0
    for _ in range(400):
        M, N, K = rng.choice([(1, 8, 24), (6, 8, 8), (5, 16, 24), (9, 24, 8)])
        w, sw = pkg.fp8_quantize(rand(N, K, seed=K), block_rows=128)
        xs = rng.choice([0, 5, K, K + N, 64, 96])
        os = rng.choice([N, N + 3, K + N, xs if xs >= N else 64, 96])
        x = buf.as_strided((M, K), (xs, 1), rng.randrange(1200))
        out = buf.as_strided((M, N), (os, 1), rng.randrange(1200))
        if places(x) & places(out):
            met += 1
            with pytest.raises(pkg.MH3AError, match="out overlaps x"):
                pkg.fp8_linear(x, w, sw, out=out)
        else:
            want = pkg.fp8_linear(x, w, sw)
            assert torch.equal(pkg.fp8_linear(x, w, sw, out=out), want)
            buf.normal_()
    assert met > 40


@pytest.mark.gpu
@pytest.mark.parametrize("K", (128, 40))
def test_gradients_are_not_lost_without_a_word(K):
    """Where autograd is recording, results lead back to a node that raises; elsewhere they are plain."""
    x, bias = rand(6, K), rand(32, seed=3)
    w, sw = pkg.fp8_quantize(rand(32, K, seed=1), block_rows=128)
    q, s = pkg.fp8_quantize(x)
    assert not any(t.requires_grad for t in (w, sw, q, s, pkg.fp8_linear(x, w, sw, bias)))

    def req(t):
        return t.clone().requires_grad_()

    for call, used in ((lambda: pkg.fp8_linear(req(x), w, sw), "fp8_linear"), (lambda: pkg.fp8_linear(x, w, req(sw)), "fp8_linear"),
                       (lambda: pkg.fp8_linear(x, w, sw, req(bias)), "fp8_linear"),
                       (lambda: pkg.fp8_matmul(q, req(s), w, sw), "fp8_matmul"),
                       (lambda: pkg.fp8_matmul(q, s, w, sw, bias=req(bias)), "fp8_matmul"),
                       (lambda: pkg.fp8_quantize(req(x))[0], "fp8_quantize"), (lambda: pkg.fp8_quantize(req(x))[1], "fp8_quantize"),
                       (lambda: pkg.fp8_linear(x, *pkg.fp8_quantize(req(rand(32, K)), block_rows=128)), "fp8_linear")):
        with pytest.raises(RuntimeError, match=f"mh3a_{used} records no gradient"):
            call().float().sum().backward()
        with torch.no_grad():
            assert not call().requires_grad
    out = torch.empty(6, 32, device="cuda")
    with pytest.raises(pkg.MH3AError, match="out cannot be given"):
        pkg.fp8_linear(req(x), w, sw, out=out)
    assert torch.equal(pkg.fp8_linear(x, w, sw, out=out), pkg.fp8_linear(x, w, sw))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("M", (1, 2, 3, 4, 5, 200))
def test_linear_of_large_and_small_values(M, dtype):
    """Results within fp32's range, from operands whose products with the stored numbers (up to 448) or with each
    other's scales are not."""
    for up, down in ((36, 0), (30, -30), (-30, 30), (-18, -3), (37, -37)):
        x = rand(M, 300, seed=M, spread=0.3) * 10.0 ** up
        w = pkg.fp8_quantize(rand(80, 300, seed=1, spread=0.3) / 16 * 10.0 ** down, block_rows=128)
        x = x.to(TYPES[dtype])
        y = pkg.fp8_linear(x, *w)
        assert bool(torch.isfinite(y).all())
        xq, xs, _ = R.quantize(x, 1)
        check_product(y, xq.float(), xs.float(), *w)


@pytest.mark.gpu
def test_linear_of_rows_far_apart():
    """Three rows more than 2^30 elements apart in a layer that is too large for the kernel of few rows, so that they are
    quantised by a launch of its own; and the output's rows as far apart."""
    far, N, K = (1 << 30) + 16, 16384, 1024
    assert Bd.load().mh3a_fp8_linear_workspace(3, N, K) > 0
    store = torch.empty(2 * far + N, device="cuda", dtype=torch.bfloat16)
    x = store.as_strided((3, K), (far, 1))
    x.copy_(rand(3, K, seed=1))
    w, sw = pkg.fp8_quantize(rand(N, K, seed=2), block_rows=128)
    want = pkg.fp8_linear(x.contiguous(), w, sw)
    assert torch.equal(pkg.fp8_linear(x, w, sw), want)
    xq, xs, _ = R.quantize(x, 1)
    check_product(want, xq.float(), xs.float(), w, sw)
    near = x.contiguous()
    out = store.as_strided((3, N), (far, 1))
    pkg.fp8_linear(near, w, sw, out=out)
    assert torch.equal(out, want)
