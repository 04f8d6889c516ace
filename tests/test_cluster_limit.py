"""Group norm where a device places smaller clusters than a whole B200: the call goes another way, not wrong."""
import ctypes as C
import os
import subprocess
import sys

import pytest
import torch

from bigvgan_waveform_decoder_b200 import binding as Bd
from bigvgan_waveform_decoder_b200 import build as B

from .test_norm_ops import case, check_backward, check_forward, norm

HERE = os.path.dirname(os.path.abspath(__file__))
NAMES = ("mh3a_group_norm_act_workspace", "mh3a_group_norm_act", "mh3a_group_norm_act_backward")
DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    """The norm's own source with its limit within reach."""
    if not os.path.exists(B.NVCC):
        pytest.skip("no nvcc")
    so = str(tmp_path_factory.mktemp("limit") / "cluster_limit.so")
    subprocess.run([B.NVCC, *B.FLAGS, "-I", B.CSRC, "-shared", os.path.join(HERE, "cluster_limit.cu"), "-o", so], check=True)
    L, real = C.CDLL(so), Bd.load()
    for n in NAMES:
        getattr(L, n).argtypes, getattr(L, n).restype = getattr(real, n).argtypes, getattr(real, n).restype
    return L


@pytest.fixture
def limited(lib):
    yield lib
    lib.set_cluster_limit(0)


def test_scratch_where_large_clusters_cannot_be_placed(limited):
    """An item of 3001 rows of 200 channels in 16 bits, 1.2 MB, takes 16 blocks of 75 KB, or 8 of 150; fewer cannot
    hold it, and the call needs scratch memory."""
    p = C.byref(norm(B=7, T=3001, C=200, groups=8))
    size = limited.mh3a_group_norm_act_workspace
    for n in (16, 8):
        limited.set_cluster_limit(n)
        assert size(p, 0, 1) == 0
    for n in (4, 2, 1):
        limited.set_cluster_limit(n)
        assert size(p, 0, 1) > 0 and size(p, 0, 1) <= size(p, 0, 0)
    small = C.byref(norm(B=1, T=4, C=512, groups=32))
    assert size(small, 0, 1) == 0  # one block is enough


@pytest.mark.gpu
def test_a_whole_device_places_16(limited):
    limited.set_cluster_limit(0)
    assert limited.get_cluster_limit() == 16


@pytest.mark.gpu
@pytest.mark.parametrize("limit", (1, 2, 4, 8))
@pytest.mark.parametrize("shape", [(7, 3001, 200, 8), (2, 2000, 512, 32), (3, 900, 64, 4)], ids=str)
@pytest.mark.parametrize("dtype", ("fp32", "fp16"))
def test_results_with_smaller_clusters(limited, limit, shape, dtype):
    limited.set_cluster_limit(limit)
    Bn, T, Cn, G = shape
    x, w, b, al, be = case(Bn, T, Cn, "snake_beta", dtype, seed=limit)
    p = norm(dtype=DTYPE[x.dtype], act=2, B=Bn, T=T, C=Cn, groups=G)
    p.weight, p.bias, p.alpha, p.beta = (t.data_ptr() for t in (w, b, al, be))
    stream = torch.cuda.current_stream().cuda_stream

    def scratch(backward):
        n = limited.mh3a_group_norm_act_workspace(C.byref(p), backward, 1)
        return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"), n

    y, (ws, n) = torch.empty_like(x), scratch(0)
    mean, rstd = (torch.empty(Bn, G, device="cuda") for _ in range(2))
    assert limited.mh3a_group_norm_act(C.byref(p), x.data_ptr(), T * Cn, Cn, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                       ws.data_ptr(), n, stream) == 0
    check_forward(x, G, w, b, "snake_beta", al, be, got=(y, mean, rstd))
    dy, dx, (ws, n) = x.flip(1).contiguous(), torch.empty_like(x), scratch(1)
    g = [torch.empty(Cn, device="cuda") for _ in range(4)]
    assert limited.mh3a_group_norm_act_backward(C.byref(p), x.data_ptr(), T * Cn, Cn, dy.data_ptr(), T * Cn, Cn, mean.data_ptr(),
                                                rstd.data_ptr(), dx.data_ptr(), *(t.data_ptr() for t in g), ws.data_ptr(), n, stream) == 0
    check_backward(dy, x, mean, rstd, G, w, b, "snake_beta", al, be, got=(dx, *g))


@pytest.mark.gpu
@pytest.mark.parametrize("op", ("norm", "linear"))
def test_the_first_call_of_a_process_may_be_captured(op):
    """What a device is asked for once, and what is set up once for a kernel, does not get in a capture's way."""
    code = f"""
import torch, bigvgan_waveform_decoder_b200 as pkg
x = torch.randn(2, 900, 64, device="cuda")
q = torch.ones(64, 64, device="cuda").to(torch.float8_e4m3fn)
s = torch.ones(1, 1, device="cuda")
def call():
    if "{op}" == "norm":
        y, m, r = pkg.group_norm_act(x, 4)
        return y, pkg.group_norm_act_backward(x, x, m, r, 4)[0]
    return pkg.fp8_linear(x[0], q, s), pkg.fp8_linear(x[0, :1], q, s)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    outs = call()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(outs, call()))
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=B.ROOT, timeout=300)
