"""The operators' waits when what they wait for comes late or never: they end, and say so."""
import ctypes as C
import os
import subprocess

import pytest
import torch

from bigvgan_waveform_decoder_b200 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    """bounded_waits.cu, which includes the library's device code."""
    if not os.path.exists(B.NVCC):
        pytest.skip("no nvcc")
    lib = str(tmp_path_factory.mktemp("waits") / "bounded_waits.so")
    subprocess.run([B.NVCC, *B.FLAGS, "-I", B.CSRC, "-shared", os.path.join(HERE, "bounded_waits.cu"), "-o", lib], check=True)
    return C.CDLL(lib)


@pytest.mark.gpu
@pytest.mark.parametrize("slow", (0, 3))
def test_blocks_of_a_cluster_outlive_what_late_peers_send(waits, slow):
    """A block that gave up its wait stays until a late peer's sums have landed in its shared memory."""
    out = torch.full((20,), -1, dtype=torch.int32, device="cuda")
    assert waits.run_peers(slow, 0, C.c_void_p(out.data_ptr())) == 0
    arrived, inbox = out[:4].tolist(), out[4:].view(4, 4).tolist()
    assert arrived == [int(k == slow) for k in range(4)]  # the late one finds the others' sums at once
    assert inbox == [[1, 2, 3, 4]] * 4


@pytest.mark.gpu
def test_a_cluster_whose_peer_never_sends_ends(waits):
    out = torch.full((20,), -1, dtype=torch.int32, device="cuda")
    assert waits.run_peers(2, 1, C.c_void_p(out.data_ptr())) == 0
    assert out[:4].tolist() == [0] * 4 and out[4:].view(4, 4).tolist() == [[1, 2, 0, 4]] * 4


@pytest.mark.gpu
def test_a_cluster_without_a_late_peer_does_not_give_up(waits):
    out = torch.full((20,), -1, dtype=torch.int32, device="cuda")
    assert waits.run_peers(-1, 0, C.c_void_p(out.data_ptr())) == 0
    assert out[:4].tolist() == [1] * 4 and out[4:].view(4, 4).tolist() == [[1, 2, 3, 4]] * 4


@pytest.mark.gpu
def test_a_warp_gives_up_together(waits):
    """Lanes whose limits run out at different times get one answer, so that no lane goes on alone."""
    out = torch.full((64,), -1, dtype=torch.int32, device="cuda")
    assert waits.run_warp(C.c_void_p(out.data_ptr())) == 0
    assert out.tolist() == [0] * 32 + [1] * 32
