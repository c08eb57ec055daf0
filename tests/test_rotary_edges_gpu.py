"""Calls of the head norm with rotation at its edges: frequencies of the user's own."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bwd_rms_norm_gb300 as lib
    lib.load_library()
    return lib


def test_assigned_frequencies_move_to_the_gpu(L):
    m = L.RMSNormRotary(64, base=500000.0, rotary_dim=32)
    want = m.inv_freq / 8
    m.inv_freq = want.clone()
    m = m.cuda().bfloat16()
    assert m.inv_freq.dtype == torch.float64 and m.inv_freq.is_cuda
    assert torch.equal(m.inv_freq.cpu(), want)
    x = torch.randn((2, 9, 6, 64), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q, k = x[:, :, :4], x[:, :, 4:]
    got = m(q, k)
    ref = L.rms_norm_rotary_fwd(q, k, m.q_weight, m.k_weight, want.cuda())
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
