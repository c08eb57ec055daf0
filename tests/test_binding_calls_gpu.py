"""What a call through the direct binding, or past it, does to its process:
version counters, errors, other threads."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bwd_rms_norm_gb300 as lib
    lib.load_library()
    assert lib._binding is not None, "the direct binding is not built"
    return lib


@pytest.mark.parametrize("direct", [True, False])
def test_outputs_that_are_given_count_a_version(L, monkeypatch, direct):
    """Autograd notices that a tensor which a graph has saved was written."""
    if not direct:
        monkeypatch.setattr(L, "_binding", None)
    x, r = torch.randn(6, 64, device="cuda"), torch.randn(6, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    outs = [torch.zeros_like(x), torch.zeros_like(x), *torch.zeros(2, 6, device="cuda")]
    leaf = torch.ones(6, 64, device="cuda", requires_grad=True)
    loss = (leaf * outs[1]).sum()
    before = [o._version for o in outs]
    L.rms_norm_block_fwd(x, r, w, None, w, 1e-6, 0, 1.0, 1.0, *outs)
    assert all(o._version > v for o, v in zip(outs, before))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    r, y, r1, r2 = outs
    dx, dres = torch.zeros_like(x), torch.zeros_like(x)
    before = [t._version for t in (dx, dres, x, r)]
    L.rms_norm_block_bwd(x, r, x, r, r1, r2, w, None, w, dx=dx, dresidual=dres)
    after = [t._version for t in (dx, dres, x, r)]
    assert after[0] > before[0] and after[1] > before[1] and after[2:] == before[2:]
    norm = torch.zeros((), device="cuda")
    v = norm._version
    L.rms_norm_grad_norm([x], norm=norm)
    assert norm._version > v
    v = norm._version
    L.rms_norm_grad_clip([x.clone()], 1.0, norm=norm)
    assert norm._version > v
    with torch.inference_mode():                                 # these have no counter
        outs = [torch.zeros_like(x), torch.zeros_like(x), *torch.zeros(2, 6, device="cuda")]
        dx = torch.zeros_like(x)
    L.rms_norm_block_fwd(x, dres, w, None, w, 1e-6, 0, 1.0, 1.0, *outs)
    L.rms_norm_block_bwd(x, dres, x, outs[0], outs[2], outs[3], w, None, w, dx=dx)
