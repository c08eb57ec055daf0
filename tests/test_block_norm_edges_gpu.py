"""The block norm where its values leave the usual range.  Tolerances are those
of test_block_norm_gpu.py, against the same float64 oracle."""
import pytest
import torch

from test_block_norm_gpu import check_backward, check_forward, cuda, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bwd_rms_norm_gb300 as lib
    lib.load_library()
    return lib


# narrow rows, one CTA a row, rows over a cluster, odd widths, single-element loops
@pytest.mark.parametrize("rows,hidden,kernel", [
    (2500, 512, "block_bwd_tma"), (9, 1024, "block_bwd_tma"), (40, 4096, "block_bwd_tma"),
    (7, 12288, "block_bwd_tma"), (300, 1001, "block_bwd_tma"), (140, 12001, "block_bwd_tma"),
    (9, 1001, "block_bwd_loop")])
@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("large,up", [(126, 0), (120, 10), (110, 16), (70, 16), (-60, -80)])
def test_backward_of_rows_beyond_fp32_squares(L, rows, hidden, kernel, dtype, res, large, up):
    """Rows that the forward takes although their squares overflow fp32: the
    backward's sums over them, of order 1 after the norm, do not.  Nor do those
    over small rows under small gradients vanish."""
    eps = 1e-5 if large > 0 else 0.0
    d, g = make(rows, hidden, dtype, res, True, 1, True, seed=hidden + large)
    x = d["x"].float()
    x = torch.copysign(1 + x.abs() / 16, x) * 2.0 ** large      # 1 to 1.5 times 2^large
    d["x"][::2] = x[::2].to(d["x"].dtype)
    for k in g:
        g[k] = g[k] * 2.0 ** up
    dc, gc = cuda(d), cuda(g)
    out = L.rms_norm_block_fwd(**dc, eps=eps)
    check_forward(out, d, eps, 0, 1.0, 1.0)
    for dr in (True, False):
        g1 = g if dr else dict(g, dresidual_out=None)
        back = L.rms_norm_block_bwd(gc["dy"], gc["dresidual_out"] if dr else None, dc["x"], out[0],
                                    out[2], out[3], dc["post_gamma"], dc["gate"],
                                    dc["next_gamma"])
        assert kernel in L.last_kernels()[0], L.last_kernels()
        check_backward(back, d, g1, out[0], out[2], out[3], 0, 1.0, 1.0)
