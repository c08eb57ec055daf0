"""Host-side checks of the gradient norm and clip: refusals before any CUDA call."""
import ctypes
import os

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    import bwd_rms_norm_gb300 as lib
    from bwd_rms_norm_gb300 import build
    if not os.path.exists(lib.LIB_PATH):
        build.build()
    lib.load_library()
    return lib


FAKE, NULL = ctypes.c_void_p(0x10000), None   # never dereferenced


def arrays(ptrs, numels, codes):
    n = len(ptrs)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numels), (ctypes.c_int * n)(*codes))


def norm(L, ptrs=(0x1000, 0x2000), numels=(8, 8), codes=(0, 1), count=None, out=FAKE, ws=FAKE,
         ws_bytes=1 << 20):
    p, n, c = arrays(ptrs, numels, codes)
    return L.load_library().rms_norm_grad_norm(p, n, c, len(ptrs) if count is None else count, out,
                                               ws, ws_bytes, None)


def clip(L, ptrs=(0x1000, 0x2000), numels=(8, 8), codes=(0, 1), outs=None, out_codes=None,
         count=None, max_norm=1.0, eps=1e-6, total=NULL, out=FAKE, ws=FAKE, ws_bytes=1 << 20):
    p, n, c = arrays(ptrs, numels, codes)
    o, _, oc = arrays(outs or ptrs, numels, out_codes or codes)
    return L.load_library().rms_norm_grad_clip(p, n, c, o, oc, len(ptrs) if count is None else count,
                                               max_norm, eps, total, out, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [norm, clip])
def test_shared_refusals(L, call):
    assert call(L, count=-1) == 2
    assert call(L, numels=(8, -1)) == 2
    assert call(L, numels=(8, (1 << 42) + 1)) == 2
    assert call(L, numels=(1 << 41, (1 << 41) + 1)) == 2       # together too many
    assert call(L, codes=(0, 3)) == 4
    assert call(L, codes=(-1, 0)) == 4
    assert call(L, ptrs=(0x1000, None)) == 1
    assert call(L, ptrs=(0x1002, 0x2000)) == 5                   # fp32 off its alignment
    assert call(L, ptrs=(0x1000, 0x2001)) == 5                   # bf16 off its alignment
    assert call(L, out=NULL) == 1
    assert call(L, ws=NULL) == 1
    assert call(L, ws=ctypes.c_void_p(0x1008)) == 5
    assert call(L, ws_bytes=L.rms_norm_grad_workspace_size(2) - 1) == 6


def test_clip_refusals(L):
    for m in (-1.0, float("nan")):
        assert clip(L, max_norm=m) == 8
    for e in (-1e-6, float("nan"), float("inf")):
        assert clip(L, eps=e) == 3
    assert clip(L, out_codes=(1, 1)) == 4                        # fp32 into bf16
    assert clip(L, out_codes=(0, 2)) == 4                        # bf16 into fp16
    # a tensor twice, two that overlap, an output in another's gradient
    assert clip(L, ptrs=(0x1000, 0x1000), codes=(0, 0)) == 8
    assert clip(L, ptrs=(0x1000, 0x101c), codes=(0, 0)) == 8
    assert clip(L, codes=(0, 0), outs=(0x2000, 0x3000)) == 8
    assert clip(L, codes=(0, 0), outs=(0x8000, 0x8010)) == 8
    assert clip(L, codes=(1, 1), outs=(0x1000, 0x8000), out_codes=(0, 1)) == 8  # wider, in place
    assert clip(L, codes=(0, 0), outs=(0x101c, 0x8000)) == 8      # shifted in place
    assert clip(L, total=FAKE, ws=NULL, outs=(0x1010, 0x8000)) == 8


def test_workspace_size(L):
    size = L.rms_norm_grad_workspace_size
    assert size(1) == size(1024) == 1216 * 16
    assert size(1025) == size(2048) == 2 * 1216 * 16
    assert size(-1) == 0


def test_python_refusals(L):
    z = torch.zeros
    with pytest.raises(RuntimeError, match="CUDA"):
        L.rms_norm_grad_norm([z(3)])
    with pytest.raises(RuntimeError, match="CUDA"):
        L.rms_norm_grad_clip([z(3)], 1.0)
    with pytest.raises(RuntimeError, match="empty"):
        L.rms_norm_grad_norm([])
    with pytest.raises(RuntimeError, match="empty"):
        L.rms_norm_grad_clip(iter(()), 1.0)
    with pytest.raises(RuntimeError, match="float32, bfloat16"):
        L.rms_norm_grad_norm(z(3, dtype=torch.float64))
    with pytest.raises(RuntimeError, match="1 tensors"):
        L.rms_norm_grad_clip([z(3), z(3)], 1.0, out=[z(3)])
    with pytest.raises(RuntimeError, match="elements"):
        L.rms_norm_grad_clip([z(3)], 1.0, out=[z(4)])
    with pytest.raises(RuntimeError, match="bfloat16"):
        L.rms_norm_grad_clip([z(3, dtype=torch.bfloat16)], 1.0, out=[z(3, dtype=torch.float16)])
