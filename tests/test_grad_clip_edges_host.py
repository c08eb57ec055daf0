"""Refusals of the gradient norm and clip before any CUDA call: a norm, a given
norm or a workspace that shares memory with the lists."""
import ctypes
import os

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    import bwd_rms_norm_gb300 as pkg
    from bwd_rms_norm_gb300 import build
    if not os.path.exists(pkg.LIB_PATH):
        build.build()
    return pkg.load_library()


# never dereferenced: 8 fp32 at 0x10000, 8 bf16 at 0x20000, outputs of 8 fp32 each
GRADS, OUTS = (0x10000, 0x20000), (0x30000, 0x40000)
BYTES = {0x10000: 32, 0x20000: 16, 0x30000: 32, 0x40000: 32}
NORM, TOTAL, WS, WS_BYTES = 0x50000, 0x60000, 0x100000, 1216 * 16


def arrays(outs=OUTS, codes=(0, 1), out_codes=(0, 0)):
    return ((P * 2)(*GRADS), (ctypes.c_int64 * 2)(8, 8), (ctypes.c_int * 2)(*codes),
            (P * 2)(*outs), (ctypes.c_int * 2)(*out_codes))


def norm(lib, at=NORM, ws=WS):
    g, n, c, _, _ = arrays()
    return lib.rms_norm_grad_norm(g, n, c, 2, P(at), P(ws), WS_BYTES, None)


def clip(lib, at=NORM, total=None, ws=WS, **k):
    g, n, c, o, oc = arrays(**k)
    return lib.rms_norm_grad_clip(g, n, c, o, oc, 2, 1.0, 1e-6, P(total), P(at), P(ws), WS_BYTES,
                                  None)


@pytest.mark.parametrize("k", [*GRADS, *OUTS])
def test_what_a_call_writes_beside_the_lists(lib, k):
    first, last = k, k + BYTES[k] - 4
    for at in (first, last):
        assert clip(lib, at=at) == 8, hex(at)                    # the norm in a list
        if k in GRADS:
            assert norm(lib, at=at) == 8, hex(at)
    for ws in (k, k - WS_BYTES + 16):
        assert clip(lib, ws=ws) == 8, hex(ws)                    # the workspace on a list
        if k in GRADS:
            assert norm(lib, ws=ws) == 8, hex(ws)
    if k in OUTS:
        for at in (first, last):
            assert clip(lib, total=at) == 8, hex(at)             # scaled while it is read
    for at in (GRADS[0], GRADS[0] + 28):
        assert clip(lib, total=at, outs=GRADS, out_codes=(0, 1)) == 8      # in place


def test_what_a_call_writes_on_itself(lib):
    for at in (WS, WS + WS_BYTES - 4):
        assert norm(lib, at=at) == 8 and clip(lib, at=at) == 8   # the norm in the workspace
    assert clip(lib, at=TOTAL + 2, total=TOTAL) == 8             # a part of the given norm
