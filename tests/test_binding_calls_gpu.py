"""What a call through the direct binding, or past it, does to its process:
version counters, errors, other threads."""
import ctypes
import subprocess
import threading
import time

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


STUB = r"""
#include <stddef.h>
#include <unistd.h>
volatile int calls, status, released, waits, saw;
/* In place of a C entry point: counts, and answers with `status`; where `waits`
   is set it first waits for another thread's `released`, 2 s at most, and says
   whether it saw it. */
int entry(void) {
  ++calls;
  for (int ms = 0; waits && !released && ms < 2000; ++ms) usleep(1000);
  saw = released;
  return status;
}
size_t workspace(void) { return 64; }
"""


@pytest.fixture(scope="module")
def stub(tmp_path_factory):
    """A library of entry points that launch nothing."""
    d = tmp_path_factory.mktemp("stub")
    (d / "stub.c").write_text(STUB)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", str(d / "stub.c"), "-o",
                    str(d / "stub.so")], check=True)
    return ctypes.CDLL(str(d / "stub.so"))


@pytest.fixture
def stubbed(L, stub):
    """The binding on the stub's entry points, its counters at zero."""
    at = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    entry, workspace = at(stub.entry), at(stub.workspace)
    names = ("calls", "status", "released", "waits", "saw")
    v = {k: ctypes.c_int.in_dll(stub, k) for k in names}
    for c in v.values():
        c.value = 0
    L._binding.init(entry, entry, workspace, entry, entry, workspace)
    yield v
    L._load_binding(L.load_library())


def calls_of(L):
    x, w, s = torch.ones(4, 8, device="cuda"), torch.ones(8, device="cuda"), torch.ones(
        4, device="cuda")
    return {"rms_norm_block_fwd": lambda: L.rms_norm_block_fwd(x, x, w, None, w),
            "rms_norm_block_bwd": lambda: L.rms_norm_block_bwd(x, x, x, x, s, s, w, None, w),
            "rms_norm_grad_norm": lambda: L.rms_norm_grad_norm([x]),
            "rms_norm_grad_clip": lambda: L.rms_norm_grad_clip([x], 1e-3)}, x


@pytest.mark.parametrize("name", ["rms_norm_block_fwd", "rms_norm_block_bwd",
                                  "rms_norm_grad_norm", "rms_norm_grad_clip"])
def test_a_failed_launch_is_not_made_again(L, stubbed, name):
    """A call that failed on its way may have scaled some tensors already: its
    error is raised, and nothing runs a second time."""
    calls, x = calls_of(L)
    stubbed["status"].value = 7
    with pytest.raises(L.RMSNormError, match=name + ".*status 7") as e:
        calls[name]()
    assert e.value.status == 7 and stubbed["calls"].value == 1
    assert bool((x == 1).all())


@pytest.mark.parametrize("name", ["rms_norm_block_fwd", "rms_norm_block_bwd",
                                  "rms_norm_grad_norm", "rms_norm_grad_clip"])
def test_other_threads_run_during_a_call(L, stubbed, name):
    """A launch that waits for room in its queue, say, holds up its thread alone."""
    calls, _ = calls_of(L)
    stubbed["waits"].value = 1

    def release():
        while stubbed["calls"].value == 0:
            time.sleep(0.001)
        stubbed["released"].value = 1

    other = threading.Thread(target=release)
    other.start()
    try:
        calls[name]()
    finally:
        stubbed["calls"].value += 1
        other.join()
    assert stubbed["calls"].value == 2 and stubbed["saw"].value == 1


def test_lists_that_change_during_a_call(L, stubbed):
    """The call keeps what it read: another thread may empty the lists."""
    stubbed["waits"].value = 1
    grads = [torch.ones(8, device="cuda") for _ in range(3)]
    out = [torch.ones(8, device="cuda") for _ in range(3)]
    kept = list(out)

    def release():
        while stubbed["calls"].value == 0:
            time.sleep(0.001)
        grads.clear()
        out.clear()
        stubbed["released"].value = 1

    before = [o._version for o in out]
    other = threading.Thread(target=release)
    other.start()
    try:
        L.rms_norm_grad_clip(grads, 1.0, out=out)
    finally:
        stubbed["calls"].value += 1
        other.join()
    assert stubbed["saw"].value == 1 and not grads
    assert all(o._version > v for o, v in zip(kept, before))
