"""Refusals of the block norm's Python calls, and rules its sources keep."""
import os
import re

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


@pytest.mark.parametrize("offset", [0.5, 1.9, -0.5, 2, -1, float("nan"), "1"])
def test_offsets_that_are_neither_0_nor_1(L, offset):
    """Refused as such, not cut to a whole number."""
    x, w, s = torch.zeros(4, 8), torch.ones(8), torch.ones(4)
    for call in (lambda: L.rms_norm_block_fwd(x, x, w, None, w, 1e-6, offset),
                 lambda: L.rms_norm_block(x, x, w, None, w, 1e-6, offset),
                 lambda: L.rms_norm_block_bwd(x, x, x, x, s, s, w, None, w, offset)):
        with pytest.raises(L.RMSNormError, match="offset") as e:
            call()
        assert e.value.status == 8


@pytest.mark.parametrize("offset", [0, 1, 0.0, 1.0, True, False])
def test_offsets_that_are_0_or_1(L, offset):
    x, w = torch.zeros(4, 8), torch.ones(8)
    with pytest.raises(RuntimeError, match="CUDA"):              # past the offset
        L.rms_norm_block_fwd(x, x, w, None, w, 1e-6, offset)


@pytest.mark.parametrize("source", ["block_fwd_tma.cu", "block_bwd_tma.cuh"])
def test_order_of_the_odd_widths_copies(source):
    """A stage of odd rows is filled by the lanes of a warp, of which lane 0
    alone waits for the stage and arrives on its barrier.  Shuffles and warp
    reductions do not order memory, so a __syncwarp stands after the wait, before
    the arrival (the tails stored by other lanes), and after it (the copies)."""
    import bwd_rms_norm_gb300 as lib
    path = os.path.join(os.path.dirname(lib.LIB_PATH), "csrc", source)
    text = re.sub(r"//[^\n]*", "", open(path).read())
    told = text.index("__shfl_sync(0xffffffffu, go, 0)")
    assert re.match(r"[^;]*\)\) break;\s*(if \(EDGE\) )?__syncwarp\(\);", text[told:])
    tails = [m.start() for m in re.finditer(r"\bcopy_tail\(", text)]
    arrive = text.index("mbar_arrive_expect_tx(full, bytes)")
    copies = text.index("copy_row(", arrive)
    assert tails and max(tails) < arrive
    assert "__syncwarp();" in text[max(tails):arrive]
    assert "__syncwarp();" in text[arrive:copies]
