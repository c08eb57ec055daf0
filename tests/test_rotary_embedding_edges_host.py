"""Calls of the head norm's and the embedding's modules and functions that need no
GPU, and that a user makes beside the usual ones."""
import copy
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


@pytest.mark.parametrize("dtype", [torch.float64, torch.float32])
def test_frequencies_that_were_assigned_stay(L, dtype):
    """Scaled frequencies, as of a longer context, outlive a cast and a move."""
    m = L.RMSNormRotary(64, base=500000.0, rotary_dim=32)
    want = (m.inv_freq / 8).to(dtype)
    m.inv_freq = want.clone()
    holder = torch.nn.Sequential(m)
    for change in (lambda t: t.to(torch.bfloat16), lambda t: t.half(), lambda t: t.float(),
                   lambda t: t.cpu(), lambda t: t.double(), copy.deepcopy,
                   lambda t: t.to_empty(device="cpu")):
        holder = change(holder)
        kept = holder[0].inv_freq
        assert kept.dtype == dtype and torch.equal(kept, want)
    assert "inv_freq" not in holder[0].state_dict()
    # values changed in place, and the same memory where nothing moves
    m = L.RMSNormRotary(64)
    at = m.inv_freq.data_ptr()
    m.inv_freq.mul_(0.25)
    want = m.inv_freq.clone()
    assert torch.equal(m.bfloat16().inv_freq, want) and m.inv_freq.data_ptr() == at


def test_frequencies_of_a_module_made_without_memory(L):
    m = L.RMSNormRotary(64, base=500000.0, rotary_dim=32, device="meta")
    assert m.bfloat16().inv_freq.is_meta
    m = m.to_empty(device="cpu")
    want = 500000.0 ** (torch.arange(16, dtype=torch.float64) * (-2.0 / 32))
    assert m.inv_freq.dtype == torch.float64 and torch.equal(m.inv_freq, want)
    # assigned ones that have values are kept on the way
    m = L.RMSNormRotary(64, rotary_dim=32, device="meta")
    m.inv_freq = want / 3
    assert torch.equal(m.to_empty(device="cpu").inv_freq, want / 3)


def test_padding_outside_the_table_is_refused_with_the_call(L):
    """Not by the backward alone, in the middle of a step."""
    ids, w = torch.zeros(4, dtype=torch.int64), torch.zeros(8, 16, requires_grad=True)
    for pad in (-1, 8, 1 << 40):
        with pytest.raises(L.RMSNormError) as e:
            L.rms_norm_embedding(ids, w, padding_idx=pad)
        assert e.value.status == 8
    for pad in (None, 0, 7):                # refused for another reason: not on a GPU
        with pytest.raises(RuntimeError, match="CUDA tensor"):
            L.rms_norm_embedding(ids, w, padding_idx=pad)
