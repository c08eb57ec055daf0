"""Python binding of the GB300 fused RMSNorm library (librms_norm_gb300.so).

Argument marshalling only: every step of the forward and the backward runs
in the library's CUDA kernels.  PyTorch supplies device memory and the
current CUDA stream.  There is no CPU fallback: without the built library,
or with tensors that are not on a CUDA device, every call raises.

The functions carry the names of the C entry points declared in
``include/rms_norm.h``:

* ``rms_norm_fwd(x, gamma, eps, offset=0, cast_mode="round_once")``
  -> ``(y, rstd)``
* ``rms_norm_bwd(dy, x, gamma, rstd, offset=0)`` -> ``(dx, dw)``
* ``rms_norm_bwd_workspace_size(rows, hidden, dtype)``
* ``rms_norm_status_string(status)``
* ``rms_norm_bwd_noalloc(dy, x, gamma, rstd, offset=0)`` -> ``(dx, dw)``
* ``rms_norm_bwd_blocked(dy, x, gamma, rstd, block_rows, offset=0)`` ->
  ``(dx, chunk_sums)``; ``rms_norm_dw_sum(chunk_sums)`` -> ``dw``;
  ``rms_norm_dw_chunk_count(rows, block_rows)``;
  ``rms_norm_bwd_blocked_workspace_size(rows, hidden, block_rows)``;
  ``rms_norm_rank_rows(rows, block_rows, world, rank)`` -> ``(lo, hi)`` (the
  weight gradient in an order that any split of the rows reproduces)
* ``rms_norm_set_sm_budget(sms)``, ``rms_norm_sm_budget()
* ``rms_norm_fwd_fp8(x, gamma, scale, eps, offset=0)`` -> ``(y8, rstd)``
  (``y8`` a torch.float8_e4m3fn tensor, ``scale`` a one-element fp32
  device tensor)
* ``softmax_fwd(x)`` -> ``y``; ``softmax_bwd(dy, y)`` -> ``dx`` (last
  dimension)
* ``group_norm_fwd(x, gamma, beta, groups, eps)`` -> ``(y, mean, rstd)``;
  ``group_norm_bwd(dy, x, gamma, mean, rstd, groups)`` ->
  ``(dx, dgamma, dbeta)`` (x of shape [n, channels, *spatial])
* ``layer_norm_fwd(x, gamma, beta, eps)`` -> ``(y, mean, rstd)``
* ``layer_norm_bwd(dy, x, gamma, mean, rstd)`` -> ``(dx, dgamma, dbeta)``
* ``rms_norm_block_fwd(x, residual, post_gamma, gate, next_gamma, eps, ...)``
  -> ``(residual_out, y, rstd_post, rstd_next)``; ``rms_norm_block_bwd(dy,
  dresidual_out, x, residual_out, rstd_post, rstd_next, ...)`` -> ``(dx,
  dresidual, dpost, dgate, dnext)``;
  ``rms_norm_block_bwd_workspace_size(rows, hidden, gate_rows)`` (the norms
  after and before a block with its gate and the scaled residual sum)
* ``rms_norm_grad_norm(grads)`` -> ``norm``; ``rms_norm_grad_clip(grads,
  max_norm, ...)`` -> ``norm`` (the 2-norm over a list of gradients, and the
  list scaled down to a largest norm); ``rms_norm_grad_workspace_size(count)``
* ``rms_norm_rotary_fwd(q, k, q_gamma, k_gamma, inv_freq, positions, ...)``
  -> ``(q_out, k_out, rstd_q, rstd_k)``; ``rms_norm_rotary_bwd(dq_out, dk_out,
  q, k, q_gamma, k_gamma, rstd_q, rstd_k, inv_freq, positions, ...)`` ->
  ``(dq, dk, dq_gamma, dk_gamma)``; ``rms_norm_rotary_bwd_workspace_size(batch,
  tokens, q_heads, k_heads, head_dim)`` (the norms of queries and keys over
  each head, with the rotation by the token's position)
* ``rms_norm_embedding_fwd(ids, weight, scale)`` -> ``y``;
  ``rms_norm_embedding_bwd(dy, ids, vocab, scale, ...)`` -> ``dweight``;
  ``rms_norm_embedding_bwd_workspace_size(tokens, vocab, hidden)`` (the rows of
  a table for a batch of tokens, and its gradient)

For autograd: ``rms_norm(x, weight, eps, offset=0, cast_mode="round_once")``
(a ``torch.autograd.Function`` over rms_norm_fwd / rms_norm_bwd) and the
module ``RMSNorm(hidden, eps, offset=0, cast_mode="round_once")``; likewise
``rms_norm_block`` and the module ``RMSNormBlock`` over rms_norm_block_fwd /
rms_norm_block_bwd, ``rms_norm_rotary`` and ``RMSNormRotary`` over
rms_norm_rotary_fwd / rms_norm_rotary_bwd, ``rms_norm_embedding`` and
``RMSNormEmbedding`` over rms_norm_embedding_fwd / rms_norm_embedding_bwd.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import importlib.util
import os
from typing import Optional, Tuple

import torch

LIB_NAME = "librms_norm_gb300.so"
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), LIB_NAME)
BINDING_PATH = os.path.join(os.path.dirname(LIB_PATH), "_binding.so")

# Values of the C enums (include/rms_norm.h).
RMSN_F32, RMSN_BF16, RMSN_F16 = 0, 1, 2
RMSN_ROUND_ONCE, RMSN_ROUND_TWICE = 0, 1
RMSN_OK = 0
RMSN_ERR_ARG = 8
RMSN_MAX_HIDDEN = 65536
RMSN_MAX_PARTIALS = 1024
RMSN_DW_CHUNK_BLOCKS = 32
RMSN_BLOCK_MAX_PARTIALS = 608
RMSN_ROTARY_MAX_DIM = 1024
RMSN_EMBEDDING_MAX_VOCAB = 1 << 30

DTYPE_CODES = {torch.float32: RMSN_F32, torch.bfloat16: RMSN_BF16, torch.float16: RMSN_F16}
CAST_MODES = {"round_once": RMSN_ROUND_ONCE, "round_twice": RMSN_ROUND_TWICE}

EXPORTED = (
    "rms_norm_fwd",
    "rms_norm_bwd_workspace_size",
    "rms_norm_bwd",
    "rms_norm_status_string",
    "rms_norm_last_cuda_error",
    "rms_norm_last_launch_count",
    "rms_norm_last_kernels",
    "rms_norm_bwd_noalloc",
    "rms_norm_bwd_blocked_workspace_size",
    "rms_norm_dw_chunk_count",
    "rms_norm_bwd_blocked",
    "rms_norm_dw_sum",
    "rms_norm_rank_rows",
    "rms_norm_set_sm_budget",
    "rms_norm_sm_budget",
    "rms_norm_wait_timeouts",
    "rms_norm_selftest_wait_limit",
    "rms_norm_fwd_fp8",
    "layer_norm_fwd",
    "layer_norm_bwd_workspace_size",
    "layer_norm_bwd",
    "softmax_fwd",
    "softmax_bwd",
    "group_norm_fwd",
    "group_norm_bwd_workspace_size",
    "group_norm_bwd",
    "rms_norm_block_fwd",
    "rms_norm_block_bwd_workspace_size",
    "rms_norm_block_bwd",
    "rms_norm_grad_workspace_size",
    "rms_norm_grad_norm",
    "rms_norm_grad_clip",
    "rms_norm_rotary_fwd",
    "rms_norm_rotary_bwd_workspace_size",
    "rms_norm_rotary_bwd",
    "rms_norm_embedding_fwd",
    "rms_norm_embedding_bwd_workspace_size",
    "rms_norm_embedding_bwd",
)


class RMSNormError(RuntimeError):
    """A C entry point returned an error status."""

    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: status {status} ({rms_norm_status_string(status)})")


class _Heads(ctypes.Structure):
    """rmsn_heads: a tensor of heads and its strides in elements."""

    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


_lib: Optional[ctypes.CDLL] = None
# The usual calls of the newer entry points without ctypes' cost (binding.cpp);
# None before load_library, or where it was not built, or against another
# PyTorch: the calls then take ctypes.
_binding = None


def _load_binding(lib: ctypes.CDLL) -> None:
    global _binding
    if not os.path.exists(BINDING_PATH):
        return
    spec = importlib.util.spec_from_file_location("bwd_rms_norm_gb300._binding", BINDING_PATH)
    try:
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError:                 # built against another PyTorch
        return
    if module.built_for != torch.__version__:
        return
    module.init(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.rms_norm_block_fwd, lib.rms_norm_block_bwd, lib.rms_norm_block_bwd_workspace_size,
        lib.rms_norm_grad_norm, lib.rms_norm_grad_clip, lib.rms_norm_grad_workspace_size)))
    module.init_more(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.rms_norm_rotary_fwd, lib.rms_norm_rotary_bwd, lib.rms_norm_rotary_bwd_workspace_size,
        lib.rms_norm_embedding_fwd, lib.rms_norm_embedding_bwd,
        lib.rms_norm_embedding_bwd_workspace_size)))
    _binding = module


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the shared library and declare the C signatures (once)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it first (python -m bwd_rms_norm_gb300.build)")
    lib = ctypes.CDLL(path)
    P, I64, I, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.rms_norm_fwd.argtypes = [P, P, P, P, I64, I64, F, I, I, I, P]
    lib.rms_norm_fwd.restype = I
    lib.rms_norm_bwd_workspace_size.argtypes = [I64, I64, I]
    lib.rms_norm_bwd_workspace_size.restype = SZ
    lib.rms_norm_bwd.argtypes = [P, P, P, P, P, P, I64, I64, I, I, P, SZ, P]
    lib.rms_norm_bwd.restype = I
    lib.rms_norm_status_string.argtypes = [I]
    lib.rms_norm_status_string.restype = ctypes.c_char_p
    lib.rms_norm_last_cuda_error.argtypes = []
    lib.rms_norm_last_cuda_error.restype = I
    lib.rms_norm_last_kernels.argtypes = [ctypes.POINTER(ctypes.c_char_p), I]
    lib.rms_norm_last_kernels.restype = I
    lib.rms_norm_last_launch_count.argtypes = []
    lib.rms_norm_last_launch_count.restype = I
    lib.rms_norm_bwd_noalloc.argtypes = [P, P, P, P, P, P, I64, I64, I, I, P]
    lib.rms_norm_bwd_noalloc.restype = I
    lib.rms_norm_bwd_blocked_workspace_size.argtypes = [I64, I64, I64]
    lib.rms_norm_bwd_blocked_workspace_size.restype = SZ
    lib.rms_norm_dw_chunk_count.argtypes = [I64, I64]
    lib.rms_norm_dw_chunk_count.restype = I64
    lib.rms_norm_bwd_blocked.argtypes = [P, P, P, P, P, P, I64, I64, I64, I, I, P, SZ, P]
    lib.rms_norm_bwd_blocked.restype = I
    lib.rms_norm_dw_sum.argtypes = [P, I64, I64, P, P]
    lib.rms_norm_dw_sum.restype = I
    lib.rms_norm_rank_rows.argtypes = [I64, I64, I, I, ctypes.POINTER(I64), ctypes.POINTER(I64)]
    lib.rms_norm_rank_rows.restype = I
    lib.rms_norm_set_sm_budget.argtypes = [I]
    lib.rms_norm_set_sm_budget.restype = I
    lib.rms_norm_sm_budget.argtypes = []
    lib.rms_norm_sm_budget.restype = I
    lib.rms_norm_wait_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint)]
    lib.rms_norm_wait_timeouts.restype = I
    lib.rms_norm_selftest_wait_limit.argtypes = [ctypes.POINTER(ctypes.c_uint),
                                                 ctypes.POINTER(ctypes.c_double)]
    lib.rms_norm_selftest_wait_limit.restype = I
    lib.rms_norm_fwd_fp8.argtypes = [P, P, P, P, P, I64, I64, F, I, I, P]
    lib.rms_norm_fwd_fp8.restype = I
    lib.group_norm_fwd.argtypes = [P, P, P, P, P, P, I64, I64, I64, I64, F, I, P]
    lib.group_norm_fwd.restype = I
    lib.group_norm_bwd_workspace_size.argtypes = [I64, I64, I64, I64, I]
    lib.group_norm_bwd_workspace_size.restype = SZ
    lib.group_norm_bwd.argtypes = [P, P, P, P, P, P, P, P, I64, I64, I64, I64, I, P, SZ, P]
    lib.group_norm_bwd.restype = I
    lib.softmax_fwd.argtypes = [P, P, I64, I64, I, P]
    lib.softmax_fwd.restype = I
    lib.softmax_bwd.argtypes = [P, P, P, I64, I64, I, P]
    lib.softmax_bwd.restype = I
    lib.layer_norm_fwd.argtypes = [P, P, P, P, P, P, I64, I64, F, I, P]
    lib.layer_norm_fwd.restype = I
    lib.layer_norm_bwd_workspace_size.argtypes = [I64, I64, I]
    lib.layer_norm_bwd_workspace_size.restype = SZ
    lib.layer_norm_bwd.argtypes = [P, P, P, P, P, P, P, P, I64, I64, I, P, SZ, P]
    lib.layer_norm_bwd.restype = I
    lib.rms_norm_block_fwd.argtypes = [P, P, P, P, I64, P, P, P, P, P, I64, I64, F, F, F, I, I, I,
                                       P]
    lib.rms_norm_block_fwd.restype = I
    lib.rms_norm_block_bwd_workspace_size.argtypes = [I64, I64, I64]
    lib.rms_norm_block_bwd_workspace_size.restype = SZ
    lib.rms_norm_block_bwd.argtypes = [P, P, P, P, P, P, I64, P, P, P, P, P, P, P, P, I64, I64, F,
                                       F, I, I, I, P, SZ, P]
    lib.rms_norm_block_bwd.restype = I
    lib.rms_norm_grad_workspace_size.argtypes = [I64]
    lib.rms_norm_grad_workspace_size.restype = SZ
    lib.rms_norm_grad_norm.argtypes = [P, P, P, I64, P, P, SZ, P]
    lib.rms_norm_grad_norm.restype = I
    lib.rms_norm_grad_clip.argtypes = [P, P, P, P, P, I64, F, F, P, P, P, SZ, P]
    lib.rms_norm_grad_clip.restype = I
    H = ctypes.POINTER(_Heads)
    lib.rms_norm_rotary_fwd.argtypes = [H, H, P, P, P, I, P, I, I64, H, H, P, P, I64, I64, I64,
                                        I64, I64, I64, I, F, I, I, P]
    lib.rms_norm_rotary_fwd.restype = I
    lib.rms_norm_rotary_bwd_workspace_size.argtypes = [I64, I64, I64, I64, I64]
    lib.rms_norm_rotary_bwd_workspace_size.restype = SZ
    lib.rms_norm_rotary_bwd.argtypes = [H, H, H, H, P, P, P, P, P, I, P, I, I64, H, H, P, P, I64,
                                        I64, I64, I64, I64, I64, I, I, I, P, SZ, P]
    lib.rms_norm_rotary_bwd.restype = I
    lib.rms_norm_embedding_fwd.argtypes = [P, I, P, P, I64, I64, I64, F, I, I, P]
    lib.rms_norm_embedding_fwd.restype = I
    lib.rms_norm_embedding_bwd_workspace_size.argtypes = [I64, I64, I64]
    lib.rms_norm_embedding_bwd_workspace_size.restype = SZ
    lib.rms_norm_embedding_bwd.argtypes = [P, P, I, P, I64, I64, I64, F, I64, I, I, I, P, SZ, P]
    lib.rms_norm_embedding_bwd.restype = I
    _load_binding(lib)
    _lib = lib
    return lib


def rms_norm_status_string(status: int) -> str:
    return load_library().rms_norm_status_string(int(status)).decode()


def rms_norm_bwd_workspace_size(rows: int, hidden: int, dtype) -> int:
    """Bytes of workspace ``rms_norm_bwd`` needs (``dtype`` a torch dtype or
    a C code)."""
    code = DTYPE_CODES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(load_library().rms_norm_bwd_workspace_size(int(rows), int(hidden), code))


def last_launch_count() -> int:
    """Kernels enqueued by the last successful call on this thread."""
    return int(load_library().rms_norm_last_launch_count())


def last_kernels() -> list:
    """Symbol names of the kernels the last call on this thread launched."""
    buf = (ctypes.c_char_p * 4)()
    n = load_library().rms_norm_last_kernels(buf, 4)
    return [buf[i].decode() for i in range(max(n, 0))]


def wait_timeouts() -> int:
    """Bounded device waits that ran out since the library was loaded (0 in
    correct operation); synchronises with the device."""
    n = ctypes.c_uint(0)
    st = load_library().rms_norm_wait_timeouts(ctypes.byref(n))
    if st != RMSN_OK:
        raise RMSNormError("rms_norm_wait_timeouts", st)
    return int(n.value)


def selftest_wait_limit() -> Tuple[int, float]:
    """Run the bounded-wait self-test (a wait on a barrier nothing completes
    runs out after about a second): returns (waits that ran out, seconds)."""
    n, t = ctypes.c_uint(0), ctypes.c_double(0.0)
    st = load_library().rms_norm_selftest_wait_limit(ctypes.byref(n), ctypes.byref(t))
    if st != RMSN_OK:
        raise RMSNormError("rms_norm_selftest_wait_limit", st)
    return int(n.value), float(t.value)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _stream_handle(device: torch.device, stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s.cuda_stream


def _check_cuda(name: str, t: torch.Tensor, device: Optional[torch.device] = None) -> None:
    if not t.is_cuda:
        raise RuntimeError(f"{name} must be a CUDA tensor (this library has no CPU path)")
    if device is not None and t.device != device:
        raise RuntimeError(f"{name} is on {t.device}, the other tensors on {device}")
    if not t.is_contiguous():
        raise RuntimeError(f"{name} must be contiguous")


def _check_like(name: str, t: Optional[torch.Tensor], dtype: torch.dtype, numel: int,
                shape=None) -> None:
    """A tensor the kernels read or write a fixed extent of: its dtype and
    size are checked on the host before anything reaches the device (a short
    buffer would be read or written out of bounds)."""
    if t is None:
        return
    if t.dtype != dtype:
        raise RuntimeError(f"{name} must be {dtype}, not {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise RuntimeError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.numel() != numel:
        raise RuntimeError(f"{name} must have {numel} elements, not {t.numel()}")


def _check_bwd_args(dy, x, gamma, rstd, dx, dw) -> Tuple[int, int]:
    """Host-side checks shared by the RMSNorm backward entry points: dtypes,
    shapes and element counts of every tensor, caller-supplied outputs
    included.  Returns (rows, hidden)."""
    if x.dtype not in DTYPE_CODES:
        raise RuntimeError(f"x must be float32, bfloat16 or float16, not {x.dtype}")
    rows, hidden = _as_rows(x)
    _check_like("dy", dy, x.dtype, x.numel(), x.shape)
    _check_like("gamma", gamma, x.dtype, hidden)
    _check_like("rstd", rstd, torch.float32, rows)
    _check_like("dx", dx, x.dtype, x.numel(), x.shape)
    _check_like("dw", dw, torch.float32, hidden)
    return rows, hidden


def _as_rows(x: torch.Tensor) -> Tuple[int, int]:
    if x.dim() < 1:
        raise RuntimeError("x must have at least one dimension")
    hidden = x.shape[-1]
    rows = x.numel() // hidden if hidden > 0 else 0
    return rows, hidden


def rms_norm_fwd(x: torch.Tensor, gamma: torch.Tensor, eps: float, offset: int = 0,
                 cast_mode: str = "round_once", y: Optional[torch.Tensor] = None,
                 rstd: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None):
    """Forward over the last dimension of ``x``; returns ``(y, rstd)`` with
    ``y`` shaped like ``x`` and ``rstd`` fp32 of shape ``x.shape[:-1]``."""
    lib = load_library()
    if x.dtype not in DTYPE_CODES:
        raise RuntimeError(f"x must be float32, bfloat16 or float16, not {x.dtype}")
    if cast_mode not in CAST_MODES:
        raise RuntimeError(f"cast_mode must be one of {sorted(CAST_MODES)}")
    rows, hidden = _as_rows(x)
    _check_like("gamma", gamma, x.dtype, hidden)
    _check_like("y", y, x.dtype, x.numel(), x.shape)
    _check_like("rstd", rstd, torch.float32, rows)
    _check_cuda("x", x)
    _check_cuda("gamma", gamma, x.device)
    if y is None:
        y = torch.empty_like(x)
    if rstd is None:
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _check_cuda("y", y, x.device)
    _check_cuda("rstd", rstd, x.device)
    with torch.cuda.device(x.device):
        st = lib.rms_norm_fwd(_ptr(x), _ptr(gamma), _ptr(y), _ptr(rstd), rows, hidden,
                              float(eps), int(offset), DTYPE_CODES[x.dtype],
                              CAST_MODES[cast_mode], _stream_handle(x.device, stream))
    if st != RMSN_OK:
        raise RMSNormError("rms_norm_fwd", st)
    return y, rstd


FP8_DTYPE = torch.float8_e4m3fn


def rms_norm_fwd_fp8(x: torch.Tensor, gamma: torch.Tensor, scale: torch.Tensor, eps: float,
                     offset: int = 0, y: Optional[torch.Tensor] = None,
                     rstd: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None):
    """Forward with an FP8 E4M3 output: ``y = e4m3(x_hat * gain * scale)``
    (saturating).  ``scale`` is a one-element fp32 tensor on the device (read
    by the kernel); returns ``(y, rstd)`` with ``y`` of dtype
    torch.float8_e4m3fn shaped like ``x``."""
    lib = load_library()
    if x.dtype not in DTYPE_CODES:
        raise RuntimeError(f"x must be float32, bfloat16 or float16, not {x.dtype}")
    rows, hidden = _as_rows(x)
    _check_like("gamma", gamma, x.dtype, hidden)
    _check_like("scale", scale, torch.float32, 1)
    _check_like("y", y, FP8_DTYPE, x.numel(), x.shape)
    _check_like("rstd", rstd, torch.float32, rows)
    _check_cuda("x", x)
    _check_cuda("gamma", gamma, x.device)
    _check_cuda("scale", scale, x.device)
    if y is None:
        y = torch.empty(x.shape, dtype=FP8_DTYPE, device=x.device)
    if rstd is None:
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _check_cuda("y", y, x.device)
    _check_cuda("rstd", rstd, x.device)
    with torch.cuda.device(x.device):
        st = lib.rms_norm_fwd_fp8(_ptr(x), _ptr(gamma), _ptr(scale), _ptr(y), _ptr(rstd), rows,
                                  hidden, float(eps), int(offset), DTYPE_CODES[x.dtype],
                                  _stream_handle(x.device, stream))
    if st != RMSN_OK:
        raise RMSNormError("rms_norm_fwd_fp8", st)
    return y, rstd


def rms_norm_bwd(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor, rstd: torch.Tensor,
                 offset: int = 0, dx: Optional[torch.Tensor] = None,
                 dw: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None):
    """Backward; returns ``(dx, dw)`` with ``dw`` fp32 of shape ``[hidden]``.
    ``workspace`` (a byte or float tensor of at least
    ``rms_norm_bwd_workspace_size`` bytes) is allocated when not given."""
    lib = load_library()
    rows, hidden = _check_bwd_args(dy, x, gamma, rstd, dx, dw)
    for name, t in (("x", x), ("dy", dy), ("gamma", gamma), ("rstd", rstd)):
        _check_cuda(name, t, x.device)
    code = DTYPE_CODES[x.dtype]
    if dx is None:
        dx = torch.empty_like(x)
    if dw is None:
        dw = torch.empty(hidden, dtype=torch.float32, device=x.device)
    need = int(lib.rms_norm_bwd_workspace_size(rows, hidden, code))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    _check_cuda("dx", dx, x.device)
    _check_cuda("dw", dw, x.device)
    _check_cuda("workspace", workspace, x.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    with torch.cuda.device(x.device):
        st = lib.rms_norm_bwd(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(rstd), _ptr(dx), _ptr(dw),
                              rows, hidden, int(offset), code, workspace.data_ptr(), ws_bytes,
                              _stream_handle(x.device, stream))
    if st != RMSN_OK:
        raise RMSNormError("rms_norm_bwd", st)
    return dx, dw


def rms_norm_bwd_noalloc(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor,
                         rstd: torch.Tensor, offset: int = 0, dx: Optional[torch.Tensor] = None,
                         dw: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None):
    """Backward for callers that cannot allocate device scratch: the library
    keeps the weight-gradient partials in its own fixed 16 MiB device array
    (sizes needing more are refused).  Pass ``dx`` and ``dw`` to avoid any
    allocation on the Python side as well.  Calls that may overlap on the GPU
    share that array and must be ordered on one stream."""
    lib = load_library()
    rows, hidden = _check_bwd_args(dy, x, gamma, rstd, dx, dw)
    for name, t in (("x", x), ("dy", dy), ("gamma", gamma), ("rstd", rstd)):
        _check_cuda(name, t, x.device)
    if dx is None:
        dx = torch.empty_like(x)
    if dw is None:
        dw = torch.empty(hidden, dtype=torch.float32, device=x.device)
    _check_cuda("dx", dx, x.device)
    _check_cuda("dw", dw, x.device)
    with torch.cuda.device(x.device):
        st = lib.rms_norm_bwd_noalloc(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(rstd), _ptr(dx),
                                      _ptr(dw), rows, hidden, int(offset), DTYPE_CODES[x.dtype],
                                      _stream_handle(x.device, stream))
    if st != RMSN_OK:
        raise RMSNormError("rms_norm_bwd_noalloc", st)
    return dx, dw


def rms_norm_dw_chunk_count(rows: int, block_rows: int) -> int:
    """Chunk sums ``rms_norm_bwd_blocked`` writes for ``rows`` rows."""
    n = int(load_library().rms_norm_dw_chunk_count(int(rows), int(block_rows)))
    if n < 0:
        raise RMSNormError("rms_norm_dw_chunk_count", -n)
    return n


def rms_norm_bwd_blocked_workspace_size(rows: int, hidden: int, block_rows: int) -> int:
    """Bytes of workspace ``rms_norm_bwd_blocked`` needs."""
    return int(load_library().rms_norm_bwd_blocked_workspace_size(int(rows), int(hidden),
                                                                  int(block_rows)))


def rms_norm_rank_rows(rows: int, block_rows: int, world: int, rank: int) -> Tuple[int, int]:
    """Rank ``rank``'s slab [lo, hi) of ``rows`` rows in whole chunks of
    ``RMSN_DW_CHUNK_BLOCKS * block_rows`` rows (no device needed)."""
    lo, hi = ctypes.c_int64(0), ctypes.c_int64(0)
    st = load_library().rms_norm_rank_rows(int(rows), int(block_rows), int(world), int(rank),
                                           ctypes.byref(lo), ctypes.byref(hi))
    if st != RMSN_OK:
        raise RMSNormError("rms_norm_rank_rows", st)
    return int(lo.value), int(hi.value)


def rms_norm_bwd_blocked(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor,
                         rstd: torch.Tensor, block_rows: int, offset: int = 0,
                         dx: Optional[torch.Tensor] = None,
                         chunk_sums: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None):
    """Backward with the weight gradient left as chunk sums over fixed blocks
    of ``block_rows`` rows; returns ``(dx, chunk_sums)``, ``chunk_sums`` fp32
    of shape [rms_norm_dw_chunk_count(rows, block_rows), hidden].  Adding
    them with ``rms_norm_dw_sum`` gives the same dw for any split of the rows
    into whole chunks (see ``rms_norm_rank_rows``)."""
    lib = load_library()
    rows, hidden = _check_bwd_args(dy, x, gamma, rstd, dx, None)
    if int(block_rows) < 1:
        raise RuntimeError("block_rows must be at least 1")
    nchunks = rms_norm_dw_chunk_count(rows, block_rows)
    _check_like("chunk_sums", chunk_sums, torch.float32, nchunks * hidden)
    for name, t in (("x", x), ("dy", dy), ("gamma", gamma), ("rstd", rstd)):
        _check_cuda(name, t, x.device)
    if dx is None:
        dx = torch.empty_like(x)
    if chunk_sums is None:
        chunk_sums = torch.empty(nchunks, hidden, dtype=torch.float32, device=x.device)
    need = rms_norm_bwd_blocked_workspace_size(rows, hidden, block_rows)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    for name, t in (("dx", dx), ("chunk_sums", chunk_sums), ("workspace", workspace)):
        _check_cuda(name, t, x.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    with torch.cuda.device(x.device):
        st = lib.rms_norm_bwd_blocked(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(rstd), _ptr(dx),
                                      _ptr(chunk_sums), rows, hidden, int(block_rows),
                                      int(offset), DTYPE_CODES[x.dtype], workspace.data_ptr(),
                                      ws_bytes, _stream_handle(x.device, stream))
    if st != RMSN_OK:
        raise RMSNormError("rms_norm_bwd_blocked", st)
    return dx, chunk_sums


def rms_norm_dw_sum(chunk_sums: torch.Tensor, dw: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """dw [hidden] = the chunk sums [nchunks, hidden] added in chunk order."""
    lib = load_library()
    if chunk_sums.dim() != 2 or chunk_sums.dtype != torch.float32:
        raise RuntimeError("chunk_sums must be a float32 [nchunks, hidden] tensor")
    nchunks, hidden = chunk_sums.shape
    _check_like("dw", dw, torch.float32, hidden)
    _check_cuda("chunk_sums", chunk_sums)
    if dw is None:
        dw = torch.empty(hidden, dtype=torch.float32, device=chunk_sums.device)
    _check_cuda("dw", dw, chunk_sums.device)
    with torch.cuda.device(chunk_sums.device):
        st = lib.rms_norm_dw_sum(_ptr(chunk_sums), nchunks, hidden, _ptr(dw),
                                 _stream_handle(chunk_sums.device, stream))
    if st != RMSN_OK:
        raise RMSNormError("rms_norm_dw_sum", st)
    return dw


def rms_norm_set_sm_budget(sms: int) -> None:
    """Let the persistent kernels use at most ``sms`` SMs' worth of
    resident CTAs (0: every SM); process-wide, read at each launch."""
    st = load_library().rms_norm_set_sm_budget(int(sms))
    if st != RMSN_OK:
        raise RMSNormError("rms_norm_set_sm_budget", st)


def rms_norm_sm_budget() -> int:
    return int(load_library().rms_norm_sm_budget())


def layer_norm_fwd(x: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor], eps: float,
                   y: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
                   rstd: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None):
    """LayerNorm forward over the last dimension; returns ``(y, mean, rstd)``
    (``beta`` may be None)."""
    lib = load_library()
    if x.dtype not in DTYPE_CODES:
        raise RuntimeError(f"x must be float32, bfloat16 or float16, not {x.dtype}")
    rows, hidden = _as_rows(x)
    _check_like("gamma", gamma, x.dtype, hidden)
    _check_like("beta", beta, x.dtype, hidden)
    _check_like("y", y, x.dtype, x.numel(), x.shape)
    _check_like("mean", mean, torch.float32, rows)
    _check_like("rstd", rstd, torch.float32, rows)
    _check_cuda("x", x)
    _check_cuda("gamma", gamma, x.device)
    if beta is not None:
        _check_cuda("beta", beta, x.device)
    y = torch.empty_like(x) if y is None else y
    mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) if mean is None else mean
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) if rstd is None else rstd
    for name, t in (("y", y), ("mean", mean), ("rstd", rstd)):
        _check_cuda(name, t, x.device)
    with torch.cuda.device(x.device):
        st = lib.layer_norm_fwd(_ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(mean), _ptr(rstd),
                                rows, hidden, float(eps), DTYPE_CODES[x.dtype],
                                _stream_handle(x.device, stream))
    if st != RMSN_OK:
        raise RMSNormError("layer_norm_fwd", st)
    return y, mean, rstd


def layer_norm_bwd_workspace_size(rows: int, hidden: int, dtype) -> int:
    code = DTYPE_CODES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(load_library().layer_norm_bwd_workspace_size(int(rows), int(hidden), code))


def layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor, mean: torch.Tensor,
                   rstd: torch.Tensor, dx: Optional[torch.Tensor] = None,
                   dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                   with_dbeta: bool = True, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None):
    """LayerNorm backward; returns ``(dx, dgamma, dbeta)`` (dbeta None when
    ``with_dbeta`` is False)."""
    lib = load_library()
    rows, hidden = _check_bwd_args(dy, x, gamma, rstd, dx, dgamma)
    _check_like("mean", mean, torch.float32, rows)
    _check_like("dbeta", dbeta if with_dbeta else None, torch.float32, hidden)
    for name, t in (("x", x), ("dy", dy), ("gamma", gamma), ("mean", mean), ("rstd", rstd)):
        _check_cuda(name, t, x.device)
    code = DTYPE_CODES[x.dtype]
    dx = torch.empty_like(x) if dx is None else dx
    dgamma = torch.empty(hidden, dtype=torch.float32, device=x.device) if dgamma is None else dgamma
    if with_dbeta and dbeta is None:
        dbeta = torch.empty(hidden, dtype=torch.float32, device=x.device)
    need = int(lib.layer_norm_bwd_workspace_size(rows, hidden, code))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    for name, t in (("dx", dx), ("dgamma", dgamma), ("workspace", workspace)):
        _check_cuda(name, t, x.device)
    if with_dbeta:
        _check_cuda("dbeta", dbeta, x.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    with torch.cuda.device(x.device):
        st = lib.layer_norm_bwd(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(mean), _ptr(rstd), _ptr(dx),
                                _ptr(dgamma), _ptr(dbeta) if with_dbeta else None, rows, hidden,
                                code, workspace.data_ptr(), ws_bytes,
                                _stream_handle(x.device, stream))
    if st != RMSN_OK:
        raise RMSNormError("layer_norm_bwd", st)
    return dx, dgamma, (dbeta if with_dbeta else None)


def softmax_fwd(x: torch.Tensor, y: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Softmax over the last dimension of ``x`` (fp32 arithmetic, one
    rounding to x's dtype at the store)."""
    lib = load_library()
    if x.dtype not in DTYPE_CODES:
        raise RuntimeError(f"x must be float32, bfloat16 or float16, not {x.dtype}")
    rows, cols = _as_rows(x)
    _check_like("y", y, x.dtype, x.numel(), x.shape)
    _check_cuda("x", x)
    y = torch.empty_like(x) if y is None else y
    _check_cuda("y", y, x.device)
    with torch.cuda.device(x.device):
        st = lib.softmax_fwd(_ptr(x), _ptr(y), rows, cols, DTYPE_CODES[x.dtype],
                             _stream_handle(x.device, stream))
    if st != RMSN_OK:
        raise RMSNormError("softmax_fwd", st)
    return y


def softmax_bwd(dy: torch.Tensor, y: torch.Tensor, dx: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Backward of softmax_fwd from its output: dx = y * (dy - sum(dy * y))
    per row, the sum in fp32."""
    lib = load_library()
    if y.dtype not in DTYPE_CODES:
        raise RuntimeError(f"y must be float32, bfloat16 or float16, not {y.dtype}")
    rows, cols = _as_rows(y)
    _check_like("dy", dy, y.dtype, y.numel(), y.shape)
    _check_like("dx", dx, y.dtype, y.numel(), y.shape)
    _check_cuda("y", y)
    _check_cuda("dy", dy, y.device)
    dx = torch.empty_like(y) if dx is None else dx
    _check_cuda("dx", dx, y.device)
    with torch.cuda.device(y.device):
        st = lib.softmax_bwd(_ptr(dy), _ptr(y), _ptr(dx), rows, cols, DTYPE_CODES[y.dtype],
                             _stream_handle(y.device, stream))
    if st != RMSN_OK:
        raise RMSNormError("softmax_bwd", st)
    return dx


def _gn_shape(x: torch.Tensor, groups: int):
    if x.dim() < 2:
        raise RuntimeError("x must be [n, channels, *spatial]")
    n, c = x.shape[0], x.shape[1]
    spatial = 1
    for d in x.shape[2:]:
        spatial *= d
    if c % groups:
        raise RuntimeError("channels must be a multiple of groups")
    return n, c, spatial


def group_norm_fwd(x: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor],
                   groups: int, eps: float, y: Optional[torch.Tensor] = None,
                   mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None):
    """GroupNorm forward over x [n, channels, *spatial]; returns ``(y, mean,
    rstd)`` with mean and rstd fp32 [n, groups] (``beta`` may be None)."""
    lib = load_library()
    if x.dtype not in DTYPE_CODES:
        raise RuntimeError(f"x must be float32, bfloat16 or float16, not {x.dtype}")
    n, c, sp = _gn_shape(x, groups)
    _check_like("gamma", gamma, x.dtype, c)
    _check_like("beta", beta, x.dtype, c)
    _check_like("y", y, x.dtype, x.numel(), x.shape)
    _check_like("mean", mean, torch.float32, n * groups)
    _check_like("rstd", rstd, torch.float32, n * groups)
    _check_cuda("x", x)
    _check_cuda("gamma", gamma, x.device)
    if beta is not None:
        _check_cuda("beta", beta, x.device)
    y = torch.empty_like(x) if y is None else y
    mean = torch.empty(n, groups, dtype=torch.float32, device=x.device) if mean is None else mean
    rstd = torch.empty(n, groups, dtype=torch.float32, device=x.device) if rstd is None else rstd
    for name, t in (("y", y), ("mean", mean), ("rstd", rstd)):
        _check_cuda(name, t, x.device)
    with torch.cuda.device(x.device):
        st = lib.group_norm_fwd(_ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(mean), _ptr(rstd),
                                n, c, sp, int(groups), float(eps), DTYPE_CODES[x.dtype],
                                _stream_handle(x.device, stream))
    if st != RMSN_OK:
        raise RMSNormError("group_norm_fwd", st)
    return y, mean, rstd


def group_norm_bwd_workspace_size(n: int, channels: int, spatial: int, groups: int,
                                  dtype) -> int:
    code = DTYPE_CODES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(load_library().group_norm_bwd_workspace_size(int(n), int(channels), int(spatial),
                                                            int(groups), code))


def group_norm_bwd(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor, mean: torch.Tensor,
                   rstd: torch.Tensor, groups: int, dx: Optional[torch.Tensor] = None,
                   dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                   with_dbeta: bool = True, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None):
    """GroupNorm backward; returns ``(dx, dgamma, dbeta)`` (fp32 weight
    gradients; dbeta None when ``with_dbeta`` is False)."""
    lib = load_library()
    if x.dtype not in DTYPE_CODES:
        raise RuntimeError(f"x must be float32, bfloat16 or float16, not {x.dtype}")
    n, c, sp = _gn_shape(x, groups)
    _check_like("dy", dy, x.dtype, x.numel(), x.shape)
    _check_like("gamma", gamma, x.dtype, c)
    _check_like("mean", mean, torch.float32, n * groups)
    _check_like("rstd", rstd, torch.float32, n * groups)
    _check_like("dx", dx, x.dtype, x.numel(), x.shape)
    _check_like("dgamma", dgamma, torch.float32, c)
    _check_like("dbeta", dbeta if with_dbeta else None, torch.float32, c)
    for name, t in (("x", x), ("dy", dy), ("gamma", gamma), ("mean", mean), ("rstd", rstd)):
        _check_cuda(name, t, x.device)
    code = DTYPE_CODES[x.dtype]
    dx = torch.empty_like(x) if dx is None else dx
    dgamma = torch.empty(c, dtype=torch.float32, device=x.device) if dgamma is None else dgamma
    if with_dbeta and dbeta is None:
        dbeta = torch.empty(c, dtype=torch.float32, device=x.device)
    need = int(lib.group_norm_bwd_workspace_size(n, c, sp, int(groups), code))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    for name, t in (("dx", dx), ("dgamma", dgamma), ("workspace", workspace)):
        _check_cuda(name, t, x.device)
    if with_dbeta:
        _check_cuda("dbeta", dbeta, x.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    with torch.cuda.device(x.device):
        st = lib.group_norm_bwd(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(mean), _ptr(rstd), _ptr(dx),
                                _ptr(dgamma), _ptr(dbeta) if with_dbeta else None, n, c, sp,
                                int(groups), code, workspace.data_ptr(), ws_bytes,
                                _stream_handle(x.device, stream))
    if st != RMSN_OK:
        raise RMSNormError("group_norm_bwd", st)
    return dx, dgamma, (dbeta if with_dbeta else None)


class _On:
    """``device`` current, and ``stream`` if one is given, so that what a call
    allocates belongs to the stream that uses it; entering gives the stream's
    handle.  Does nothing where both are current already: a call's fixed cost
    on the host is what a short call costs."""

    __slots__ = ("index", "stream", "undo")

    def __init__(self, device: torch.device, stream: Optional[torch.cuda.Stream]):
        if stream is not None and stream.device != device:
            raise RuntimeError(f"stream is on {stream.device}, the tensors on {device}")
        self.index, self.stream, self.undo = device.index, stream, None

    def __enter__(self) -> int:
        if self.stream is not None or torch.cuda.current_device() != self.index:
            self.undo = contextlib.ExitStack()
            self.undo.enter_context(torch.cuda.device(self.index))
            if self.stream is not None:
                self.undo.enter_context(torch.cuda.stream(self.stream))
        return torch._C._cuda_getCurrentRawStream(self.index)

    def __exit__(self, *exc) -> None:
        if self.undo is not None:
            self.undo.close()


def _written(*tensors: Optional[torch.Tensor]) -> None:
    """Counts a version of each caller's tensor that a call wrote, which is how
    autograd notices that a tensor it saved has changed."""
    for t in tensors:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _address(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _plain(index: int, dtype: torch.dtype, shape, *tensors: Optional[torch.Tensor]) -> bool:
    """Whether every tensor given is contiguous, on GPU ``index``, and of this
    dtype and shape: the quick look before a call; what it does not pass goes
    through the checks that say what is wrong."""
    for t in tensors:
        if t is not None and not (t.dtype is dtype and t.shape == shape and t.is_contiguous()
                                  and t.get_device() == index):
            return False
    return True


def _block_sizes(x, post_gamma, gate, next_gamma) -> Tuple[int, int, int]:
    """(rows, hidden, gate rows) of a block-norm call."""
    if x.dtype not in DTYPE_CODES:
        raise RuntimeError(f"x must be float32, bfloat16 or float16, not {x.dtype}")
    if post_gamma is None and next_gamma is None:
        raise RuntimeError("post_gamma and next_gamma are both None: nothing to normalise")
    rows, hidden = _as_rows(x)
    if gate is None:
        return rows, hidden, 0
    if gate.dim() < 1 or gate.shape[-1] != hidden:
        raise RuntimeError(f"gate must have {hidden} columns, not shape {tuple(gate.shape)}")
    gate_rows = gate.numel() // hidden if hidden > 0 else 0
    if rows == gate_rows == 0:
        return rows, hidden, 0
    if gate_rows < 1 or rows % gate_rows:
        raise RuntimeError(f"gate has {gate_rows} rows, which do not divide the {rows} rows of x")
    if gate_rows > 1 and x.dim() > 2 and _broadcasts_otherwise(gate.shape[:-1], x.shape[:-1]):
        raise RuntimeError(f"gate of shape {tuple(gate.shape)} would repeat over dimensions of x "
                           f"{tuple(x.shape)} before its own, but a gate row is for consecutive "
                           "rows: expand it, or give it x's leading dimensions")
    return rows, hidden, gate_rows


def _broadcasts_otherwise(gate, x) -> bool:
    """Whether these leading dimensions of a gate broadcast to x's, by the
    usual rules, and not to runs of consecutive rows."""
    gate = (1,) * (len(x) - len(gate)) + tuple(gate)
    if len(gate) > len(x) or any(a not in (1, b) for a, b in zip(gate, x)):
        return False
    repeated = False
    for a, b in zip(gate, x):
        if a > 1 and repeated:
            return True
        repeated = repeated or a < b
    return False


def _check_offset(fn: str, offset) -> None:
    if offset not in (0, 1):            # int() would cut 0.5 to 0
        raise RMSNormError(fn, RMSN_ERR_ARG)


def _check_block(x, stream_name, stream, post_gamma, gate, next_gamma) -> None:
    """Checks shared by the block-norm calls, with a message for each."""
    hidden = x.shape[-1]
    want = torch.float32 if stream.dtype == torch.float32 else x.dtype
    _check_like(stream_name, stream, want, x.numel(), x.shape)
    _check_like("post_gamma", post_gamma, x.dtype, hidden, (hidden,))
    _check_like("next_gamma", next_gamma, x.dtype, hidden, (hidden,))
    if gate is not None:
        _check_like("gate", gate, x.dtype, gate.numel())


def rms_norm_block_fwd(x: torch.Tensor, residual: torch.Tensor,
                       post_gamma: Optional[torch.Tensor] = None,
                       gate: Optional[torch.Tensor] = None,
                       next_gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
                       offset: int = 0, residual_scale: float = 1.0, branch_scale: float = 1.0,
                       residual_out: Optional[torch.Tensor] = None,
                       y: Optional[torch.Tensor] = None,
                       rstd_post: Optional[torch.Tensor] = None,
                       rstd_next: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None):
    """The norms after and before a block, its gate and the residual sum:
    ``r = residual_scale * residual + branch_scale * gate * norm(x, post_gamma)``
    and ``y = norm(r, next_gamma)``.  ``x`` is the block's output; ``residual``
    has its shape and its dtype, or float32.  Either gamma may be None (no norm
    of x; no y).  ``gate`` is ``[hidden]``, or ``[..., hidden]`` with a number
    of rows that divides x's: each run of rows / gate rows consecutive rows of
    x uses one (a gate that would broadcast to x in another way is refused).
    Returns ``(r, y, rstd_post, rstd_next)``, None for what a missing norm
    would give; an output given must not share memory with an input."""
    lib = load_library()
    if _binding is not None and stream is None:
        got = _binding.block_fwd(x, residual, post_gamma, gate, next_gamma, eps, offset,
                                 residual_scale, branch_scale, residual_out, y, rstd_post,
                                 rstd_next)
        if got is not None:
            return got
    _check_offset("rms_norm_block_fwd", offset)
    dev, dtype, shape = x.device, x.dtype, x.shape
    res_dtype, index = residual.dtype, x.get_device()
    rows, hidden, gate_rows = _block_sizes(x, post_gamma, gate, next_gamma)
    if not (index >= 0 and (res_dtype is dtype or res_dtype is torch.float32)
            and _plain(index, dtype, shape, x, y)
            and _plain(index, res_dtype, shape, residual, residual_out)
            and _plain(index, dtype, shape[-1:], post_gamma, next_gamma)
            and _plain(index, torch.float32, shape[:-1], rstd_post, rstd_next)
            and (gate is None or _plain(index, dtype, gate.shape, gate))):
        _check_block(x, "residual", residual, post_gamma, gate, next_gamma)
        _check_like("residual_out", residual_out, res_dtype, x.numel(), shape)
        _check_like("y", y, dtype, x.numel(), shape)
        _check_like("rstd_post", rstd_post, torch.float32, rows)
        _check_like("rstd_next", rstd_next, torch.float32, rows)
        for name, t in (("x", x), ("residual", residual), ("post_gamma", post_gamma),
                        ("gate", gate), ("next_gamma", next_gamma),
                        ("residual_out", residual_out), ("y", y), ("rstd_post", rstd_post),
                        ("rstd_next", rstd_next)):
            if t is not None:
                _check_cuda(name, t, dev)
    given = (residual_out, y if next_gamma is not None else None,
             rstd_post if post_gamma is not None else None,
             rstd_next if next_gamma is not None else None)
    with _On(dev, stream) as handle:
        if residual_out is None:
            residual_out = torch.empty_like(residual)
        if post_gamma is None:
            rstd_post = None
        elif rstd_post is None:
            rstd_post = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
        if next_gamma is None:
            y = rstd_next = None
        else:
            y = torch.empty_like(x) if y is None else y
            if rstd_next is None:
                rstd_next = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
        st = lib.rms_norm_block_fwd(x.data_ptr(), residual.data_ptr(), _address(post_gamma),
                                    _address(gate), gate_rows, _address(next_gamma),
                                    residual_out.data_ptr(), _address(y), _address(rstd_post),
                                    _address(rstd_next), rows, hidden, float(residual_scale + 0.0),
                                    float(branch_scale + 0.0), float(eps), int(offset),
                                    DTYPE_CODES[dtype], DTYPE_CODES[res_dtype], handle)
    if st != RMSN_OK:
        raise RMSNormError("rms_norm_block_fwd", st)
    _written(*given)
    return residual_out, y, rstd_post, rstd_next


def rms_norm_block_bwd_workspace_size(rows: int, hidden: int, gate_rows: int = 0) -> int:
    """Bytes of workspace ``rms_norm_block_bwd`` needs."""
    return int(load_library().rms_norm_block_bwd_workspace_size(int(rows), int(hidden),
                                                                int(gate_rows)))


def rms_norm_block_bwd(dy: Optional[torch.Tensor], dresidual_out: Optional[torch.Tensor],
                       x: torch.Tensor, residual_out: torch.Tensor,
                       rstd_post: Optional[torch.Tensor], rstd_next: Optional[torch.Tensor],
                       post_gamma: Optional[torch.Tensor] = None,
                       gate: Optional[torch.Tensor] = None,
                       next_gamma: Optional[torch.Tensor] = None, offset: int = 0,
                       residual_scale: float = 1.0, branch_scale: float = 1.0,
                       with_dgate: bool = True, dx: Optional[torch.Tensor] = None,
                       dresidual: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None):
    """Backward of ``rms_norm_block_fwd`` from the gradients of its y (``dy``,
    only with ``next_gamma``) and of its r (``dresidual_out``; None: none).
    Returns ``(dx, dresidual, dpost, dgate, dnext)``: the sums over rows are
    fp32, ``dgate`` shaped like ``gate`` (None without a gate or with
    ``with_dgate`` False), ``dpost`` / ``dnext`` None for a missing norm."""
    lib = load_library()
    if _binding is not None and stream is None:
        got = _binding.block_bwd(dy, dresidual_out, x, residual_out, rstd_post, rstd_next,
                                 post_gamma, gate, next_gamma, offset, residual_scale,
                                 branch_scale, with_dgate, dx, dresidual, workspace)
        if got is not None:
            return got
    _check_offset("rms_norm_block_bwd", offset)
    rows, hidden, gate_rows = _block_sizes(x, post_gamma, gate, next_gamma)
    if next_gamma is None:
        dy = None
        if dresidual_out is None:
            raise RuntimeError("dresidual_out is needed without next_gamma")
    elif dy is None or rstd_next is None:
        raise RuntimeError("dy and rstd_next are needed with next_gamma")
    if post_gamma is not None and rstd_post is None:
        raise RuntimeError("rstd_post is needed with post_gamma")
    dev, dtype, shape = x.device, x.dtype, x.shape
    res_dtype, index = residual_out.dtype, x.get_device()
    if not (index >= 0 and (res_dtype is dtype or res_dtype is torch.float32)
            and _plain(index, dtype, shape, x, dy, dx)
            and _plain(index, res_dtype, shape, residual_out, dresidual_out, dresidual)
            and _plain(index, dtype, shape[-1:], post_gamma, next_gamma)
            and _plain(index, torch.float32, shape[:-1], rstd_post, rstd_next)
            and (gate is None or _plain(index, dtype, gate.shape, gate)) and workspace is None):
        _check_block(x, "residual_out", residual_out, post_gamma, gate, next_gamma)
        _check_like("dy", dy, dtype, x.numel(), shape)
        _check_like("dresidual_out", dresidual_out, res_dtype, x.numel(), shape)
        _check_like("rstd_post", rstd_post, torch.float32, rows)
        _check_like("rstd_next", rstd_next, torch.float32, rows)
        _check_like("dx", dx, dtype, x.numel(), shape)
        _check_like("dresidual", dresidual, res_dtype, x.numel(), shape)
        for name, t in (("x", x), ("residual_out", residual_out), ("dy", dy),
                        ("dresidual_out", dresidual_out), ("rstd_post", rstd_post),
                        ("rstd_next", rstd_next), ("post_gamma", post_gamma), ("gate", gate),
                        ("next_gamma", next_gamma), ("dx", dx), ("dresidual", dresidual),
                        ("workspace", workspace)):
            if t is not None:
                _check_cuda(name, t, dev)
    given = (dx, dresidual)
    with _On(dev, stream) as handle:
        dx = torch.empty_like(x) if dx is None else dx
        dresidual = torch.empty_like(residual_out) if dresidual is None else dresidual
        dpost = dnext = dgate = None
        if post_gamma is not None:
            dpost = torch.empty(hidden, dtype=torch.float32, device=dev)
        if next_gamma is not None:
            dnext = torch.empty(hidden, dtype=torch.float32, device=dev)
        if gate is not None and with_dgate:
            dgate = torch.empty(gate.shape, dtype=torch.float32, device=dev)
        if workspace is None:
            need = int(lib.rms_norm_block_bwd_workspace_size(rows, hidden, gate_rows))
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        st = lib.rms_norm_block_bwd(_address(dy), _address(dresidual_out), x.data_ptr(),
                                    residual_out.data_ptr(), _address(post_gamma),
                                    _address(gate), gate_rows, _address(next_gamma),
                                    _address(rstd_post), _address(rstd_next), dx.data_ptr(),
                                    dresidual.data_ptr(), _address(dpost), _address(dgate),
                                    _address(dnext), rows, hidden, float(residual_scale + 0.0),
                                    float(branch_scale + 0.0), int(offset), DTYPE_CODES[dtype],
                                    DTYPE_CODES[res_dtype], workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(), handle)
    if st != RMSN_OK:
        raise RMSNormError("rms_norm_block_bwd", st)
    _written(*given)
    return dx, dresidual, dpost, dgate, dnext


def rms_norm_grad_workspace_size(count: int) -> int:
    """Bytes of workspace a norm over ``count`` gradients needs."""
    return int(load_library().rms_norm_grad_workspace_size(int(count)))


_Tensor = torch.Tensor


def _grad_list(name: str, grads, device: torch.device):
    """Host arrays (pointers, element counts, dtype codes) of a list of
    tensors.  The checks run over the list one property at a time (half the
    time of tensor by tensor on lists of hundreds)."""
    if (set(map(_Tensor.get_device, grads)) != {device.index if device.type == "cuda" else None}
            or not all(map(_Tensor.is_contiguous, grads))):
        for t in grads:
            if t.dtype not in DTYPE_CODES:
                raise RuntimeError(f"{name} must be float32, bfloat16 or float16, not {t.dtype}")
            _check_cuda(name, t, device)
    dtypes = [t.dtype for t in grads]
    kinds = set(dtypes)
    for d in kinds:
        if d not in DTYPE_CODES:
            raise RuntimeError(f"{name} must be float32, bfloat16 or float16, not {d}")
    if len(kinds) == 1:
        codes = array.array("i", [DTYPE_CODES[dtypes[0]]]) * len(dtypes)
    else:
        codes = array.array("i", [DTYPE_CODES[d] for d in dtypes])
    return (array.array("Q", list(map(_Tensor.data_ptr, grads))),
            array.array("q", list(map(_Tensor.numel, grads))), codes)


def _scalar(name: str, t: Optional[torch.Tensor], device: torch.device) -> None:
    if t is not None:
        _check_like(name, t, torch.float32, 1)
        _check_cuda(name, t, device)


def _grads_of(grads):
    grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
    if not grads:
        raise RuntimeError("the list of gradients is empty")
    return grads


def rms_norm_grad_norm(grads, norm: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The 2-norm over a list of gradients (contiguous CUDA tensors of one
    device, of any of the three dtypes): an fp32 tensor of no dimensions."""
    lib = load_library()
    if _binding is not None and norm is workspace is stream is None:
        got = _binding.grad_norm(grads)
        if got is not None:
            return got
    grads = _grads_of(grads)
    dev = grads[0].device
    ptrs, numels, codes = _grad_list("a gradient", grads, dev)
    _scalar("norm", norm, dev)
    given = norm
    with _On(dev, stream) as handle:
        if norm is None:
            norm = torch.empty((), dtype=torch.float32, device=dev)
        if workspace is None:
            need = int(lib.rms_norm_grad_workspace_size(len(grads)))
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        _check_cuda("workspace", workspace, dev)
        st = lib.rms_norm_grad_norm(ptrs.buffer_info()[0], numels.buffer_info()[0],
                                    codes.buffer_info()[0], len(grads), norm.data_ptr(),
                                    workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(), handle)
    if st != RMSN_OK:
        raise RMSNormError("rms_norm_grad_norm", st)
    _written(given)
    return norm


def rms_norm_grad_clip(grads, max_norm: float, eps: float = 1e-6, out=None,
                       total_norm: Optional[torch.Tensor] = None,
                       norm: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Scale a list of gradients by ``min(1, max_norm / (norm + eps))``, in
    place, or into the tensors of ``out`` (same sizes, the gradient's dtype or
    float32).  Returns the norm before the scaling, an fp32 tensor of no
    dimensions.  Where an element, or ``total_norm``, is not finite the
    gradients are not scaled: look at the norm before the update.  (A finite
    list whose norm is beyond fp32 is scaled, and its norm comes out
    infinite.)  With ``total_norm`` (a one-element fp32 tensor) that norm is
    taken instead of the list's own, e.g. one summed over ranks."""
    lib = load_library()
    if _binding is not None and norm is workspace is stream is None:
        got = _binding.grad_clip(grads, max_norm, eps, out, total_norm)
        if got is not None:
            return got
    grads = _grads_of(grads)
    dev = grads[0].device
    outs = grads if out is None else _grads_of(out)
    if len(outs) != len(grads):
        raise RuntimeError(f"out has {len(outs)} tensors, the list {len(grads)}")
    if out is not None and (
            list(map(_Tensor.numel, outs)) != list(map(_Tensor.numel, grads))
            or any(o.dtype != torch.float32 and o.dtype != g.dtype for g, o in zip(grads, outs))):
        for g, o in zip(grads, outs):
            _check_like("a tensor of out", o,
                        o.dtype if o.dtype == torch.float32 else g.dtype, g.numel())
    ptrs, numels, codes = outs_of = _grad_list("a gradient", grads, dev)
    if out is not None:
        outs_of = _grad_list("a tensor of out", outs, dev)
    _scalar("total_norm", total_norm, dev)
    _scalar("norm", norm, dev)
    given = norm
    with _On(dev, stream) as handle:
        if norm is None:
            norm = torch.empty((), dtype=torch.float32, device=dev)
        if workspace is None and total_norm is None:
            need = int(lib.rms_norm_grad_workspace_size(len(grads)))
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        size = 0
        if workspace is not None:
            _check_cuda("workspace", workspace, dev)
            size = workspace.numel() * workspace.element_size()
        st = lib.rms_norm_grad_clip(ptrs.buffer_info()[0], numels.buffer_info()[0],
                                    codes.buffer_info()[0], outs_of[0].buffer_info()[0],
                                    outs_of[2].buffer_info()[0], len(grads), float(max_norm),
                                    float(eps), _ptr(total_norm), norm.data_ptr(),
                                    _ptr(workspace), size, handle)
    if st != RMSN_OK:
        raise RMSNormError("rms_norm_grad_clip", st)
    _written(given, *outs)
    return norm


def _check_strided(name: str, t: torch.Tensor, device: torch.device) -> None:
    if not t.is_cuda:
        raise RuntimeError(f"{name} must be a CUDA tensor (this library has no CPU path)")
    if t.device != device:
        raise RuntimeError(f"{name} is on {t.device}, the other tensors on {device}")


def _check_heads(name: str, t: Optional[torch.Tensor], dtype: torch.dtype, shape,
                 device: torch.device) -> None:
    """A tensor of heads: of any strides but the last dimension's."""
    if t is None:
        raise RuntimeError(f"{name} is missing")
    if t.dtype != dtype:
        raise RuntimeError(f"{name} must be {dtype}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise RuntimeError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    _check_strided(name, t, device)
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise RuntimeError(f"{name} must be contiguous in its last dimension")


def _heads_of(t: Optional[torch.Tensor]):
    """The C call's view of a tensor of heads."""
    if t is None:
        return None
    st = t.stride()
    return _Heads(t.data_ptr(), st[0] if t.dim() == 4 else 0, st[-3], st[-2])


class _RotaryCall:
    """Sizes of a head-norm call, with the checks its two directions share."""

    __slots__ = ("batch", "tokens", "q_heads", "k_heads", "dim", "rotary", "pos_stride")

    def __init__(self, q, k, q_gamma, k_gamma, inv_freq, positions):
        dev = q.device
        if q.dtype not in DTYPE_CODES:
            raise RuntimeError(f"q must be float32, bfloat16 or float16, not {q.dtype}")
        if q.dim() not in (3, 4):
            raise RuntimeError("q must be [tokens, heads, head_dim] or [batch, tokens, heads, "
                               f"head_dim], not of shape {tuple(q.shape)}")
        _check_heads("q", q, q.dtype, q.shape, dev)
        self.dim, self.q_heads, self.tokens = q.shape[-1], q.shape[-2], q.shape[-3]
        self.batch = q.shape[0] if q.dim() == 4 else 1
        self.k_heads = 0
        if k is not None:
            if k.dim() != q.dim():
                raise RuntimeError(f"k must have {q.dim()} dimensions, not {k.dim()}")
            self.k_heads = k.shape[-2]
            _check_heads("k", k, q.dtype, (*q.shape[:-2], self.k_heads, self.dim), dev)
            if self.k_heads < 1:
                raise RuntimeError("k has no heads: leave it out")
        if (k is None) != (k_gamma is None):
            raise RuntimeError("k and k_gamma belong together")
        for name, g in (("q_gamma", q_gamma), ("k_gamma", k_gamma)):
            if g is not None:
                _check_like(name, g, q.dtype, self.dim, (self.dim,))
                _check_cuda(name, g, dev)
        self.rotary = 0
        if inv_freq is not None:
            if inv_freq.dtype not in (torch.float32, torch.float64):
                raise RuntimeError(f"inv_freq must be float32 or float64, not {inv_freq.dtype}")
            if inv_freq.dim() != 1 or 2 * inv_freq.numel() > self.dim:
                raise RuntimeError(f"inv_freq must be one value a pair, at most {self.dim // 2}, "
                                   f"not of shape {tuple(inv_freq.shape)}")
            _check_cuda("inv_freq", inv_freq, dev)
            self.rotary = 2 * inv_freq.numel()
        self.pos_stride = 0
        if positions is not None:
            if positions.dtype not in (torch.int32, torch.int64):
                raise RuntimeError(f"positions must be int32 or int64, not {positions.dtype}")
            if tuple(positions.shape) not in ((self.tokens,), tuple(q.shape[:-2])):
                raise RuntimeError(f"positions must have shape {tuple(q.shape[:-2])} or "
                                   f"{(self.tokens,)}, not {tuple(positions.shape)}")
            _check_strided("positions", positions, dev)
            if self.tokens > 1 and positions.stride(-1) != 1:
                raise RuntimeError("positions must be contiguous in their last dimension")
            self.pos_stride = positions.stride(0) if positions.dim() == 2 else 0

    def turn(self, inv_freq, positions):
        """The C call's arguments of the rotation."""
        return (_address(inv_freq) if self.rotary else None,
                int(inv_freq is not None and inv_freq.dtype == torch.float64),
                _address(positions),
                int(positions is not None and positions.dtype == torch.int64), self.pos_stride)

    def sizes(self):
        return self.batch, self.tokens, self.q_heads, self.k_heads, self.dim, self.rotary


def _flag(fn: str, value) -> int:
    if value not in (False, True):
        raise RMSNormError(fn, RMSN_ERR_ARG)
    return int(value)


def rms_norm_rotary_fwd(q: torch.Tensor, k: Optional[torch.Tensor], q_gamma: torch.Tensor,
                        k_gamma: Optional[torch.Tensor], inv_freq: Optional[torch.Tensor],
                        positions: Optional[torch.Tensor] = None, eps: float = 1e-6,
                        offset: int = 0, interleaved: bool = False,
                        q_out: Optional[torch.Tensor] = None,
                        k_out: Optional[torch.Tensor] = None,
                        rstd_q: Optional[torch.Tensor] = None,
                        rstd_k: Optional[torch.Tensor] = None, with_rstd: bool = True,
                        stream: Optional[torch.cuda.Stream] = None):
    """The norms of queries and keys over each head, and the rotation by the
    token's position.  ``q`` is [tokens, heads, head_dim] or [batch, tokens,
    heads, head_dim], of any strides but the last dimension's (a view of the
    packed product, a head's tokens next to one another); ``k``, with heads of
    its own number, alike, or None together with ``k_gamma``.  ``inv_freq``
    [pairs] (fp32 or fp64) holds the angle a position for each pair of the
    head's first ``2 * pairs`` columns, halves of them paired, or neighbours
    where ``interleaved``; None rotates nothing.  ``positions`` (int32 or
    int64) is [tokens] or q's leading dimensions; None: 0, 1, ... in every
    batch entry; the angle is off by 2^-63 of a turn a position, nothing that
    fp32 shows at positions up to 2^31.  Returns ``(q_out, k_out, rstd_q, rstd_k)``: outputs like
    ``torch.empty_like`` of the inputs, or those given (any strides; the inputs
    themselves for a call in place), and the fp32 statistics that the backward
    reads (None without ``with_rstd``, as in serving)."""
    lib = load_library()
    if _binding is not None and stream is None:
        got = _binding.rotary_fwd(q, k, q_gamma, k_gamma, inv_freq, positions, eps, offset,
                                  interleaved, with_rstd, q_out, k_out, rstd_q, rstd_k)
        if got is not None:
            return got
    fn = "rms_norm_rotary_fwd"
    _check_offset(fn, offset)
    interleaved = _flag(fn, interleaved)
    call = _RotaryCall(q, k, q_gamma, k_gamma, inv_freq, positions)
    dev, dtype = q.device, q.dtype
    given = []
    for name, t, like in (("q_out", q_out, q), ("k_out", k_out, k)):
        if t is not None:
            if like is None:
                raise RuntimeError(f"{name} is given without k")
            _check_heads(name, t, dtype, like.shape, dev)
            given.append(t)
    for name, t, like in (("rstd_q", rstd_q, q), ("rstd_k", rstd_k, k)):
        if t is not None:
            if like is None or not with_rstd:
                raise RuntimeError(f"{name} is given, but not wanted")
            _check_like(name, t, torch.float32, like.numel() // call.dim, like.shape[:-1])
            _check_cuda(name, t, dev)
            given.append(t)
    with _On(dev, stream) as handle:
        q_out = torch.empty_like(q) if q_out is None else q_out
        k_out = torch.empty_like(k) if k_out is None and k is not None else k_out
        if with_rstd and rstd_q is None:
            rstd_q = torch.empty(q.shape[:-1], dtype=torch.float32, device=dev)
        if with_rstd and rstd_k is None and k is not None:
            rstd_k = torch.empty(k.shape[:-1], dtype=torch.float32, device=dev)
        st = lib.rms_norm_rotary_fwd(
            _heads_of(q), _heads_of(k), _address(q_gamma), _address(k_gamma),
            *call.turn(inv_freq, positions), _heads_of(q_out), _heads_of(k_out),
            _address(rstd_q), _address(rstd_k), *call.sizes(), interleaved, float(eps),
            int(offset), DTYPE_CODES[dtype], handle)
    if st != RMSN_OK:
        raise RMSNormError(fn, st)
    _written(*given)
    return q_out, k_out, rstd_q, rstd_k


def rms_norm_rotary_bwd_workspace_size(batch: int, tokens: int, q_heads: int, k_heads: int,
                                       head_dim: int) -> int:
    """Bytes of workspace ``rms_norm_rotary_bwd`` needs: none for few rows."""
    return int(load_library().rms_norm_rotary_bwd_workspace_size(
        int(batch), int(tokens), int(q_heads), int(k_heads), int(head_dim)))


def rms_norm_rotary_bwd(dq_out: torch.Tensor, dk_out: Optional[torch.Tensor], q: torch.Tensor,
                        k: Optional[torch.Tensor], q_gamma: torch.Tensor,
                        k_gamma: Optional[torch.Tensor], rstd_q: torch.Tensor,
                        rstd_k: Optional[torch.Tensor], inv_freq: Optional[torch.Tensor],
                        positions: Optional[torch.Tensor] = None, offset: int = 0,
                        interleaved: bool = False, dq: Optional[torch.Tensor] = None,
                        dk: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None):
    """Backward of ``rms_norm_rotary_fwd`` from the gradients of its outputs, of
    any strides but the last dimension's.  ``dq`` and ``dk`` may be views of the
    packed product's gradient, or ``dq_out`` and ``dk_out`` themselves.  Returns
    ``(dq, dk, dq_gamma, dk_gamma)``, the gammas' gradients fp32 sums."""
    lib = load_library()
    if _binding is not None and stream is None:
        got = _binding.rotary_bwd(dq_out, dk_out, q, k, q_gamma, k_gamma, rstd_q, rstd_k, inv_freq,
                                  positions, offset, interleaved, dq, dk, workspace)
        if got is not None:
            return got
    fn = "rms_norm_rotary_bwd"
    _check_offset(fn, offset)
    interleaved = _flag(fn, interleaved)
    call = _RotaryCall(q, k, q_gamma, k_gamma, inv_freq, positions)
    dev, dtype = q.device, q.dtype
    given = []
    for names, dy, x, rstd, dx in ((("dq_out", "rstd_q", "dq"), dq_out, q, rstd_q, dq),
                                   (("dk_out", "rstd_k", "dk"), dk_out, k, rstd_k, dk)):
        if x is None:
            for name, t in zip(names, (dy, rstd, dx)):
                if t is not None:
                    raise RuntimeError(f"{name} is given without k")
            continue
        _check_heads(names[0], dy, dtype, x.shape, dev)
        if rstd is None:
            raise RuntimeError(f"{names[1]} is missing")
        _check_like(names[1], rstd, torch.float32, x.numel() // call.dim, x.shape[:-1])
        _check_cuda(names[1], rstd, dev)
        if dx is not None:
            _check_heads(names[2], dx, dtype, x.shape, dev)
            given.append(dx)
    if workspace is not None:
        _check_cuda("workspace", workspace, dev)
    with _On(dev, stream) as handle:
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None and k is not None else dk
        dq_gamma = torch.empty(call.dim, dtype=torch.float32, device=dev)
        dk_gamma = None if k is None else torch.empty(call.dim, dtype=torch.float32, device=dev)
        if workspace is None:
            need = int(lib.rms_norm_rotary_bwd_workspace_size(*call.sizes()[:5]))
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        st = lib.rms_norm_rotary_bwd(
            _heads_of(dq_out), _heads_of(dk_out), _heads_of(q), _heads_of(k), _address(q_gamma),
            _address(k_gamma), _address(rstd_q), _address(rstd_k),
            *call.turn(inv_freq, positions), _heads_of(dq), _heads_of(dk), _address(dq_gamma),
            _address(dk_gamma), *call.sizes(), interleaved, int(offset), DTYPE_CODES[dtype],
            _ptr(workspace), workspace.numel() * workspace.element_size(), handle)
    if st != RMSN_OK:
        raise RMSNormError(fn, st)
    _written(*given)
    return dq, dk, dq_gamma, dk_gamma


def _check_ids(ids: torch.Tensor) -> None:
    if ids.dtype not in (torch.int32, torch.int64):
        raise RuntimeError(f"ids must be int32 or int64, not {ids.dtype}")
    _check_cuda("ids", ids)


def _embedding_dtype(name: str, dtype: torch.dtype, other: torch.dtype) -> None:
    if dtype not in DTYPE_CODES:
        raise RuntimeError(f"{name} must be float32, bfloat16 or float16, not {dtype}")
    if dtype != other and torch.float32 not in (dtype, other):
        raise RuntimeError(f"{name} is {dtype} beside {other}: one of the two must be float32")


def rms_norm_embedding_fwd(ids: torch.Tensor, weight: torch.Tensor, scale: float = 1.0,
                           dtype: Optional[torch.dtype] = None, y: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The rows of ``weight`` [vocab, hidden] at ``ids`` (int32 or int64, any
    shape), times ``scale``: ``y`` of shape [*ids.shape, hidden] in ``dtype`` (the
    weight's, or float32 from or to a 16-bit one).  An id outside [0, vocab), as a
    batch's padding, gives a row of zeros.  No norm is applied."""
    lib = load_library()
    if _binding is not None and stream is None:
        got = _binding.embedding_fwd(ids, weight, scale, dtype, y)
        if got is not None:
            return got
    if weight.dim() != 2 or 0 in weight.shape:
        raise RuntimeError(f"weight must be [vocab, hidden], not of shape {tuple(weight.shape)}")
    dev, (vocab, hidden) = weight.device, weight.shape
    shape = (*ids.shape, hidden)
    dtype = (weight.dtype if y is None else y.dtype) if dtype is None else dtype
    _embedding_dtype("weight", weight.dtype, weight.dtype)
    _embedding_dtype("y", dtype, weight.dtype)
    _check_like("y", y, dtype, ids.numel() * hidden, shape)
    _check_ids(ids)
    _check_cuda("weight", weight, ids.device)
    if y is not None:
        _check_cuda("y", y, dev)
    given = y
    with _On(dev, stream) as handle:
        y = torch.empty(shape, dtype=dtype, device=dev) if y is None else y
        st = lib.rms_norm_embedding_fwd(
            _address(ids), int(ids.dtype == torch.int64), _address(weight), _address(y),
            ids.numel(), vocab, hidden, float(scale), DTYPE_CODES[weight.dtype],
            DTYPE_CODES[dtype], handle)
    if st != RMSN_OK:
        raise RMSNormError("rms_norm_embedding_fwd", st)
    _written(given)
    return y


def rms_norm_embedding_bwd_workspace_size(tokens: int, vocab: int, hidden: int) -> int:
    """Bytes of workspace ``rms_norm_embedding_bwd`` needs: none for few tokens."""
    return int(load_library().rms_norm_embedding_bwd_workspace_size(int(tokens), int(vocab),
                                                                    int(hidden)))


def rms_norm_embedding_bwd(dy: torch.Tensor, ids: torch.Tensor, vocab: int, scale: float = 1.0,
                           padding_idx: Optional[int] = None,
                           dtype: Optional[torch.dtype] = None,
                           dweight: Optional[torch.Tensor] = None, accumulate: bool = False,
                           workspace: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Backward of ``rms_norm_embedding_fwd``: ``dweight`` [vocab, hidden], the
    sums of ``scale * dy`` over each id's tokens, in ``dtype`` (float32 where it is
    not given, or dy's, or any under a float32 ``dy``).  Tokens of ``padding_idx``,
    and of ids outside the table, have no part.  With ``accumulate`` the sums are
    added to the ``dweight`` given, of which the tokens' rows alone are touched."""
    lib = load_library()
    if _binding is not None and stream is None:
        got = _binding.embedding_bwd(dy, ids, vocab, scale, padding_idx, dtype, dweight,
                                     accumulate, workspace)
        if got is not None:
            return got
    fn = "rms_norm_embedding_bwd"
    accumulate = _flag(fn, accumulate)
    if accumulate and dweight is None:
        raise RuntimeError("accumulate needs the dweight to add to")
    if dy.dim() < 1 or tuple(dy.shape[:-1]) != tuple(ids.shape):
        raise RuntimeError(f"dy must have shape {tuple(ids.shape)} + (hidden,), not "
                           f"{tuple(dy.shape)}")
    dev, hidden, vocab = dy.device, dy.shape[-1], int(vocab)
    if dtype is None:
        dtype = torch.float32 if dweight is None else dweight.dtype
    _embedding_dtype("dy", dy.dtype, dy.dtype)
    _embedding_dtype("dweight", dtype, dy.dtype)
    if padding_idx is not None and not 0 <= padding_idx < vocab:
        raise RMSNormError(fn, RMSN_ERR_ARG)
    _check_like("dweight", dweight, dtype, vocab * hidden, (vocab, hidden))
    _check_ids(ids)
    _check_cuda("dy", dy, ids.device)
    for name, t in (("dweight", dweight), ("workspace", workspace)):
        if t is not None:
            _check_cuda(name, t, dev)
    given = dweight
    with _On(dev, stream) as handle:
        if dweight is None:
            dweight = torch.empty((max(vocab, 0), hidden), dtype=dtype, device=dev)
        if workspace is None:
            need = int(lib.rms_norm_embedding_bwd_workspace_size(ids.numel(), vocab, hidden))
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        st = lib.rms_norm_embedding_bwd(
            _address(dy), _address(ids), int(ids.dtype == torch.int64), _address(dweight),
            ids.numel(), vocab, hidden, float(scale), -1 if padding_idx is None else padding_idx,
            accumulate, DTYPE_CODES[dy.dtype], DTYPE_CODES[dtype], _ptr(workspace),
            workspace.numel() * workspace.element_size(), handle)
    if st != RMSN_OK:
        raise RMSNormError(fn, st)
    _written(given)
    return dweight


class RMSNormFunction(torch.autograd.Function):
    """RMSNorm over the last dimension with this library's forward and
    backward.  The backward's weight gradient, summed in fp32 by the library,
    is cast to the weight's dtype (autograd wants the parameter's dtype)."""

    @staticmethod
    def forward(ctx, x, weight, eps, offset, cast_mode):
        x = x.contiguous()
        weight = weight.contiguous()
        y, rstd = rms_norm_fwd(x, weight, eps, offset, cast_mode)
        ctx.save_for_backward(x, weight, rstd)
        ctx.offset = offset
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, rstd = ctx.saved_tensors
        dx, dw = rms_norm_bwd(dy.contiguous(), x, weight, rstd, ctx.offset)
        return dx, dw.to(weight.dtype), None, None, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float, offset: int = 0,
             cast_mode: str = "round_once") -> torch.Tensor:
    """Differentiable RMSNorm of ``x`` over its last dimension (gain
    ``weight``, or ``1 + weight`` with ``offset=1``)."""
    return RMSNormFunction.apply(x, weight, eps, offset, cast_mode)


class RMSNorm(torch.nn.Module):
    """RMSNorm layer over the last dimension of its input.  The weight starts
    at 1 (gain ``weight``) or at 0 with ``offset=1`` (gain ``1 + weight``)."""

    def __init__(self, hidden: int, eps: float = 1e-6, offset: int = 0,
                 cast_mode: str = "round_once", device=None, dtype=None):
        super().__init__()
        if offset not in (0, 1):
            raise ValueError("offset must be 0 or 1")
        if cast_mode not in CAST_MODES:
            raise ValueError(f"cast_mode must be one of {sorted(CAST_MODES)}")
        self.weight = torch.nn.Parameter(
            torch.full((hidden,), 0.0 if offset else 1.0, device=device, dtype=dtype))
        self.eps, self.offset, self.cast_mode = eps, offset, cast_mode

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return rms_norm(x, self.weight, self.eps, self.offset, self.cast_mode)

    def extra_repr(self) -> str:
        return (f"{self.weight.numel()}, eps={self.eps}, offset={self.offset}, "
                f"cast_mode={self.cast_mode!r}")


class RMSNormBlockFunction(torch.autograd.Function):
    """The block norm with this library's forward and backward.  The fp32 sums
    of the backward are cast to the parameters' dtype."""

    @staticmethod
    def forward(ctx, x, residual, post_weight, gate, next_weight, eps, offset, residual_scale,
                branch_scale):
        x, residual = x.contiguous(), residual.contiguous()
        weights = [None if w is None else w.contiguous() for w in (post_weight, gate, next_weight)]
        r, y, rstd_post, rstd_next = rms_norm_block_fwd(
            x, residual, *weights, eps, offset, residual_scale, branch_scale)
        ctx.save_for_backward(x, r, rstd_post, rstd_next, *weights)
        ctx.scales = offset, residual_scale, branch_scale
        ctx.set_materialize_grads(False)
        return r if y is None else (r, y)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dr, dy=None):
        x, r, rstd_post, rstd_next, post_weight, gate, next_weight = ctx.saved_tensors
        if dr is None and dy is None:
            return (None,) * 9
        if dy is None and post_weight is None:
            dy = torch.zeros_like(x)       # r alone was used, and there is no other norm
        used_next = None if dy is None else next_weight
        dx, dres, dpost, dgate, dnext = rms_norm_block_bwd(
            None if dy is None else dy.contiguous(), None if dr is None else dr.contiguous(), x, r,
            rstd_post, rstd_next, post_weight, gate, used_next, *ctx.scales,
            with_dgate=ctx.needs_input_grad[3])
        dpost, dgate, dnext = (None if d is None else d.to(x.dtype) for d in (dpost, dgate, dnext))
        return dx, dres, dpost, dgate, dnext, None, None, None, None


def rms_norm_block(x: torch.Tensor, residual: torch.Tensor,
                   post_weight: Optional[torch.Tensor] = None,
                   gate: Optional[torch.Tensor] = None,
                   next_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   offset: int = 0, residual_scale: float = 1.0, branch_scale: float = 1.0):
    """Differentiable ``rms_norm_block_fwd``: returns ``(r, y)``, or ``r``
    alone without ``next_weight``.  Differentiable in x, the residual, both
    weights and the gate.  A training step captured into a CUDA graph is, as
    any with autograd, warmed up on a side stream, with no eager graph of the
    same leaves alive during the capture."""
    return RMSNormBlockFunction.apply(x, residual, post_weight, gate, next_weight, eps, offset,
                                      residual_scale, branch_scale)


class RMSNormBlock(torch.nn.Module):
    """What stands between one transformer block and the next: the norm of the
    block's output (``post``), its gate (``gate_init``: a weight for each
    channel that starts there; or a gate given to the call), the scaled
    residual sum, and the norm before the next block (``next``)."""

    def __init__(self, hidden: int, eps: float = 1e-6, offset: int = 0, post: bool = True,
                 next: bool = True, gate_init: Optional[float] = None,
                 residual_scale: float = 1.0, branch_scale: float = 1.0, device=None, dtype=None):
        super().__init__()
        if offset not in (0, 1):
            raise ValueError("offset must be 0 or 1")
        if not post and not next:
            raise ValueError("post and next are both False: nothing to normalise")

        def weight(value):
            return torch.nn.Parameter(torch.full((hidden,), value, device=device, dtype=dtype))

        start = 0.0 if offset else 1.0
        self.post_weight = weight(start) if post else None
        self.next_weight = weight(start) if next else None
        self.gate = weight(float(gate_init)) if gate_init is not None else None
        self.eps, self.offset = eps, offset
        self.residual_scale, self.branch_scale = residual_scale, branch_scale

    def forward(self, x: torch.Tensor, residual: torch.Tensor,
                gate: Optional[torch.Tensor] = None):
        if gate is not None and self.gate is not None:
            raise ValueError("this layer has a gate of its own")
        return rms_norm_block(x, residual, self.post_weight,
                              self.gate if gate is None else gate, self.next_weight, self.eps,
                              self.offset, self.residual_scale, self.branch_scale)

    def extra_repr(self) -> str:
        return (f"post={self.post_weight is not None}, gate={self.gate is not None}, "
                f"next={self.next_weight is not None}, eps={self.eps}, offset={self.offset}, "
                f"residual_scale={self.residual_scale}, branch_scale={self.branch_scale}")


def _rows_contiguous(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """The tensor where its last dimension is contiguous, else a copy."""
    if t is None or t.shape[-1] <= 1 or t.stride(-1) == 1:
        return t
    return t.contiguous()


class RMSNormRotaryFunction(torch.autograd.Function):
    """The head norm and rotation with this library's forward and backward.  The
    fp32 sums of the backward are cast to the weights' dtype."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, inv_freq, positions, eps, offset, interleaved):
        q, k = _rows_contiguous(q), _rows_contiguous(k)
        q_weight = q_weight.contiguous()
        k_weight = None if k_weight is None else k_weight.contiguous()
        q_out, k_out, rstd_q, rstd_k = rms_norm_rotary_fwd(
            q, k, q_weight, k_weight, inv_freq, positions, eps, offset, interleaved)
        ctx.save_for_backward(q, k, q_weight, k_weight, rstd_q, rstd_k, inv_freq, positions)
        ctx.kind = offset, interleaved
        return q_out if k is None else (q_out, k_out)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out=None):
        q, k, q_weight, k_weight, rstd_q, rstd_k, inv_freq, positions = ctx.saved_tensors
        dq, dk, dwq, dwk = rms_norm_rotary_bwd(
            _rows_contiguous(dq_out), _rows_contiguous(dk_out), q, k, q_weight, k_weight, rstd_q,
            rstd_k, inv_freq, positions, *ctx.kind)
        dwk = None if dwk is None else dwk.to(q.dtype)
        return dq, dk, dwq.to(q.dtype), dwk, None, None, None, None, None


def rms_norm_rotary(q: torch.Tensor, k: Optional[torch.Tensor], q_weight: torch.Tensor,
                    k_weight: Optional[torch.Tensor], inv_freq: Optional[torch.Tensor],
                    positions: Optional[torch.Tensor] = None, eps: float = 1e-6, offset: int = 0,
                    interleaved: bool = False):
    """Differentiable ``rms_norm_rotary_fwd``: returns ``(q_out, k_out)``, or
    ``q_out`` alone without ``k``.  Differentiable in q, k and both weights.  A
    training step captured into a CUDA graph is, as any with autograd, warmed up
    on a side stream, with no eager graph of the same leaves alive during the
    capture."""
    return RMSNormRotaryFunction.apply(q, k, q_weight, k_weight, inv_freq, positions, eps, offset,
                                       interleaved)


class RMSNormRotary(torch.nn.Module):
    """The norms of an attention's queries and keys over each head, with their
    rotation: ``rotary_dim`` columns (all of them where it is not given) turn by
    ``position * base ** (-2 p / rotary_dim)`` for the pair p.  The weights start
    at 1, or at 0 with ``offset=1``.  Other frequencies, as those of a longer
    context, are assigned to ``inv_freq`` (fp64 or fp32, one a pair); casts and
    moves of the module keep them and their dtype.  They are not in the state
    dict, and a module on the meta device gets those of ``base`` when it leaves
    it."""

    def __init__(self, head_dim: int, eps: float = 1e-6, offset: int = 0, base: float = 10000.0,
                 rotary_dim: Optional[int] = None, interleaved: bool = False, device=None,
                 dtype=None):
        super().__init__()
        if offset not in (0, 1):
            raise ValueError("offset must be 0 or 1")
        rotary_dim = head_dim // 2 * 2 if rotary_dim is None else rotary_dim
        if rotary_dim % 2 or not 0 <= rotary_dim <= head_dim:
            raise ValueError(f"rotary_dim must be even and at most {head_dim}")

        def weight():
            return torch.nn.Parameter(torch.full((head_dim,), 0.0 if offset else 1.0,
                                                 device=device, dtype=dtype))

        self.q_weight, self.k_weight = weight(), weight()
        self.eps, self.offset, self.interleaved = eps, offset, interleaved
        self.base, self.rotary_dim = base, rotary_dim
        self.register_buffer("inv_freq", self._frequencies(self.q_weight.device),
                             persistent=False)

    def _frequencies(self, device) -> torch.Tensor:
        p = torch.arange(self.rotary_dim // 2, dtype=torch.float64, device=device)
        return float(self.base) ** (p * (-2.0 / max(self.rotary_dim, 1)))

    def _apply(self, fn, *args, **kwargs):
        freq = self.inv_freq
        super()._apply(fn, *args, **kwargs)
        # the frequencies, assigned ones too, go where the weights go, and stay what
        # they are; on the meta device they have no values to keep
        device = self.q_weight.device
        if freq is not None:
            lost = freq.is_meta and device.type != "meta"
            self.inv_freq = self._frequencies(device) if lost else freq.to(device)
        return self

    def forward(self, q: torch.Tensor, k: torch.Tensor,
                positions: Optional[torch.Tensor] = None):
        return rms_norm_rotary(q, k, self.q_weight, self.k_weight, self.inv_freq, positions,
                               self.eps, self.offset, self.interleaved)

    def extra_repr(self) -> str:
        return (f"{self.q_weight.numel()}, eps={self.eps}, offset={self.offset}, "
                f"base={self.base}, rotary_dim={self.rotary_dim}, "
                f"interleaved={self.interleaved}")


class RMSNormEmbeddingFunction(torch.autograd.Function):
    """The embedding with this library's forward and backward; the weight's
    gradient, summed in fp32, is written in the weight's dtype."""

    @staticmethod
    def forward(ctx, ids, weight, scale, padding_idx, dtype):
        if padding_idx is not None and not 0 <= padding_idx < weight.shape[0]:
            raise RMSNormError("rms_norm_embedding", RMSN_ERR_ARG)  # as the backward would
        ids, weight = ids.contiguous(), weight.contiguous()
        ctx.save_for_backward(ids)
        ctx.table = weight.shape[0], weight.dtype, scale, padding_idx
        return rms_norm_embedding_fwd(ids, weight, scale, dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        (ids,) = ctx.saved_tensors
        vocab, dtype, scale, padding_idx = ctx.table
        dweight = rms_norm_embedding_bwd(dy.contiguous(), ids, vocab, scale, padding_idx, dtype)
        return None, dweight, None, None, None


def rms_norm_embedding(ids: torch.Tensor, weight: torch.Tensor, scale: float = 1.0,
                       padding_idx: Optional[int] = None,
                       dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Differentiable ``rms_norm_embedding_fwd``, in the weight.  Tokens of
    ``padding_idx``, a row of the table, take it, and give it no gradient.
    Captured into a CUDA graph as ``rms_norm_rotary``."""
    return RMSNormEmbeddingFunction.apply(ids, weight, scale, padding_idx, dtype)


class RMSNormEmbedding(torch.nn.Module):
    """A table of ``vocab`` rows, of which a batch of tokens takes its own, times
    ``scale``; ``out_dtype`` float32 begins an fp32 residual stream under 16-bit
    weights (as ``RMSNormBlock`` carries it).  The name has the library's prefix:
    no norm is applied to the rows."""

    def __init__(self, vocab: int, hidden: int, scale: float = 1.0,
                 padding_idx: Optional[int] = None, out_dtype: Optional[torch.dtype] = None,
                 init_std: float = 0.02, device=None, dtype=None):
        super().__init__()
        if padding_idx is not None and not 0 <= padding_idx < vocab:
            raise ValueError(f"padding_idx must be in the table, not {padding_idx}")
        self.weight = torch.nn.Parameter(torch.empty((vocab, hidden), device=device, dtype=dtype))
        with torch.no_grad():
            self.weight.normal_(0.0, init_std)
            if padding_idx is not None:
                self.weight[padding_idx] = 0.0
        self.scale, self.padding_idx, self.out_dtype = scale, padding_idx, out_dtype

    def forward(self, ids: torch.Tensor) -> torch.Tensor:
        return rms_norm_embedding(ids, self.weight, self.scale, self.padding_idx, self.out_dtype)

    def extra_repr(self) -> str:
        return (f"{self.weight.shape[0]}, {self.weight.shape[1]}, scale={self.scale}, "
                f"padding_idx={self.padding_idx}, out_dtype={self.out_dtype}")
