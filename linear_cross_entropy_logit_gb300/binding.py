"""Thin ctypes binding of ``libflce.so`` (include/flce.h).

Argument marshalling only: every step of the forward and backward runs in the
library's CUDA kernels.  PyTorch provides device memory and the stream.  If the
library is missing, ``lib()`` raises instead of falling back to anything.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libflce.so")
# The same library built with FLCE_DEBUG: index math range-checked on the
# device (an out-of-range index sets FLCE_ERR_BOUNDS instead of being used).
DEBUG_LIB_PATH = os.path.join(_HERE, "_lib", "libflce_debug.so")

FLCE_OK = 0
FLCE_ERR_ARG = 1
FLCE_ERR_UNSUPPORTED = 2
FLCE_ERR_WORKSPACE = 3
FLCE_ERR_LABEL = 4
FLCE_ERR_TIMEOUT = 5
FLCE_ERR_CUDA = 6
FLCE_ERR_BOUNDS = 7
FLCE_ERR_INDEX = 8

FLCE_BF16 = 0
FLCE_FP32 = 1
FLCE_MEAN = 0
FLCE_SUM = 1
MODE_FWD = 1
MODE_BWD = 2
MODE_FWD_BWD = 3

EXPORTED = (
    "flce_workspace_size", "flce_set_vocab_chunk", "flce_vocab_chunk", "flce_forward",
    "flce_backward", "flce_fwd_bwd", "flce_status_string", "flce_last_cuda_error",
    "flce_last_launch_count", "flce_abi_version", "flce_debug_gemm", "flce_profile_enable",
    "flce_profile_read", "flce_profile_reset", "flce_forward_noalloc", "flce_noalloc_last_error",
    "flce_set_cta_pair", "flce_cta_pair", "flce_set_l2_hints", "flce_options_init",
    "flce_forward_ex", "flce_backward_ex", "flce_fwd_bwd_ex", "flce_forward_vocab_shard",
    "flce_combine_workspace_size", "flce_combine_vocab_shards", "flce_backward_vocab_shard",
    "flce_debug_wait_timeout", "flce_set_backward_merge", "flce_backward_merge",
    "flce_workspace_size_ex", "flce_vocab_chunk_ex", "flce_set_cluster_multicast",
    "flce_cluster_multicast", "flce_debug_last_multicast_launches",
    "flce_qk_norm_rope_forward", "flce_qk_norm_rope_workspace_size", "flce_qk_norm_rope_backward",
    "flce_attention_forward", "flce_attention_workspace_size", "flce_attention_backward",
    "flce_layer_norm_forward", "flce_layer_norm_workspace_size", "flce_layer_norm_backward",
    "flce_rope_forward", "flce_rope_backward",
    "flce_distill_workspace_size", "flce_distill_forward", "flce_distill_backward",
)

PROFILE_KINDS = ("fwd_logits_lse", "bwd_dz_recompute", "bwd_dw_gemm", "bwd_dx_gemm",
                 "bwd_merged")

_lib = None


class FlceOptions(ctypes.Structure):
    """Mirror of ``flce_options`` in include/flce.h."""
    _fields_ = [("struct_size", ctypes.c_size_t), ("ignore_index", ctypes.c_int64),
                ("smoothing", ctypes.c_float), ("z_loss", ctypes.c_float),
                ("reduction", ctypes.c_int), ("row_loss", ctypes.c_void_p),
                ("skip_ignored_blocks", ctypes.c_int), ("grad_filter", ctypes.c_float),
                ("cta_pair", ctypes.c_int), ("backward_merge", ctypes.c_int),
                ("l2_hints", ctypes.c_int), ("vocab_chunk", ctypes.c_int64),
                ("cluster_multicast", ctypes.c_int)]


class FlceQkNormRopeDesc(ctypes.Structure):
    """Mirror of ``flce_qk_norm_rope_desc`` in include/flce.h."""
    _fields_ = [("struct_size", ctypes.c_size_t), ("tokens", ctypes.c_int64),
                ("q_heads", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("rot_dim", ctypes.c_int64),
                ("table_rows", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("eps", ctypes.c_float), ("interleaved", ctypes.c_int),
                ("q_row", ctypes.c_int64), ("q_head", ctypes.c_int64),
                ("k_row", ctypes.c_int64), ("k_head", ctypes.c_int64)]


class FlceAttentionDesc(ctypes.Structure):
    """Mirror of ``flce_attention_desc`` in include/flce.h."""
    _fields_ = [("struct_size", ctypes.c_size_t), ("tokens", ctypes.c_int64),
                ("sequences", ctypes.c_int64), ("q_heads", ctypes.c_int64),
                ("kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("scale", ctypes.c_float),
                ("q_row", ctypes.c_int64), ("q_head", ctypes.c_int64),
                ("k_row", ctypes.c_int64), ("k_head", ctypes.c_int64),
                ("v_row", ctypes.c_int64), ("v_head", ctypes.c_int64)]


class FlceLayerNormDesc(ctypes.Structure):
    """Mirror of ``flce_layer_norm_desc`` in include/flce.h."""
    _fields_ = [("struct_size", ctypes.c_size_t), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("rms", ctypes.c_int), ("x_row", ctypes.c_int64),
                ("residual_row", ctypes.c_int64)]


class FlceRopeDesc(ctypes.Structure):
    """Mirror of ``flce_rope_desc`` in include/flce.h."""
    _fields_ = [("struct_size", ctypes.c_size_t), ("tokens", ctypes.c_int64),
                ("q_heads", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("rot_dim", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("magnitude", ctypes.c_float),
                ("interleaved", ctypes.c_int), ("q_row", ctypes.c_int64),
                ("q_head", ctypes.c_int64), ("k_row", ctypes.c_int64),
                ("k_head", ctypes.c_int64)]


class FlceDistillDesc(ctypes.Structure):
    """Mirror of ``flce_distill_desc`` in include/flce.h."""
    _fields_ = [("struct_size", ctypes.c_size_t), ("N", ctypes.c_int64), ("H", ctypes.c_int64),
                ("V", ctypes.c_int64), ("K", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("teacher_dtype", ctypes.c_int), ("dw_dtype", ctypes.c_int),
                ("temperature", ctypes.c_float), ("reduction", ctypes.c_int)]


_DISTILL_DESC_BYTES = ctypes.sizeof(FlceDistillDesc)
_LAYER_NORM_DESC_BYTES = ctypes.sizeof(FlceLayerNormDesc)
_ROPE_DESC_BYTES = ctypes.sizeof(FlceRopeDesc)
_QK_DESC_BYTES = ctypes.sizeof(FlceQkNormRopeDesc)
_ATTENTION_DESC_BYTES = ctypes.sizeof(FlceAttentionDesc)


class FlceError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        detail = ""
        if status == FLCE_ERR_CUDA:
            detail = " (" + lib().flce_last_cuda_error().decode() + ")"
        super().__init__(f"{what}: {lib().flce_status_string(status).decode()}{detail}")


def lib() -> ctypes.CDLL:
    """Load the library (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        _lib = load(LIB_PATH)
    return _lib


def use_library(L: Optional[ctypes.CDLL]) -> Optional[ctypes.CDLL]:
    """Make every wrapper below call ``L`` (e.g. ``load(DEBUG_LIB_PATH)``);
    returns the library used before.  ``None`` goes back to the default."""
    global _lib
    prev = _lib
    _lib = L
    return prev


def load(path: str) -> ctypes.CDLL:
    """Open a build of the library and declare its C signatures."""
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with "
            "`python -m linear_cross_entropy_logit_gb300.build` (needs nvcc)")
    L = ctypes.CDLL(path)
    P, I64, I32, F32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.flce_workspace_size.argtypes = [I64, I64, I64, I32, I32]
    L.flce_workspace_size.restype = SZ
    L.flce_set_vocab_chunk.argtypes = [I64]
    L.flce_set_vocab_chunk.restype = I32
    L.flce_vocab_chunk.argtypes = [I64, I64, I64]
    L.flce_vocab_chunk.restype = I64
    L.flce_forward.argtypes = [P, P, P, I64, I64, I64, I64, F32, I32, I32, P, P, P, P, SZ, P, P]
    L.flce_forward.restype = I32
    L.flce_backward.argtypes = [P, P, P, I64, I64, I64, I64, F32, I32, I32, P, P, P, P, P, I32,
                                P, SZ, P, P]
    L.flce_backward.restype = I32
    L.flce_fwd_bwd.argtypes = [P, P, P, I64, I64, I64, I64, F32, I32, I32, P, P, P, P, P, P, I32,
                               P, SZ, P, P]
    L.flce_fwd_bwd.restype = I32
    L.flce_status_string.argtypes = [I32]
    L.flce_status_string.restype = ctypes.c_char_p
    L.flce_last_cuda_error.argtypes = []
    L.flce_last_cuda_error.restype = ctypes.c_char_p
    L.flce_last_launch_count.argtypes = []
    L.flce_last_launch_count.restype = I32
    L.flce_abi_version.argtypes = []
    L.flce_abi_version.restype = I32
    L.flce_debug_gemm.argtypes = [P, P, P, I64, I64, I64, I32, I32, I32, P, P]
    L.flce_debug_gemm.restype = I32
    L.flce_profile_enable.argtypes = [I32]
    L.flce_profile_enable.restype = I32
    L.flce_profile_read.argtypes = [I32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(I32)]
    L.flce_profile_read.restype = I32
    L.flce_profile_reset.argtypes = []
    L.flce_profile_reset.restype = None
    L.flce_forward_noalloc.argtypes = [P, P, P, I64, I64, I64, I64, F32, I32, P, P, P, P, P]
    L.flce_forward_noalloc.restype = I32
    L.flce_noalloc_last_error.argtypes = []
    L.flce_noalloc_last_error.restype = ctypes.c_char_p
    L.flce_set_cta_pair.argtypes = [I32]
    L.flce_set_cta_pair.restype = I32
    L.flce_cta_pair.argtypes = []
    L.flce_cta_pair.restype = I32
    L.flce_set_l2_hints.argtypes = [I32]
    L.flce_set_l2_hints.restype = I32
    L.flce_set_backward_merge.argtypes = [I32]
    L.flce_set_backward_merge.restype = I32
    L.flce_backward_merge.argtypes = []
    L.flce_backward_merge.restype = I32
    OPT = ctypes.POINTER(FlceOptions)
    L.flce_options_init.argtypes = [OPT]
    L.flce_options_init.restype = None
    L.flce_forward_ex.argtypes = [P, P, P, I64, I64, I64, I32, OPT, P, P, P, P, SZ, P, P]
    L.flce_forward_ex.restype = I32
    L.flce_backward_ex.argtypes = [P, P, P, I64, I64, I64, I32, OPT, P, P, P, P, P, I32, P, SZ,
                                   P, P]
    L.flce_backward_ex.restype = I32
    L.flce_fwd_bwd_ex.argtypes = [P, P, P, I64, I64, I64, I32, OPT, P, P, P, P, P, P, I32, P, SZ,
                                  P, P]
    L.flce_fwd_bwd_ex.restype = I32
    L.flce_forward_vocab_shard.argtypes = [P, P, P, I64, I64, I64, I64, I64, I32, OPT, P, P, SZ,
                                           P, P]
    L.flce_forward_vocab_shard.restype = I32
    L.flce_combine_workspace_size.argtypes = [I64]
    L.flce_combine_workspace_size.restype = SZ
    L.flce_combine_vocab_shards.argtypes = [P, I32, I64, P, I64, OPT, P, P, P, P, SZ, P, P]
    L.flce_combine_vocab_shards.restype = I32
    L.flce_backward_vocab_shard.argtypes = [P, P, P, I64, I64, I64, I64, I64, I32, OPT, P, P, P,
                                            P, P, I32, P, SZ, P, P]
    L.flce_backward_vocab_shard.restype = I32
    L.flce_debug_wait_timeout.argtypes = [P, ctypes.c_uint64, P, P]
    L.flce_debug_wait_timeout.restype = I32
    L.flce_workspace_size_ex.argtypes = [I64, I64, I64, I32, I32, OPT]
    L.flce_workspace_size_ex.restype = SZ
    L.flce_vocab_chunk_ex.argtypes = [I64, I64, I64, OPT]
    L.flce_vocab_chunk_ex.restype = I64
    L.flce_set_cluster_multicast.argtypes = [I32]
    L.flce_set_cluster_multicast.restype = I32
    L.flce_cluster_multicast.argtypes = []
    L.flce_cluster_multicast.restype = I32
    L.flce_debug_last_multicast_launches.argtypes = []
    L.flce_debug_last_multicast_launches.restype = I32
    QD, AD = ctypes.POINTER(FlceQkNormRopeDesc), ctypes.POINTER(FlceAttentionDesc)
    L.flce_qk_norm_rope_forward.argtypes = [QD, P, P, P, P, P, P, P, P, P, P, P]
    L.flce_qk_norm_rope_forward.restype = I32
    L.flce_qk_norm_rope_workspace_size.argtypes = [QD]
    L.flce_qk_norm_rope_workspace_size.restype = SZ
    L.flce_qk_norm_rope_backward.argtypes = [QD, P, P, P, P, P, P, P, P, P, P, P, P, P, P, SZ, P, P]
    L.flce_qk_norm_rope_backward.restype = I32
    L.flce_attention_forward.argtypes = [AD, P, P, P, P, P, P, P, P]
    L.flce_attention_forward.restype = I32
    L.flce_attention_workspace_size.argtypes = [AD]
    L.flce_attention_workspace_size.restype = SZ
    L.flce_attention_backward.argtypes = [AD, P, P, P, P, P, P, P, P, P, P, P, SZ, P, P]
    L.flce_attention_backward.restype = I32
    DD = ctypes.POINTER(FlceDistillDesc)
    L.flce_distill_workspace_size.argtypes = [DD, I32]
    L.flce_distill_workspace_size.restype = SZ
    L.flce_distill_forward.argtypes = [DD, P, P, P, P, P, P, P, P, P, P, P, SZ, P, P]
    L.flce_distill_forward.restype = I32
    L.flce_distill_backward.argtypes = [DD, P, P, P, P, P, P, P, P, P, P, P, I32, P, SZ, P, P]
    L.flce_distill_backward.restype = I32
    ND, RD = ctypes.POINTER(FlceLayerNormDesc), ctypes.POINTER(FlceRopeDesc)
    L.flce_layer_norm_forward.argtypes = [ND, P, P, P, P, P, P, P, P, P]
    L.flce_layer_norm_forward.restype = I32
    L.flce_layer_norm_workspace_size.argtypes = [ND]
    L.flce_layer_norm_workspace_size.restype = SZ
    L.flce_layer_norm_backward.argtypes = [ND, P, P, P, P, P, P, P, P, P, P, SZ, P]
    L.flce_layer_norm_backward.restype = I32
    L.flce_rope_forward.argtypes = [RD, P, P, P, P, P, P, P]
    L.flce_rope_forward.restype = I32
    L.flce_rope_backward.argtypes = [RD, P, P, P, P, P, P, P]
    L.flce_rope_backward.restype = I32
    return L


def _check(status: int, what: str) -> None:
    if status != FLCE_OK:
        raise FlceError(status, what)


def _dtype_code(t: torch.Tensor, names: str = "X and W") -> int:
    if t.dtype == torch.bfloat16:
        return FLCE_BF16
    if t.dtype == torch.float32:
        return FLCE_FP32
    raise TypeError(f"{names} must be bfloat16 or float32, got {t.dtype}")


def _red_code(reduction: str) -> int:
    if reduction == "mean":
        return FLCE_MEAN
    if reduction == "sum":
        return FLCE_SUM
    raise ValueError(f"reduction must be 'mean' or 'sum', got {reduction!r}")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _current_device() -> int:
    return torch._C._cuda_getDevice()


def _check_device(name, t):
    """Refuses a CUDA tensor of another GPU than the one that the library launches on."""
    if t.get_device() != _current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_current_device()}")


def _check_inputs(X, W, labels):
    for name, t in (("X", X), ("W", W), ("labels", labels)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
        _check_device(name, t)
    if X.dtype != W.dtype:
        raise TypeError("X and W must have the same dtype")
    if labels.dtype != torch.int64:
        raise TypeError("labels must be int64")
    N, H = X.shape
    V, H2 = W.shape
    if H2 != H or labels.shape != (N,):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}, labels {tuple(labels.shape)}")
    return N, H, V


def flce_workspace_size(N: int, H: int, V: int, dtype: int = FLCE_BF16, mode: int = MODE_FWD_BWD,
                        options: Optional["FlceOptions"] = None) -> int:
    """Workspace bytes; with ``options`` the launch settings are taken from them
    (flce_workspace_size_ex), else from the process-wide defaults."""
    if options is None:
        return int(lib().flce_workspace_size(N, H, V, dtype, mode))
    return int(lib().flce_workspace_size_ex(N, H, V, dtype, mode, ctypes.byref(options)))


def flce_set_vocab_chunk(cols: int) -> None:
    _check(lib().flce_set_vocab_chunk(cols), "flce_set_vocab_chunk")


def flce_set_cta_pair(on: bool) -> None:
    """1: 256 x 256 tiles on CTA pairs (default); 0: 128 x 256 tiles on single CTAs."""
    _check(lib().flce_set_cta_pair(int(bool(on))), "flce_set_cta_pair")


def flce_set_l2_hints(on: bool) -> None:
    _check(lib().flce_set_l2_hints(int(bool(on))), "flce_set_l2_hints")


def flce_cta_pair() -> bool:
    return bool(lib().flce_cta_pair())


def flce_set_cluster_multicast(on: bool) -> None:
    """1: pair launches whose tiles pair up take 4-CTA clusters with operand
    multicast (default); 0: plain CTA pairs.  Bit-identical results."""
    _check(lib().flce_set_cluster_multicast(int(bool(on))), "flce_set_cluster_multicast")


def flce_cluster_multicast() -> bool:
    return bool(lib().flce_cluster_multicast())


def flce_set_backward_merge(mode) -> None:
    """Backward layout: 0 three launches per chunk (default); 1 (or True) one
    merged dW(c) + dX(c) + dZ(c+1) launch per chunk (two dZ buffers); 2 the dZ
    recompute alone, then one merged dW(c) + dX(c) launch (one dZ buffer)."""
    _check(lib().flce_set_backward_merge(int(mode)), "flce_set_backward_merge")


def flce_backward_merge() -> int:
    return int(lib().flce_backward_merge())


def flce_vocab_chunk(N: int, H: int, V: int, options: Optional["FlceOptions"] = None) -> int:
    if options is None:
        return int(lib().flce_vocab_chunk(N, H, V))
    return int(lib().flce_vocab_chunk_ex(N, H, V, ctypes.byref(options)))


def workspace(N: int, H: int, V: int, dtype: int, mode: int, device,
              options: Optional["FlceOptions"] = None) -> torch.Tensor:
    """A workspace of the required size (torch-allocated, 256-byte aligned)."""
    n = flce_workspace_size(N, H, V, dtype, mode, options)
    if n == 0:
        raise ValueError(f"no workspace plan for N={N}, H={H}, V={V} with these options")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def new_err_word(device) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


def make_options(ignore_index: int = -100, smoothing: float = 0.0, reduction: str = "mean",
                 z_loss: float = 0.0, row_loss=None, skip_ignored_blocks: bool = False,
                 grad_filter: float = 0.0, *, cta_pair: Optional[bool] = None,
                 backward_merge: Optional[int] = None, l2_hints: Optional[bool] = None,
                 vocab_chunk: Optional[int] = None,
                 cluster_multicast: Optional[bool] = None) -> FlceOptions:
    """An ``flce_options``; the launch settings left at None take the
    process-wide defaults at the time of each call."""
    o = FlceOptions()
    lib().flce_options_init(ctypes.byref(o))
    o.ignore_index = ignore_index
    o.smoothing = smoothing
    o.z_loss = z_loss
    o.reduction = _red_code(reduction)
    o.row_loss = _ptr(row_loss)
    o.skip_ignored_blocks = int(bool(skip_ignored_blocks))
    o.grad_filter = grad_filter
    if cta_pair is not None:
        o.cta_pair = int(bool(cta_pair))
    if backward_merge is not None:
        o.backward_merge = int(backward_merge)
    if l2_hints is not None:
        o.l2_hints = int(bool(l2_hints))
    if vocab_chunk is not None:
        o.vocab_chunk = int(vocab_chunk)
    if cluster_multicast is not None:
        o.cluster_multicast = int(bool(cluster_multicast))
    return o


def flce_forward(X, W, labels, ignore_index: int = -100, smoothing: float = 0.0,
                 reduction: str = "mean", *, loss=None, lse=None, valid_count=None,
                 workspace_buf=None, err_word=None, stream=None, z_loss: float = 0.0,
                 row_loss=None, skip_ignored_blocks: bool = False):
    """Returns (loss[1] fp32, lse[N] fp32, valid_count[1] int32, err_word[1] int32).
    With z_loss, row_loss or skip_ignored_blocks set it calls flce_forward_ex."""
    if z_loss or row_loss is not None or skip_ignored_blocks:
        return flce_forward_ex(X, W, labels, make_options(ignore_index, smoothing, reduction,
                                                          z_loss, row_loss, skip_ignored_blocks),
                               loss=loss, lse=lse, valid_count=valid_count,
                               workspace_buf=workspace_buf, err_word=err_word, stream=stream)
    N, H, V = _check_inputs(X, W, labels)
    dev = X.device
    dt = _dtype_code(X)
    loss = torch.empty(1, dtype=torch.float32, device=dev) if loss is None else loss
    lse = torch.empty(N, dtype=torch.float32, device=dev) if lse is None else lse
    valid_count = torch.empty(1, dtype=torch.int32, device=dev) if valid_count is None else valid_count
    ws = workspace(N, H, V, dt, MODE_FWD, dev) if workspace_buf is None else workspace_buf
    err_word = new_err_word(dev) if err_word is None else err_word
    st = lib().flce_forward(_ptr(X), _ptr(W), _ptr(labels), N, H, V, ignore_index, smoothing, dt,
                            _red_code(reduction), _ptr(loss), _ptr(lse), _ptr(valid_count),
                            _ptr(ws), ws.numel(), _ptr(err_word), _stream(stream))
    _check(st, "flce_forward")
    return loss, lse, valid_count, err_word


def flce_forward_ex(X, W, labels, options: FlceOptions, *, loss=None, lse=None,
                    valid_count=None, workspace_buf=None, err_word=None, stream=None):
    N, H, V = _check_inputs(X, W, labels)
    dev = X.device
    dt = _dtype_code(X)
    loss = torch.empty(1, dtype=torch.float32, device=dev) if loss is None else loss
    lse = torch.empty(N, dtype=torch.float32, device=dev) if lse is None else lse
    valid_count = torch.empty(1, dtype=torch.int32, device=dev) if valid_count is None else valid_count
    ws = workspace(N, H, V, dt, MODE_FWD, dev, options) if workspace_buf is None else workspace_buf
    err_word = new_err_word(dev) if err_word is None else err_word
    st = lib().flce_forward_ex(_ptr(X), _ptr(W), _ptr(labels), N, H, V, dt, ctypes.byref(options),
                               _ptr(loss), _ptr(lse), _ptr(valid_count), _ptr(ws), ws.numel(),
                               _ptr(err_word), _stream(stream))
    _check(st, "flce_forward_ex")
    return loss, lse, valid_count, err_word


def flce_backward(X, W, labels, lse, valid_count, ignore_index: int = -100,
                  smoothing: float = 0.0, reduction: str = "mean", *, grad_loss=None,
                  dX=None, dW=None, accumulate_dW: bool = False, workspace_buf=None,
                  err_word=None, stream=None, z_loss: float = 0.0,
                  skip_ignored_blocks: bool = False, grad_filter: float = 0.0):
    """Returns (dX [N, H] in X's dtype, dW [V, H] fp32, err_word).
    With z_loss, skip_ignored_blocks or grad_filter set it calls flce_backward_ex."""
    if z_loss or skip_ignored_blocks or grad_filter:
        return flce_backward_ex(X, W, labels, lse, valid_count,
                                make_options(ignore_index, smoothing, reduction, z_loss,
                                             skip_ignored_blocks=skip_ignored_blocks,
                                             grad_filter=grad_filter),
                                grad_loss=grad_loss, dX=dX, dW=dW, accumulate_dW=accumulate_dW,
                                workspace_buf=workspace_buf, err_word=err_word, stream=stream)
    N, H, V = _check_inputs(X, W, labels)
    dev = X.device
    dt = _dtype_code(X)
    dX = torch.empty_like(X) if dX is None else dX
    if dW is None:
        if accumulate_dW:
            raise ValueError("accumulate_dW needs an existing dW")
        dW = torch.empty(V, H, dtype=torch.float32, device=dev)
    ws = workspace(N, H, V, dt, MODE_BWD, dev) if workspace_buf is None else workspace_buf
    err_word = new_err_word(dev) if err_word is None else err_word
    st = lib().flce_backward(_ptr(X), _ptr(W), _ptr(labels), N, H, V, ignore_index, smoothing, dt,
                             _red_code(reduction), _ptr(lse), _ptr(valid_count), _ptr(grad_loss),
                             _ptr(dX), _ptr(dW), int(bool(accumulate_dW)), _ptr(ws), ws.numel(),
                             _ptr(err_word), _stream(stream))
    _check(st, "flce_backward")
    return dX, dW, err_word


def flce_backward_ex(X, W, labels, lse, valid_count, options: FlceOptions, *, grad_loss=None,
                     dX=None, dW=None, accumulate_dW: bool = False, workspace_buf=None,
                     err_word=None, stream=None):
    N, H, V = _check_inputs(X, W, labels)
    dev = X.device
    dt = _dtype_code(X)
    dX = torch.empty_like(X) if dX is None else dX
    if dW is None:
        if accumulate_dW:
            raise ValueError("accumulate_dW needs an existing dW")
        dW = torch.empty(V, H, dtype=torch.float32, device=dev)
    ws = workspace(N, H, V, dt, MODE_BWD, dev, options) if workspace_buf is None else workspace_buf
    err_word = new_err_word(dev) if err_word is None else err_word
    st = lib().flce_backward_ex(_ptr(X), _ptr(W), _ptr(labels), N, H, V, dt,
                                ctypes.byref(options), _ptr(lse), _ptr(valid_count),
                                _ptr(grad_loss), _ptr(dX), _ptr(dW), int(bool(accumulate_dW)),
                                _ptr(ws), ws.numel(), _ptr(err_word), _stream(stream))
    _check(st, "flce_backward_ex")
    return dX, dW, err_word


def flce_fwd_bwd(X, W, labels, ignore_index: int = -100, smoothing: float = 0.0,
                 reduction: str = "mean", *, grad_loss=None, loss=None, lse=None,
                 valid_count=None, dX=None, dW=None, accumulate_dW: bool = False,
                 workspace_buf=None, err_word=None, stream=None, z_loss: float = 0.0,
                 row_loss=None, skip_ignored_blocks: bool = False, grad_filter: float = 0.0):
    """Returns (loss, lse, valid_count, dX, dW, err_word).
    With z_loss, row_loss, skip_ignored_blocks or grad_filter set it calls flce_fwd_bwd_ex."""
    if z_loss or row_loss is not None or skip_ignored_blocks or grad_filter:
        return flce_fwd_bwd_ex(X, W, labels, make_options(ignore_index, smoothing, reduction,
                                                          z_loss, row_loss, skip_ignored_blocks,
                                                          grad_filter),
                               grad_loss=grad_loss, loss=loss, lse=lse, valid_count=valid_count,
                               dX=dX, dW=dW, accumulate_dW=accumulate_dW,
                               workspace_buf=workspace_buf, err_word=err_word, stream=stream)
    N, H, V = _check_inputs(X, W, labels)
    dev = X.device
    dt = _dtype_code(X)
    loss = torch.empty(1, dtype=torch.float32, device=dev) if loss is None else loss
    lse = torch.empty(N, dtype=torch.float32, device=dev) if lse is None else lse
    valid_count = torch.empty(1, dtype=torch.int32, device=dev) if valid_count is None else valid_count
    dX = torch.empty_like(X) if dX is None else dX
    if dW is None:
        if accumulate_dW:
            raise ValueError("accumulate_dW needs an existing dW")
        dW = torch.empty(V, H, dtype=torch.float32, device=dev)
    ws = workspace(N, H, V, dt, MODE_FWD_BWD, dev) if workspace_buf is None else workspace_buf
    err_word = new_err_word(dev) if err_word is None else err_word
    st = lib().flce_fwd_bwd(_ptr(X), _ptr(W), _ptr(labels), N, H, V, ignore_index, smoothing, dt,
                            _red_code(reduction), _ptr(grad_loss), _ptr(loss), _ptr(lse),
                            _ptr(valid_count), _ptr(dX), _ptr(dW), int(bool(accumulate_dW)),
                            _ptr(ws), ws.numel(), _ptr(err_word), _stream(stream))
    _check(st, "flce_fwd_bwd")
    return loss, lse, valid_count, dX, dW, err_word


def flce_fwd_bwd_ex(X, W, labels, options: FlceOptions, *, grad_loss=None, loss=None, lse=None,
                    valid_count=None, dX=None, dW=None, accumulate_dW: bool = False,
                    workspace_buf=None, err_word=None, stream=None):
    N, H, V = _check_inputs(X, W, labels)
    dev = X.device
    dt = _dtype_code(X)
    loss = torch.empty(1, dtype=torch.float32, device=dev) if loss is None else loss
    lse = torch.empty(N, dtype=torch.float32, device=dev) if lse is None else lse
    valid_count = torch.empty(1, dtype=torch.int32, device=dev) if valid_count is None else valid_count
    dX = torch.empty_like(X) if dX is None else dX
    if dW is None:
        if accumulate_dW:
            raise ValueError("accumulate_dW needs an existing dW")
        dW = torch.empty(V, H, dtype=torch.float32, device=dev)
    ws = workspace(N, H, V, dt, MODE_FWD_BWD, dev, options) if workspace_buf is None else workspace_buf
    err_word = new_err_word(dev) if err_word is None else err_word
    st = lib().flce_fwd_bwd_ex(_ptr(X), _ptr(W), _ptr(labels), N, H, V, dt, ctypes.byref(options),
                               _ptr(grad_loss), _ptr(loss), _ptr(lse), _ptr(valid_count),
                               _ptr(dX), _ptr(dW), int(bool(accumulate_dW)), _ptr(ws),
                               ws.numel(), _ptr(err_word), _stream(stream))
    _check(st, "flce_fwd_bwd_ex")
    return loss, lse, valid_count, dX, dW, err_word


def flce_forward_vocab_shard(X, W_shard, labels, vocab_offset: int, vocab_total: int,
                             options: FlceOptions = None, *, partials=None, workspace_buf=None,
                             err_word=None, stream=None):
    """This shard's per-row partial statistics, a float32 [N, 4] tensor."""
    N, H, Vs = _check_inputs(X, W_shard, labels)
    dev = X.device
    dt = _dtype_code(X)
    options = make_options() if options is None else options
    partials = torch.empty(N, 4, dtype=torch.float32, device=dev) if partials is None else partials
    ws = workspace(N, H, Vs, dt, MODE_FWD, dev, options) if workspace_buf is None else workspace_buf
    err_word = new_err_word(dev) if err_word is None else err_word
    st = lib().flce_forward_vocab_shard(_ptr(X), _ptr(W_shard), _ptr(labels), N, H, Vs,
                                        vocab_offset, vocab_total, dt, ctypes.byref(options),
                                        _ptr(partials), _ptr(ws), ws.numel(), _ptr(err_word),
                                        _stream(stream))
    _check(st, "flce_forward_vocab_shard")
    return partials, err_word


def flce_combine_vocab_shards(partials, labels, vocab_total: int, options: FlceOptions = None, *,
                              loss=None, lse=None, valid_count=None, err_word=None, stream=None):
    """LSE-combine of P shards' partials (float32 [P, N, 4]) -> (loss, lse, valid_count, err)."""
    _check_device("partials", partials)
    n_shards, N = partials.shape[0], partials.shape[1]
    dev = partials.device
    options = make_options() if options is None else options
    loss = torch.empty(1, dtype=torch.float32, device=dev) if loss is None else loss
    lse = torch.empty(N, dtype=torch.float32, device=dev) if lse is None else lse
    valid_count = torch.empty(1, dtype=torch.int32, device=dev) if valid_count is None else valid_count
    n = max(int(lib().flce_combine_workspace_size(N)), 256)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    err_word = new_err_word(dev) if err_word is None else err_word
    st = lib().flce_combine_vocab_shards(_ptr(partials.contiguous()), n_shards, N, _ptr(labels),
                                         vocab_total, ctypes.byref(options), _ptr(loss), _ptr(lse),
                                         _ptr(valid_count), _ptr(ws), ws.numel(), _ptr(err_word),
                                         _stream(stream))
    _check(st, "flce_combine_vocab_shards")
    return loss, lse, valid_count, err_word


def flce_backward_vocab_shard(X, W_shard, labels, vocab_offset: int, vocab_total: int, lse,
                              valid_count, options: FlceOptions = None, *, grad_loss=None,
                              dX_partial=None, dW_shard=None, accumulate_dW: bool = False,
                              workspace_buf=None, err_word=None, stream=None):
    """(fp32 partial dX [N, H], dW rows of this shard [V_shard, H] fp32, err)."""
    N, H, Vs = _check_inputs(X, W_shard, labels)
    dev = X.device
    dt = _dtype_code(X)
    options = make_options() if options is None else options
    dX_partial = torch.empty(N, H, dtype=torch.float32, device=dev) if dX_partial is None else dX_partial
    dW_shard = torch.empty(Vs, H, dtype=torch.float32, device=dev) if dW_shard is None else dW_shard
    ws = workspace(N, H, Vs, dt, MODE_BWD, dev, options) if workspace_buf is None else workspace_buf
    err_word = new_err_word(dev) if err_word is None else err_word
    st = lib().flce_backward_vocab_shard(_ptr(X), _ptr(W_shard), _ptr(labels), N, H, Vs,
                                         vocab_offset, vocab_total, dt, ctypes.byref(options),
                                         _ptr(lse), _ptr(valid_count), _ptr(grad_loss),
                                         _ptr(dX_partial), _ptr(dW_shard), int(bool(accumulate_dW)),
                                         _ptr(ws), ws.numel(), _ptr(err_word), _stream(stream))
    _check(st, "flce_backward_vocab_shard")
    return dX_partial, dW_shard, err_word


def flce_debug_gemm(A, B, M: int, Nn: int, K: int, a_mn: bool, b_mn: bool, D=None,
                    accumulate: bool = False, err_word=None, stream=None):
    """Test-only: D (M x Nn fp32) = A B^T through the tcgen05 GEMM core."""
    dev = A.device
    D = torch.empty(M, Nn, dtype=torch.float32, device=dev) if D is None else D
    err_word = new_err_word(dev) if err_word is None else err_word
    st = lib().flce_debug_gemm(_ptr(A), _ptr(B), _ptr(D), M, Nn, K, int(a_mn), int(b_mn),
                               int(accumulate), _ptr(err_word), _stream(stream))
    _check(st, "flce_debug_gemm")
    return D, err_word


def flce_forward_noalloc(X, W, labels, ignore_index: int = -100, smoothing: float = 0.0,
                         reduction: str = "mean", *, loss, lse, valid_count, err_word,
                         stream=None):
    """Forward for callers that cannot allocate: every output buffer is the
    caller's and no workspace is passed (the library uses its own fixed device
    scratch).  bf16 X and W only.  Returns (loss, lse, valid_count, err_word)."""
    N, H, V = _check_inputs(X, W, labels)
    if X.dtype != torch.bfloat16:
        raise TypeError("flce_forward_noalloc takes bf16 X and W")
    st = lib().flce_forward_noalloc(_ptr(X), _ptr(W), _ptr(labels), N, H, V, ignore_index,
                                    smoothing, _red_code(reduction), _ptr(loss), _ptr(lse),
                                    _ptr(valid_count), _ptr(err_word), _stream(stream))
    if st != FLCE_OK:
        raise RuntimeError(f"flce_forward_noalloc: {lib().flce_status_string(st).decode()} "
                           f"({lib().flce_noalloc_last_error().decode()})")
    return loss, lse, valid_count, err_word


# The attention and head-norm calls below are made for single tokens too, where
# the host's time is the call's: their checks are kept to a few attribute reads.
def _current_stream(dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev)


def _with_stream(stream, call, *args, **kwargs):
    """``call`` with ``stream`` as the current one, so that the tensors it makes belong to
    the stream it runs on and their memory does not reach another stream's work too early."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        return call(*args, **kwargs)


def _cuda_device(q) -> int:
    dev = q.get_device()
    if dev < 0:
        raise ValueError(f"q must be a CUDA tensor, got one on {q.device}")
    _check_device("q", q)
    return dev


def _heads(name, t, dtype, dev):
    """(tokens, heads, head_dim, row stride, head stride) of a [tokens, heads, head_dim]
    tensor whose heads are contiguous."""
    if t.get_device() != dev or t.dtype is not dtype:
        raise TypeError(f"{name} must have the dtype and device of q ({dtype}, cuda:{dev}), "
                        f"got {t.dtype} on {t.device}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(t.shape)}")
    T, H, D = t.shape
    row, head, one = t.stride()
    if one != 1 and D > 1:
        raise ValueError(f"{name}: the head_dim values of a head must be contiguous")
    # the stride of a single token or head means nothing
    return T, H, D, (row if T > 1 else H * D), (head if H > 1 else D)


def _array(name, t, shape, dtype, dev):
    """Checks a contiguous operand or output of the given shape and type; its address."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on cuda:{dev}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _output(name, t, like, shape, dtype, dev):
    """The caller's output, checked, or a new contiguous one; its address."""
    if t is not None:
        return t, _array(name, t, shape, dtype, dev)
    t = torch.empty(shape, dtype=dtype, device=like.device)
    return t, t.data_ptr()


def _error_word(t, like, dev):
    """The caller's error word, checked, or a new one; its address."""
    if t is None:
        t = new_err_word(like.device)
    elif t.dtype is not torch.int32 or t.get_device() != dev or not t.numel():
        raise ValueError(f"err_word must be an int32 tensor on cuda:{dev}, got {t.numel()} {t.dtype} on {t.device}")
    return t, t.data_ptr()


def _scratch(t, need, like, dev):
    """The caller's workspace, checked, or a new one; its address and size."""
    if t is None:
        t = torch.empty(max(need, 256), dtype=torch.uint8, device=like.device)
    elif t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace_buf must be a contiguous tensor on cuda:{dev}, "
                         f"got {tuple(t.shape)} on {t.device}")
    return t, t.data_ptr(), t.numel()


def _qk_norm_rope_args(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved):
    """(desc, device, the inputs' addresses)."""
    dev, dtype = _cuda_device(q), q.dtype
    T, HQ, D, q_row, q_head = _heads("q", q, dtype, dev)
    Tk, HK, Dk, k_row, k_head = _heads("k", k, dtype, dev)
    if Tk != T or Dk != D:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}")
    wq = None if q_weight is None else _array("q_weight", q_weight, (D,), dtype, dev)
    wk = None if k_weight is None else _array("k_weight", k_weight, (D,), dtype, dev)
    rows = half = 0
    pc = ps = pp = None
    if cos is not None or sin is not None:
        if cos is None or sin is None or cos.dim() != 2:
            raise ValueError("cos and sin must both be [positions, rot_dim / 2] tensors, or None")
        rows, half = shape = cos.shape
        pc = _array("cos", cos, shape, torch.float32, dev)
        ps = _array("sin", sin, shape, torch.float32, dev)
    if positions is not None:
        pp = _array("positions", positions, (T,), torch.int64, dev)
    d = FlceQkNormRopeDesc(_QK_DESC_BYTES, T, HQ, HK, D, 2 * half, rows, _dtype_code(q, "q and k"),
                           eps, 1 if interleaved else 0, q_row, q_head, k_row, k_head)
    return d, dev, (q.data_ptr(), k.data_ptr(), wq, wk, pc, ps, pp)


def flce_qk_norm_rope_forward(q, k, q_weight, k_weight, cos, sin, positions=None,
                              eps: float = 1e-6, *, interleaved: bool = False, q_out=None,
                              k_out=None, err_word=None, stream=None):
    """RMS norm of each head of q [T, Hq, D] and k [T, Hk, D], weighted and turned
    to its position in one pass.  Returns (q_out, k_out, err_word), contiguous.

    cos, sin: float32 [positions, rot_dim / 2], or None for no rotation; the
    first rot_dim values of a head are turned, in pairs (j, j + rot_dim / 2), or
    (2j, 2j + 1) when interleaved.  positions: int64 [T] or None (0, 1, 2, ...)."""
    if stream is not None:
        return _with_stream(stream, flce_qk_norm_rope_forward, q, k, q_weight, k_weight, cos, sin,
                            positions, eps, interleaved=interleaved, q_out=q_out, k_out=k_out,
                            err_word=err_word)
    d, dev, ptrs = _qk_norm_rope_args(q, k, q_weight, k_weight, cos, sin, positions, eps,
                                      interleaved)
    dtype = q.dtype
    q_out, p_q = _output("q_out", q_out, q, q.shape, dtype, dev)
    k_out, p_k = _output("k_out", k_out, q, k.shape, dtype, dev)
    err_word, p_err = _error_word(err_word, q, dev)
    st = lib().flce_qk_norm_rope_forward(
        d, *ptrs, p_q, p_k, p_err, _current_stream(dev))
    if st:
        _check(st, "flce_qk_norm_rope_forward")
    return q_out, k_out, err_word


def flce_qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, cos, sin, positions=None,
                               eps: float = 1e-6, *, interleaved: bool = False, dq=None, dk=None,
                               dq_weight=None, dk_weight=None, workspace_buf=None, err_word=None,
                               stream=None):
    """Gradients of flce_qk_norm_rope_forward: (dq, dk in q's dtype, dq_weight,
    dk_weight float32 [D], err_word)."""
    if stream is not None:
        return _with_stream(stream, flce_qk_norm_rope_backward, dq_out, dk_out, q, k, q_weight,
                            k_weight, cos, sin, positions, eps, interleaved=interleaved, dq=dq,
                            dk=dk, dq_weight=dq_weight, dk_weight=dk_weight,
                            workspace_buf=workspace_buf, err_word=err_word)
    d, dev, ptrs = _qk_norm_rope_args(q, k, q_weight, k_weight, cos, sin, positions, eps,
                                      interleaved)
    dtype, f32, w_shape = q.dtype, torch.float32, (q.shape[2],)
    dq, p_dq = _output("dq", dq, q, q.shape, dtype, dev)
    dk, p_dk = _output("dk", dk, q, k.shape, dtype, dev)
    dq_weight, p_dwq = _output("dq_weight", dq_weight, q, w_shape, f32, dev)
    dk_weight, p_dwk = _output("dk_weight", dk_weight, q, w_shape, f32, dev)
    L = lib()
    need = L.flce_qk_norm_rope_workspace_size(d) if workspace_buf is None else 0
    ws, p_ws, ws_bytes = _scratch(workspace_buf, need, q, dev)
    err_word, p_err = _error_word(err_word, q, dev)
    st = L.flce_qk_norm_rope_backward(
        d, _array("dq_out", dq_out, q.shape, dtype, dev), _array("dk_out", dk_out, k.shape, dtype, dev),
        *ptrs, p_dq, p_dk, p_dwq, p_dwk, p_ws, ws_bytes, p_err,
        _current_stream(dev))
    if st:
        _check(st, "flce_qk_norm_rope_backward")
    return dq, dk, dq_weight, dk_weight, err_word


def _attention_args(q, k, v, cu_seqlens, scale):
    """(desc, device, lse's shape)."""
    dev, dtype = _cuda_device(q), q.dtype
    if dtype is not torch.bfloat16:
        raise TypeError(f"attention takes bfloat16 q, k and v, got {dtype}")
    T, HQ, D, q_row, q_head = _heads("q", q, dtype, dev)
    Tk, HK, Dk, k_row, k_head = _heads("k", k, dtype, dev)
    Tv, Hv, Dv, v_row, v_head = _heads("v", v, dtype, dev)
    if Tk != T or Dk != D or Tv != T or Hv != HK or Dv != D:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    n = cu_seqlens.numel()
    if (n < 1 or cu_seqlens.dim() != 1 or cu_seqlens.dtype is not torch.int32
            or cu_seqlens.get_device() != dev or not cu_seqlens.is_contiguous()):
        raise ValueError("cu_seqlens must be a contiguous int32 tensor of the sequences' offsets, "
                         f"one more than sequences, on cuda:{dev}")
    return FlceAttentionDesc(_ATTENTION_DESC_BYTES, T, n - 1, HQ, HK, D, FLCE_BF16,
                             D ** -0.5 if scale is None else scale, q_row, q_head, k_row, k_head,
                             v_row, v_head), dev, (HQ, T)


def flce_attention_forward(q, k, v, cu_seqlens, scale: Optional[float] = None, *, out=None,
                           lse=None, err_word=None, stream=None):
    """Causal attention within each packed sequence: q [T, Hq, D], k and v
    [T, Hk, D] bf16 (views are fine), cu_seqlens int32 offsets.  Returns
    (out [T, Hq, D] bf16, lse [Hq, T] float32, err_word); scale defaults to
    D ** -0.5.  Rows outside the sequences get out 0 and lse -inf."""
    if stream is not None:
        return _with_stream(stream, flce_attention_forward, q, k, v, cu_seqlens, scale, out=out,
                            lse=lse, err_word=err_word)
    d, dev, lse_shape = _attention_args(q, k, v, cu_seqlens, scale)
    out, p_out = _output("out", out, q, q.shape, q.dtype, dev)
    lse, p_lse = _output("lse", lse, q, lse_shape, torch.float32, dev)
    err_word, p_err = _error_word(err_word, q, dev)
    st = lib().flce_attention_forward(
        d, q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), p_out, p_lse,
        p_err, _current_stream(dev))
    if st:
        _check(st, "flce_attention_forward")
    return out, lse, err_word


def flce_attention_backward(dout, q, k, v, out, lse, cu_seqlens, scale: Optional[float] = None, *,
                            dq=None, dk=None, dv=None, workspace_buf=None, err_word=None,
                            stream=None):
    """Gradients (dq, dk, dv, err_word) of flce_attention_forward, contiguous bf16;
    those of a key / value head are summed over the query heads that read it."""
    if stream is not None:
        return _with_stream(stream, flce_attention_backward, dout, q, k, v, out, lse, cu_seqlens,
                            scale, dq=dq, dk=dk, dv=dv, workspace_buf=workspace_buf,
                            err_word=err_word)
    d, dev, lse_shape = _attention_args(q, k, v, cu_seqlens, scale)
    dtype, shape, kv_shape = q.dtype, q.shape, k.shape
    dq, p_dq = _output("dq", dq, q, shape, dtype, dev)
    dk, p_dk = _output("dk", dk, q, kv_shape, dtype, dev)
    dv, p_dv = _output("dv", dv, q, kv_shape, dtype, dev)
    L = lib()
    need = L.flce_attention_workspace_size(d) if workspace_buf is None else 0
    ws, p_ws, ws_bytes = _scratch(workspace_buf, need, q, dev)
    err_word, p_err = _error_word(err_word, q, dev)
    st = L.flce_attention_backward(
        d, _array("dout", dout, shape, dtype, dev), q.data_ptr(), k.data_ptr(), v.data_ptr(),
        _array("out", out, shape, dtype, dev), _array("lse", lse, lse_shape, torch.float32, dev),
        cu_seqlens.data_ptr(), p_dq, p_dk, p_dv, p_ws, ws_bytes, p_err,
        _current_stream(dev))
    if st:
        _check(st, "flce_attention_backward")
    return dq, dk, dv, err_word


def _cuda_rows(name, x) -> int:
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor, got one on {x.device}")
    _check_device(name, x)
    return dev


def _rows(name, t, shape, dtype, dev):
    """The row stride of a [rows, cols] tensor whose rows are contiguous."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} tensor {tuple(shape)} on cuda:{dev}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    if t.stride(1) != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the values of a row must be contiguous")
    return t.stride(0) if shape[0] > 1 else shape[1]


def _layer_norm_args(x, weight, eps, rms):
    """(desc, device, shape, dtype, the weight's address)."""
    dev, dtype = _cuda_rows("x", x), x.dtype
    if x.dim() != 2:
        raise ValueError(f"x must be [rows, cols], got {tuple(x.shape)}")
    shape = x.shape
    row = _rows("x", x, shape, dtype, dev)
    w = None if weight is None else _array("weight", weight, (shape[1],), dtype, dev)
    d = FlceLayerNormDesc(_LAYER_NORM_DESC_BYTES, shape[0], shape[1], _dtype_code(x, "x"), eps,
                          1 if rms else 0, row, shape[1])
    return d, dev, shape, dtype, w


def flce_layer_norm_forward(x, weight, bias=None, eps: float = 1e-5, *, residual=None,
                            rms: bool = False, out=None, sum_out=None, mean=None, rstd=None,
                            stream=None):
    """Layer norm (or RMS norm) of the rows of x [rows, cols], or of x + residual.
    Returns (y, sum, mean, rstd): sum is x + residual as it was normed, or x itself
    without a residual; mean is None for rms.  The backward takes the last three."""
    if stream is not None:
        return _with_stream(stream, flce_layer_norm_forward, x, weight, bias, eps,
                            residual=residual, rms=rms, out=out, sum_out=sum_out, mean=mean,
                            rstd=rstd)
    d, dev, shape, dtype, w = _layer_norm_args(x, weight, eps, rms)
    b = None if bias is None else _array("bias", bias, (shape[1],), dtype, dev)
    p_res = p_sum = p_mean = None
    if residual is not None:
        d.residual_row = _rows("residual", residual, shape, dtype, dev)
        p_res = residual.data_ptr()
        sum_out, p_sum = _output("sum_out", sum_out, x, shape, dtype, dev)
    f32, rows = torch.float32, shape[:1]
    out, p_out = _output("out", out, x, shape, dtype, dev)
    if not rms:
        mean, p_mean = _output("mean", mean, x, rows, f32, dev)
    rstd, p_rstd = _output("rstd", rstd, x, rows, f32, dev)
    st = lib().flce_layer_norm_forward(d, x.data_ptr(), p_res, w, b, p_out, p_sum, p_mean, p_rstd,
                                       _current_stream(dev))
    if st:
        _check(st, "flce_layer_norm_forward")
    return out, x if residual is None else sum_out, None if rms else mean, rstd


def flce_layer_norm_backward(dy, x, weight, mean, rstd, *, dsum=None, rms: bool = False,
                             bias: bool = True, dx=None, dweight=None, dbias=None,
                             workspace_buf=None, stream=None):
    """Gradients of flce_layer_norm_forward, whose sum is x here: (dx in x's dtype, of the
    sum and so of x and residual alike; dweight, dbias float32 [cols]).  dsum, the gradient
    that reached the stored sum itself, is added to dx.  dbias is None if not bias."""
    if stream is not None:
        return _with_stream(stream, flce_layer_norm_backward, dy, x, weight, mean, rstd, dsum=dsum,
                            rms=rms, bias=bias, dx=dx, dweight=dweight, dbias=dbias,
                            workspace_buf=workspace_buf)
    d, dev, shape, dtype, w = _layer_norm_args(x, weight, 0.0, rms)
    f32, rows, cols = torch.float32, shape[:1], shape[1:]
    p_db = None
    dx, p_dx = _output("dx", dx, x, shape, dtype, dev)
    dweight, p_dw = _output("dweight", dweight, x, cols, f32, dev)
    if bias:
        dbias, p_db = _output("dbias", dbias, x, cols, f32, dev)
    L = lib()
    need = L.flce_layer_norm_workspace_size(d) if workspace_buf is None else 0
    ws, p_ws, ws_bytes = _scratch(workspace_buf, need, x, dev)
    st = L.flce_layer_norm_backward(
        d, _array("dy", dy, shape, dtype, dev), x.data_ptr(), w,
        None if rms else _array("mean", mean, rows, f32, dev), _array("rstd", rstd, rows, f32, dev),
        None if dsum is None else _array("dsum", dsum, shape, dtype, dev), p_dx, p_dw, p_db, p_ws,
        ws_bytes, _current_stream(dev))
    if st:
        _check(st, "flce_layer_norm_backward")
    return dx, dweight, dbias if bias else None


def rope_frequencies(rot_dim: int, theta: float = 10000.0, scaling: str = "none", *,
                     factor: float = 1.0, trained_length: int = 8192, low: float = 1.0,
                     high: Optional[float] = None, device="cuda"):
    """(inv_freq float64 [rot_dim / 2], magnitude) for ``rope``: theta^(-2j / rot_dim), for
    contexts of factor times the trained length changed by ``scaling``:

      "linear"  every frequency divided by factor
      "ntk"     theta grown so that the lowest frequency is divided by factor
      "llama3"  frequencies with fewer than ``low`` turns in the trained length divided by
                factor, those with more than ``high`` (4) kept, linear in turns between
      "yarn"    the same, with ``high`` 32 and linear in the index between, and magnitude
                1 + 0.1 ln(factor)"""
    if rot_dim <= 0 or rot_dim % 2 or not theta > 1.0 or not factor >= 1.0:
        raise ValueError(f"rot_dim must be even, theta above 1 and factor at least 1: got {rot_dim}, {theta}, {factor}")
    half, magnitude = rot_dim // 2, 1.0
    if scaling == "ntk" and half > 1:
        theta *= factor ** (half / (half - 1.0))
    j = torch.arange(half, dtype=torch.float64)
    inv = theta ** (-j / half)
    if scaling == "linear":
        inv = inv / factor
    elif scaling in ("llama3", "yarn"):
        high = (4.0 if scaling == "llama3" else 32.0) if high is None else high
        if not 0.0 < low < high:
            raise ValueError(f"0 < low < high is needed, got {low}, {high}")
        if scaling == "llama3":
            kept = (trained_length * inv / (2.0 * math.pi) - low) / (high - low)
        else:
            def index_of(turns):
                return half * math.log(trained_length / (2.0 * math.pi * turns)) / math.log(theta)

            first = max(math.floor(index_of(high)), 0)
            last = min(math.ceil(index_of(low)), rot_dim - 1)
            kept = 1.0 - (j - first) / max(last - first, 1e-3)
            magnitude = 1.0 + 0.1 * math.log(factor)
        kept = kept.clamp(0.0, 1.0)
        inv = inv * kept + inv / factor * (1.0 - kept)
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"scaling must be none, linear, ntk, llama3 or yarn, got {scaling!r}")
    return inv.to(device), magnitude


def _rope(name, backward, q, k, inv_freq, positions, magnitude, interleaved, q_out, k_out):
    dev, dtype = _cuda_device(q), q.dtype
    T, HQ, D, q_row, q_head = _heads("q", q, dtype, dev)
    Tk, HK, Dk, k_row, k_head = _heads("k", k, dtype, dev)
    if Tk != T or Dk != D:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}")
    p_f = _array("inv_freq", inv_freq, inv_freq.shape[:1], torch.float64, dev)
    p_p = None if positions is None else _array("positions", positions, (T,), torch.int64, dev)
    d = FlceRopeDesc(_ROPE_DESC_BYTES, T, HQ, HK, D, 2 * inv_freq.numel(), _dtype_code(q, "q and k"), magnitude,
                     1 if interleaved else 0, q_row, q_head, k_row, k_head)
    q_out, p_q = _output("q_out", q_out, q, q.shape, dtype, dev)
    k_out, p_k = _output("k_out", k_out, q, k.shape, dtype, dev)
    L = lib()
    st = (L.flce_rope_backward if backward else L.flce_rope_forward)(
        d, q.data_ptr(), k.data_ptr(), p_f, p_p, p_q, p_k, _current_stream(dev))
    if st:
        _check(st, name)
    return q_out, k_out


def flce_rope_forward(q, k, inv_freq, positions=None, *, magnitude: float = 1.0,
                      interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """Rotary positions of q [T, Hq, D] and k [T, Hk, D] (views are fine): the first
    2 * len(inv_freq) values of each head turned by positions * inv_freq and multiplied by
    magnitude, in pairs (j, j + rot_dim / 2), or (2j, 2j + 1) when interleaved.  Returns
    (q_out, k_out), contiguous.  inv_freq: float64, a multiple of 4 of them, any (see
    rope_frequencies); positions: int64 [T] or None (0, 1, 2, ...), any."""
    if stream is not None:
        return _with_stream(stream, flce_rope_forward, q, k, inv_freq, positions, magnitude=magnitude,
                            interleaved=interleaved, q_out=q_out, k_out=k_out)
    return _rope("flce_rope_forward", False, q, k, inv_freq, positions, magnitude, interleaved, q_out, k_out)


def flce_rope_backward(dq_out, dk_out, inv_freq, positions=None, *, magnitude: float = 1.0,
                       interleaved: bool = False, dq=None, dk=None, stream=None):
    """Gradients (dq, dk) of flce_rope_forward: the heads turned back."""
    if stream is not None:
        return _with_stream(stream, flce_rope_backward, dq_out, dk_out, inv_freq, positions,
                            magnitude=magnitude, interleaved=interleaved, dq=dq, dk=dk)
    return _rope("flce_rope_backward", True, dq_out, dk_out, inv_freq, positions, magnitude, interleaved, dq, dk)


def _distill_args(X, W, ids, teacher_logits, temperature, reduction, teacher_lse, dw_dtype):
    """(desc, device, the teacher's addresses)."""
    dev = _cuda_rows("X", X)
    if X.dtype is not torch.bfloat16:
        raise TypeError(f"distillation takes bfloat16 X and W, got {X.dtype}")
    if X.dim() != 2 or W.dim() != 2 or X.shape[1] != W.shape[1] or ids.dim() != 2 or ids.shape[0] != X.shape[0]:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}, ids {tuple(ids.shape)}")
    (N, H), V = X.shape, W.shape[0]
    _array("X", X, X.shape, torch.bfloat16, dev)
    _array("W", W, W.shape, torch.bfloat16, dev)
    p_ids = _array("ids", ids, ids.shape, torch.int64, dev)
    t_code = _dtype_code(teacher_logits, "the teacher's logits")
    p_t = _array("teacher_logits", teacher_logits, ids.shape, teacher_logits.dtype, dev)
    p_tl = None if teacher_lse is None else _array("teacher_lse", teacher_lse, (N,), torch.float32, dev)
    d = FlceDistillDesc(_DISTILL_DESC_BYTES, N, H, V, ids.shape[1], FLCE_BF16, t_code,
                        FLCE_FP32 if dw_dtype is torch.float32 else FLCE_BF16, temperature, _red_code(reduction))
    return d, dev, (p_ids, p_t, p_tl)


def flce_distill_workspace_size(N: int, H: int, V: int, K: int, mode: int = MODE_FWD_BWD) -> int:
    """Workspace bytes of a distillation of N tokens with K entries each."""
    return int(lib().flce_distill_workspace_size(
        FlceDistillDesc(_DISTILL_DESC_BYTES, N, H, V, K, FLCE_BF16, FLCE_FP32, FLCE_BF16, 1.0, FLCE_MEAN), mode))


def flce_distill_forward(X, W, ids, teacher_logits, temperature: float = 1.0, reduction: str = "mean", *,
                         teacher_lse=None, loss=None, lse=None, logits=None, valid_count=None, row_loss=None,
                         workspace_buf=None, err_word=None, stream=None):
    """Divergence of the student's softmax (X [N, H] W [V, H]^T / temperature, bf16, logits never
    stored) from the teacher's top logits: ids int64 [N, K], negative for no entry, and
    teacher_logits [N, K] bf16 or float32.  Without teacher_lse (float32 [N], the teacher's
    log-sum-exp over its whole vocabulary at the same temperature) the entries' probabilities
    are normed to one.  Returns (loss[1], lse[N], logits[N, K] of the student at the ids,
    valid_count[1], err_word); the backward takes the middle three."""
    if stream is not None:
        return _with_stream(stream, flce_distill_forward, X, W, ids, teacher_logits, temperature, reduction,
                            teacher_lse=teacher_lse, loss=loss, lse=lse, logits=logits, valid_count=valid_count,
                            row_loss=row_loss, workspace_buf=workspace_buf, err_word=err_word)
    d, dev, teacher = _distill_args(X, W, ids, teacher_logits, temperature, reduction, teacher_lse, torch.bfloat16)
    f32, N = torch.float32, X.shape[0]
    loss, p_loss = _output("loss", loss, X, (1,), f32, dev)
    lse, p_lse = _output("lse", lse, X, (N,), f32, dev)
    logits, p_logits = _output("logits", logits, X, ids.shape, f32, dev)
    valid_count, p_valid = _output("valid_count", valid_count, X, (1,), torch.int32, dev)
    p_rows = None if row_loss is None else _array("row_loss", row_loss, (N,), f32, dev)
    L = lib()
    need = L.flce_distill_workspace_size(d, MODE_FWD) if workspace_buf is None else 0
    ws, p_ws, ws_bytes = _scratch(workspace_buf, need, X, dev)
    err_word, p_err = _error_word(err_word, X, dev)
    st = L.flce_distill_forward(d, X.data_ptr(), W.data_ptr(), *teacher, p_loss, p_rows, p_lse, p_logits, p_valid,
                                p_ws, ws_bytes, p_err, _current_stream(dev))
    if st:
        _check(st, "flce_distill_forward")
    return loss, lse, logits, valid_count, err_word


def flce_distill_backward(X, W, ids, teacher_logits, lse, logits, valid_count, temperature: float = 1.0,
                          reduction: str = "mean", *, teacher_lse=None, grad_loss=None, dX=None, dW=None,
                          accumulate_dW: bool = False, need_dX: bool = True, need_dW: bool = True,
                          workspace_buf=None, err_word=None, stream=None):
    """Gradients (dX [N, H] bf16, dW [V, H], err_word) of flce_distill_forward.  dW is bf16, or
    the caller's float32 tensor, which alone can be accumulated into.  A gradient that is not
    needed is not computed, and None."""
    if stream is not None:
        return _with_stream(stream, flce_distill_backward, X, W, ids, teacher_logits, lse, logits, valid_count,
                            temperature, reduction, teacher_lse=teacher_lse, grad_loss=grad_loss, dX=dX, dW=dW,
                            accumulate_dW=accumulate_dW, need_dX=need_dX, need_dW=need_dW,
                            workspace_buf=workspace_buf, err_word=err_word)
    f32 = torch.float32
    dw_dtype = f32 if dW is not None and dW.dtype is f32 else torch.bfloat16
    d, dev, teacher = _distill_args(X, W, ids, teacher_logits, temperature, reduction, teacher_lse, dw_dtype)
    if accumulate_dW and (dW is None or dw_dtype is not f32):
        raise ValueError("accumulate_dW needs an existing float32 dW")
    dX, p_dx = _output("dX", dX, X, X.shape, torch.bfloat16, dev) if need_dX else (None, None)
    dW, p_dw = _output("dW", dW, X, W.shape, dw_dtype, dev) if need_dW else (None, None)
    p_grad = None if grad_loss is None else _array("grad_loss", grad_loss, (1,), f32, dev)
    L = lib()
    need = L.flce_distill_workspace_size(d, MODE_BWD) if workspace_buf is None else 0
    ws, p_ws, ws_bytes = _scratch(workspace_buf, need, X, dev)
    err_word, p_err = _error_word(err_word, X, dev)
    st = L.flce_distill_backward(
        d, X.data_ptr(), W.data_ptr(), *teacher, _array("lse", lse, X.shape[:1], f32, dev),
        _array("logits", logits, ids.shape, f32, dev), _array("valid_count", valid_count, (1,), torch.int32, dev),
        p_grad, p_dx, p_dw, int(bool(accumulate_dW)), p_ws, ws_bytes, p_err, _current_stream(dev))
    if st:
        _check(st, "flce_distill_backward")
    return dX, dW, err_word


def last_launch_count() -> int:
    return int(lib().flce_last_launch_count())


def last_multicast_launches() -> int:
    """Test-only: launches of the last call made with the operand-multicast walk."""
    return int(lib().flce_debug_last_multicast_launches())


def flce_profile_enable(on: bool) -> None:
    _check(lib().flce_profile_enable(int(bool(on))), "flce_profile_enable")


def flce_profile_reset() -> None:
    lib().flce_profile_reset()


def flce_profile_read() -> dict:
    """{kind: (total_ms, launches)} accumulated since the last reset."""
    out = {}
    for k, name in enumerate(PROFILE_KINDS):
        ms, n = ctypes.c_double(0.0), ctypes.c_int(0)
        _check(lib().flce_profile_read(k, ctypes.byref(ms), ctypes.byref(n)), "flce_profile_read")
        out[name] = (ms.value, n.value)
    return out


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, labels, ignore_index, smoothing, reduction, z_loss):
        loss, lse, nv, err = flce_forward(X, W, labels, ignore_index, smoothing, reduction,
                                          z_loss=z_loss)
        ctx.save_for_backward(X, W, labels, lse, nv, err)
        ctx.cfg = (ignore_index, smoothing, reduction, z_loss)
        return loss[0]

    @staticmethod
    def backward(ctx, g):
        X, W, labels, lse, nv, err = ctx.saved_tensors
        ii, eps, red, zl = ctx.cfg
        g1 = g.reshape(1).to(torch.float32).contiguous()
        dX, dW, _ = flce_backward(X, W, labels, lse, nv, ii, eps, red, grad_loss=g1, err_word=err,
                                  z_loss=zl)
        return dX, dW.to(W.dtype), None, None, None, None, None


def linear_cross_entropy(h, W, labels, ignore_index: int = -100, smoothing: float = 0.0,
                         reduction: str = "mean", z_loss: float = 0.0):
    """Autograd entry with the pages' call shape: linear_cross_entropy(h, W, labels,
    ignore_index=-100).  h may be [..., H]; labels [...] of the same leading shape."""
    H = h.shape[-1]
    return _LinearCrossEntropy.apply(h.reshape(-1, H).contiguous(), W.contiguous(),
                                     labels.reshape(-1).contiguous(), ignore_index, smoothing,
                                     reduction, z_loss)


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, err):
        q_out, k_out, err = flce_qk_norm_rope_forward(q, k, q_weight, k_weight, cos, sin, positions,
                                                      eps, interleaved=interleaved, err_word=err)
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, positions)
        # not saved: the caller may read and clear it before the backward
        ctx.cfg = (eps, interleaved, err)
        return q_out, k_out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gq, gk):
        q, k, wq, wk, cos, sin, positions = ctx.saved_tensors
        eps, interleaved, err = ctx.cfg
        dq, dk, dwq, dwk, _ = flce_qk_norm_rope_backward(
            gq.contiguous(), gk.contiguous(), q, k, wq, wk, cos, sin, positions, eps,
            interleaved=interleaved, err_word=err)
        return (dq, dk, None if wq is None else dwq.to(wq.dtype),
                None if wk is None else dwk.to(wk.dtype), None, None, None, None, None, None)


def qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions=None, eps: float = 1e-6,
                 interleaved: bool = False, *, err_word=None):
    """Autograd entry of flce_qk_norm_rope_forward: (q_out, k_out).  The forward and the
    backward report into err_word; without one what goes wrong on the device is not seen."""
    return _QkNormRope.apply(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, err_word)


class _PackedAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, scale, err):
        out, lse, err = flce_attention_forward(q, k, v, cu_seqlens, scale, err_word=err)
        ctx.save_for_backward(q, k, v, out, lse, cu_seqlens)
        # err is not saved: the caller may read and clear it before the backward
        ctx.cfg = (scale, err)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        q, k, v, out, lse, cu_seqlens = ctx.saved_tensors
        scale, err = ctx.cfg
        dq, dk, dv, _ = flce_attention_backward(g.contiguous(), q, k, v, out, lse, cu_seqlens,
                                                scale, err_word=err)
        return dq, dk, dv, None, None, None


def packed_attention(q, k, v, cu_seqlens, scale: Optional[float] = None, *, err_word=None):
    """Autograd entry of flce_attention_forward: out [T, Hq, D].  The forward and the
    backward report into err_word; without one what goes wrong on the device is not seen."""
    return _PackedAttention.apply(q, k, v, cu_seqlens, scale, err_word)


def _aligned(t):
    """t contiguous from a 16-byte boundary on: itself, or a copy."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _dense_rows(t):
    """t, or a contiguous copy where its rows are not what the kernels read (a broadcast row,
    a stride or a start off their alignment)."""
    row, one = t.stride()
    return t if one == 1 and row >= t.shape[1] and row % 8 == 0 and t.data_ptr() % 16 == 0 else _aligned(t)


def _dense_heads(name, t):
    """The same of [tokens, heads, head_dim]."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(t.shape)}")
    row, head, one = t.stride()
    ok = one == 1 and head >= t.shape[2] and row > 0 and row % 8 == 0 and head % 8 == 0 and t.data_ptr() % 16 == 0
    return t if ok else _aligned(t)


class _LayerNorm(torch.autograd.Function):
    # Shapes are changed in here, not by views around it: x and the residual then get one
    # gradient tensor, which autograd copies where both are leaves; through views they would
    # come to share its memory unseen.
    @staticmethod
    def forward(ctx, x, residual, weight, bias, eps, rms):
        shape = x.shape
        rows = _dense_rows(x.reshape(-1, shape[-1]))
        r = None if residual is None else _dense_rows(residual.reshape(-1, shape[-1]))
        y, s, mean, rstd = flce_layer_norm_forward(rows, weight, bias, eps, residual=r, rms=rms)
        ctx.save_for_backward(s, weight, mean, rstd)
        ctx.cfg = (shape, residual is not None, None if bias is None else bias.dtype, rms)
        ctx.set_materialize_grads(False)
        return y.view(shape) if residual is None else (y.view(shape), s.view(shape))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, ds=None):
        s, weight, mean, rstd = ctx.saved_tensors
        shape, summed, bias_dtype, rms = ctx.cfg
        dx = dw = db = None
        if dy is None:  # only the sum was used
            dx = ds
        else:
            dx, dw, db = flce_layer_norm_backward(_aligned(dy).view(s.shape), s, weight, mean, rstd,
                                                  dsum=None if ds is None else _aligned(ds).view(s.shape), rms=rms,
                                                  bias=bias_dtype is not None)
            dx = dx.view(shape)
        return (dx, dx if summed else None, None if weight is None or dw is None else dw.to(weight.dtype),
                None if db is None else db.to(bias_dtype), None, None)


def layer_norm(x, weight, bias=None, eps: float = 1e-5, *, residual=None, rms: bool = False):
    """Autograd entry of flce_layer_norm_forward for x [..., cols]: y, or with a residual of x's
    shape (y, x + residual)."""
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual {tuple(residual.shape)} must have the shape of x {tuple(x.shape)}")
    return _LayerNorm.apply(x, residual, None if weight is None else _aligned(weight),
                            None if bias is None else _aligned(bias), eps, rms)


class _Rope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, inv_freq, positions, magnitude, interleaved):
        ctx.save_for_backward(inv_freq, positions)
        ctx.cfg = {"magnitude": magnitude, "interleaved": interleaved}
        return flce_rope_forward(q, k, inv_freq, positions, **ctx.cfg)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gq, gk):
        inv_freq, positions = ctx.saved_tensors
        dq, dk = flce_rope_backward(_dense_heads("dq_out", gq), _dense_heads("dk_out", gk), inv_freq, positions,
                                    **ctx.cfg)
        return dq, dk, None, None, None, None


def rope(q, k, inv_freq, positions=None, *, magnitude: float = 1.0, interleaved: bool = False):
    """Autograd entry of flce_rope_forward: (q_out, k_out)."""
    return _Rope.apply(_dense_heads("q", q), _dense_heads("k", k), inv_freq, positions, magnitude, interleaved)


class _LinearDistillation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, ids, teacher_logits, temperature, reduction, teacher_lse, err):
        loss, lse, logits, valid, err = flce_distill_forward(X, W, ids, teacher_logits, temperature, reduction,
                                                             teacher_lse=teacher_lse, err_word=err)
        ctx.save_for_backward(X, W, ids, teacher_logits, teacher_lse, lse, logits, valid)
        # err is not saved: the caller may read and clear it before the backward
        ctx.cfg = (temperature, reduction, err)
        return loss[0]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        X, W, ids, teacher_logits, teacher_lse, lse, logits, valid = ctx.saved_tensors
        temperature, reduction, err = ctx.cfg
        dX, dW, _ = flce_distill_backward(X, W, ids, teacher_logits, lse, logits, valid, temperature, reduction,
                                          teacher_lse=teacher_lse,
                                          grad_loss=g.reshape(1).to(torch.float32).contiguous(), err_word=err,
                                          need_dX=ctx.needs_input_grad[0], need_dW=ctx.needs_input_grad[1])
        return dX, dW, None, None, None, None, None, None


def linear_distillation(h, W, ids, teacher_logits, temperature: float = 1.0, reduction: str = "mean", *,
                        teacher_lse=None, err_word=None):
    """Autograd entry of flce_distill_forward, in the shape of linear_cross_entropy: the loss.
    h may be [..., H]; ids and teacher_logits [..., K] and teacher_lse [...] of the same leading
    shape.  The teacher's side gets no gradient.  The forward and the backward report into
    err_word; without one what goes wrong on the device is not seen."""
    H, K = h.shape[-1], ids.shape[-1]
    return _LinearDistillation.apply(
        _aligned(h.reshape(-1, H)), _aligned(W), ids.reshape(-1, K).contiguous(),
        teacher_logits.detach().reshape(-1, K).contiguous(), temperature, reduction,
        None if teacher_lse is None else teacher_lse.detach().reshape(-1).contiguous(), err_word)
