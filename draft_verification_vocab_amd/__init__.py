"""Speculative verify-and-accept and the P-EAGLE draft batch on MI355X.

Thin Python binding over ``libspecverify.so`` (C ABI in include/spec_verify.h).
The functions here only marshal arguments: they check tensor shapes, dtypes
and devices, allocate outputs with torch when the caller passes none, and call
the library on the current HIP stream.  All computation runs in the library's
HIP kernels; there is no other implementation to fall back to, and every call
raises if the library is missing or returns an error.

One decode round, with the drafter's distributions handed over as its logits
and row descriptors (tensors on the GPU; shapes as in the C header)::

    tok, _, desc = spec_draft_sample(drafter_logits, K, T, uniforms=u_draft,
                                     row_index=sample_rows, want_draft_probs=False,
                                     want_row_desc=True)
    out, acc, _ = spec_verify_sample_lq(target_logits, drafter_logits, desc, tok,
                                        u_verify, T, drafter_rows=sample_rows)
    batch = peagle_build_draft_batch(out, acc, tok, start_pos, block_table,
                                     block_size, target_hidden, h_shared, mask_id)

spec_draft_sample_filtered and spec_verify_filtered(_lq) are the forms for
requests with top-k, top-p and min-p, and peagle_append_kv writes the rebuilt
batch's keys and values into the paged cache.  spec_verify_greedy /
spec_verify_sample / spec_verify_mixed take a dense q instead; spec_verify_tree verifies draft trees; StepGraph captures a verify,
build and acceptance-metrics step as one HIP graph.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

__all__ = [
    "require_library", "library_path", "sv_status_string", "spec_verify_workspace_bytes",
    "spec_verify_greedy", "spec_verify_sample", "peagle_build_draft_batch",
    "SpecVerifyError", "SV_F32", "SV_BF16", "SV_F16", "PADDING_SLOT_ID",
    "spec_verify_mixed", "spec_verify_sample_lq", "spec_verify_mixed_lq",
    "spec_verify_sample_noalloc", "spec_verify_greedy_early_exit",
    "spec_verify_sample_early_exit", "spec_verify_mixed_early_exit",
    "spec_verify_sample_lq_early_exit", "spec_verify_mixed_lq_early_exit",
    "spec_verify_tree_early_exit", "spec_verify_tree_lq_early_exit", "spec_verify_tree_mixed",
    "spec_verify_tree_mixed_early_exit",
    "noalloc_scratch_bytes", "spec_verify_tree", "spec_verify_tree_lq", "spec_draft_sample",
    "spec_accept_metrics", "accept_metrics_buffer", "acceptance_summary", "StepGraph",
    "trace_begin", "trace_read", "trace_end",
    "spec_draft_sample_filtered", "spec_verify_filtered", "spec_verify_filtered_lq",
    "spec_filter_workspace_bytes", "peagle_append_kv",
    "DEVERR_DRAFT_TOKEN", "DEVERR_ACCEPT_COUNT", "DEVERR_BLOCK_TABLE",
]

SV_F32, SV_BF16, SV_F16, SV_E4M3 = 0, 1, 2, 3
PADDING_SLOT_ID = -1
DEVERR_DRAFT_TOKEN, DEVERR_ACCEPT_COUNT, DEVERR_BLOCK_TABLE = 1, 2, 4
DEVERR_ROW_INDEX, DEVERR_TEMPERATURE, DEVERR_TREE = 8, 16, 32
DEVERR_FILTER, DEVERR_EMPTY_ROW, DEVERR_SLOT = 64, 128, 256
MAX_B, MAX_K, MAX_V = 1 << 20, 63, 1 << 19      # SV_MAX_B, SV_MAX_K, SV_MAX_V

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libspecverify.so")
_lib = None
_lock = threading.Lock()

_p = ctypes.c_void_p
_i = ctypes.c_int
_SIGS = {
    "sv_status_string": (ctypes.c_char_p, [_i]),
    "spec_verify_workspace_bytes": (ctypes.c_size_t, [_i, _i, _i]),
    "spec_verify_greedy": (_i, [_p, _i, _p, _i, _i, _i, _p, _p, _p, ctypes.c_size_t, _p, _p]),
    "spec_verify_sample": (_i, [_p, _i, _p, _p, _p, ctypes.c_float, _i, _i, _i, _p, _p, _p, _p,
                                ctypes.c_size_t, _p, _p]),
    "peagle_build_draft_batch": (_i, [_p, _p, _p, _p, _p, _i, _i, _p, _p, _i, ctypes.c_int32,
                                      _i, _i, _i, _p, _p, _p, _p, _p, _p, _p]),
    "spec_verify_noalloc_scratch_bytes": (ctypes.c_size_t, []),
    "spec_verify_sample_noalloc": (_i, [_p, _i, _p, _p, _p, ctypes.c_float, _i, _i, _i, _p, _p,
                                        _p, _p, _p]),
    "spec_verify_mixed": (_i, [_p, _i, _p, _p, _p, _p, _i, _i, _i, _p, _p, _p, _p,
                               ctypes.c_size_t, _p, _p]),
    "spec_verify_greedy_early_exit": (_i, [_p, _i, _p, _i, _i, _i, _p, _p, _p, ctypes.c_size_t,
                                           _p, _p]),
    "spec_verify_sample_early_exit": (_i, [_p, _i, _p, _p, _p, ctypes.c_float, _i, _i, _i, _p,
                                           _p, _p, _p, ctypes.c_size_t, _p, _p]),
    "spec_verify_mixed_early_exit": (_i, [_p, _i, _p, _p, _p, _p, _i, _i, _i, _p, _p, _p, _p,
                                          ctypes.c_size_t, _p, _p]),
    "spec_draft_sample": (_i, [_p, _i, ctypes.c_int64, _p, _p, ctypes.c_float, _p, _i, _i, _i,
                               _p, _p, _p, _p, _p]),
    "spec_verify_sample_lq": (_i, [_p, _i, _p, ctypes.c_int64, _p, _p, _p, _p, ctypes.c_float,
                                   _i, _i, _i, _p, _p, _p, _p, ctypes.c_size_t, _p, _p]),
    "spec_verify_mixed_lq": (_i, [_p, _i, _p, ctypes.c_int64, _p, _p, _p, _p, _p,
                                  _i, _i, _i, _p, _p, _p, _p, ctypes.c_size_t, _p, _p]),
    "spec_verify_sample_lq_early_exit": (_i, [_p, _i, _p, ctypes.c_int64, _p, _p, _p, _p,
                                              ctypes.c_float, _i, _i, _i, _p, _p, _p, _p,
                                              ctypes.c_size_t, _p, _p]),
    "spec_verify_mixed_lq_early_exit": (_i, [_p, _i, _p, ctypes.c_int64, _p, _p, _p, _p, _p,
                                             _i, _i, _i, _p, _p, _p, _p, ctypes.c_size_t, _p,
                                             _p]),
    "spec_verify_tree": (_i, [_p, _i, _p, _p, _p, _p, ctypes.c_float, _i, _i, _i, _p, _p, _p, _p,
                              ctypes.c_size_t, _p, _p]),
    "spec_verify_tree_lq": (_i, [_p, _i, _p, ctypes.c_int64, _p, _p, _p, _p, _p, ctypes.c_float,
                                 _i, _i, _i, _p, _p, _p, _p, ctypes.c_size_t, _p, _p]),
    "spec_verify_tree_early_exit": (_i, [_p, _i, _p, _p, _p, _p, ctypes.c_float, _i, _i, _i, _p,
                                         _p, _p, _p, ctypes.c_size_t, _p, _p]),
    "spec_verify_tree_lq_early_exit": (_i, [_p, _i, _p, ctypes.c_int64, _p, _p, _p, _p, _p,
                                            ctypes.c_float, _i, _i, _i, _p, _p, _p, _p,
                                            ctypes.c_size_t, _p, _p]),
    "spec_verify_tree_mixed": (_i, [_p, _i, _p, _p, _p, _p, _p, _i, _i, _i, _p, _p, _p, _p,
                                    ctypes.c_size_t, _p, _p]),
    "spec_verify_tree_mixed_early_exit": (_i, [_p, _i, _p, _p, _p, _p, _p, _i, _i, _i, _p, _p,
                                               _p, _p, ctypes.c_size_t, _p, _p]),
    "spec_filter_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, _i]),
    "spec_draft_sample_filtered": (_i, [_p, _i, ctypes.c_int64, ctypes.c_int64, _p, _p,
                                        ctypes.c_float, _p, _p, _p, _p, _i, _i, _i, _p, _p, _p, _p,
                                        ctypes.c_size_t, _p, _p]),
    "spec_verify_filtered": (_i, [_p, _i, ctypes.c_int64, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i,
                                  _p, _p, _p, _p, ctypes.c_size_t, _p, _p]),
    "spec_verify_filtered_lq": (_i, [_p, _i, ctypes.c_int64, _p, ctypes.c_int64, ctypes.c_int64,
                                     _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _p, _p, _p, _p,
                                     ctypes.c_size_t, _p, _p]),
    "peagle_append_kv": (_i, [_p, _p, _p, _i, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _p,
                              _p, _p, _i, _i, ctypes.c_float, ctypes.c_int64, _i, _i, _i, _p, _p,
                              _i, ctypes.c_int64, _i, ctypes.c_int64, ctypes.c_int64,
                              ctypes.c_int64, _p, _p, _p, ctypes.c_int64, _p, _p]),
    "spec_accept_metrics_words": (ctypes.c_size_t, [_i]),
    "spec_accept_metrics": (_i, [_p, _i, _i, _p, _p, _p]),
    "sv_step_graph_create": (_i, [_p, _p]),
    "sv_step_graph_launch": (_i, [_p, _p]),
    "sv_step_graph_destroy": (None, [_p]),
    "sv_kernel_name": (ctypes.c_char_p, [_i]),
    "sv_trace_begin": (_i, [_i, ctypes.c_uint]),
    "sv_trace_count": (_i, []),
    "sv_trace_read": (_i, [_i, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_float)]),
    "sv_trace_end": (None, []),
    "sv_trace_enable": (None, [_i]),
}


class SpecVerifyError(RuntimeError):
    pass


def library_path() -> str:
    return _LIB_PATH


def require_library():
    """Load libspecverify.so (raises if it has not been built)."""
    global _lib
    lib = _lib
    if lib is not None:
        return lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise SpecVerifyError(
                    f"{_LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
            lib = ctypes.CDLL(_LIB_PATH)
            for name, (res, args) in _SIGS.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def sv_status_string(status: int) -> str:
    return require_library().sv_status_string(status).decode()


_ws_bytes = {}


def spec_verify_workspace_bytes(B: int, K: int, V: int) -> int:
    key = (B, K, V)
    n = _ws_bytes.get(key)
    if n is None:
        n = _ws_bytes[key] = int(require_library().spec_verify_workspace_bytes(B, K, V))
    return n


def _check(status: int, what: str):
    if status != 0:
        raise SpecVerifyError(f"{what}: {sv_status_string(status)} (status {status})")


# ---------------------------------------------------------------- tracing
KERNEL_IDS = {"verify_greedy_rows": 0, "verify_sample_rows": 1, "verify_sample_draw": 2,
              "peagle_build": 3, "verify_greedy_accept": 4, "verify_sample_locate": 5,
              "draft_sample": 6, "verify_mixed_rows": 7, "accept_metrics": 8, "tree_rows": 9,
              "tree_walk": 10, "filter_rows": 12, "filtered_verify": 13, "append_kv": 14}


def trace_begin(capacity: int, kernels=None):
    """Start kernel tracing on this host thread for up to `capacity` launches
    of the named kernels (all kernels when `kernels` is None)."""
    mask = 0xFFFFFFFF if kernels is None else sum(1 << KERNEL_IDS[k] for k in kernels)
    _check(require_library().sv_trace_begin(int(capacity), mask), "sv_trace_begin")


def trace_read():
    """[(kernel name, duration ms)] of the launches traced so far (waits for them)."""
    lib = require_library()
    out = []
    kid, ms = ctypes.c_int(), ctypes.c_float()
    for i in range(lib.sv_trace_count()):
        _check(lib.sv_trace_read(i, ctypes.byref(kid), ctypes.byref(ms)), "sv_trace_read")
        out.append((lib.sv_kernel_name(kid.value).decode(), float(ms.value)))
    return out


def trace_end():
    require_library().sv_trace_end()


def trace_enable(on: bool):
    """Pause (False) or resume (True) the active trace of this host thread."""
    require_library().sv_trace_enable(1 if on else 0)


# ---------------------------------------------------------------- helpers
_DTYPES = {torch.float32: SV_F32, torch.bfloat16: SV_BF16, torch.float16: SV_F16}


# The checks below run on every call, so they use the cheapest tensor
# queries (a small verify call spends more time here than on the GPU).
def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _dev(t: torch.Tensor, name: str, dtype=None, shape=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.get_device() != device.index:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device):
    """The current HIP stream of `device` (the library enqueues on it)."""
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


_ws_cache = {}


def _workspace(device, nbytes: int) -> torch.Tensor:
    """A zero-filled workspace per device.  The kernels leave it zero-filled,
    so it is reused without clearing; calls on one device must share a stream."""
    key = (device.type, device.index)
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    return ws


# ---------------------------------------------------------------- verify
def spec_verify_greedy(target_logits: torch.Tensor, draft_tokens: torch.Tensor,
                       out_tokens: Optional[torch.Tensor] = None,
                       out_num_accepted: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       device_error: Optional[torch.Tensor] = None,
                       _symbol: str = "spec_verify_greedy"):
    """Greedy verify; see spec_verify_greedy in include/spec_verify.h.

    target_logits [B, K+1, V] float32/bfloat16, draft_tokens [B, K] int32.
    Returns (out_tokens [B, K+1] int32, num_accepted [B] int32).
    """
    lib = require_library()
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, K+1, V]")
    B, K1, V = target_logits.shape
    K = K1 - 1
    dev = target_logits.device
    _dev(target_logits, "target_logits")
    if target_logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("target_logits must be float32 or bfloat16")
    _dev(draft_tokens, "draft_tokens", torch.int32, (B, K), dev)
    out_tokens = torch.empty((B, K + 1), dtype=torch.int32, device=dev) if out_tokens is None \
        else _dev(out_tokens, "out_tokens", torch.int32, (B, K + 1), dev)
    out_num_accepted = torch.empty(B, dtype=torch.int32, device=dev) if out_num_accepted is None \
        else _dev(out_num_accepted, "out_num_accepted", torch.int32, (B,), dev)
    need = spec_verify_workspace_bytes(B, K, V)
    if workspace is None:
        workspace = _workspace(dev, need)
    _dev(workspace, "workspace", device=dev)
    if device_error is not None:
        _dev(device_error, "device_error", torch.int32, (1,), dev)
    st = getattr(lib, _symbol)(_ptr(target_logits), _DTYPES[target_logits.dtype],
                               _ptr(draft_tokens), B, K, V, _ptr(out_tokens),
                               _ptr(out_num_accepted), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _ptr(device_error),
                               _stream(dev))
    _check(st, _symbol)
    return out_tokens, out_num_accepted


def spec_verify_sample(target_logits: torch.Tensor, draft_probs: torch.Tensor,
                       draft_tokens: torch.Tensor, uniforms: torch.Tensor, temperature: float,
                       out_tokens: Optional[torch.Tensor] = None,
                       out_num_accepted: Optional[torch.Tensor] = None,
                       out_draft_target_prob: Optional[torch.Tensor] = None,
                       want_draft_target_prob: bool = False,
                       workspace: Optional[torch.Tensor] = None,
                       device_error: Optional[torch.Tensor] = None,
                       _symbol: str = "spec_verify_sample"):
    """Rejection-sampling verify; see spec_verify_sample in include/spec_verify.h.

    Returns (out_tokens, num_accepted, draft_target_prob or None).
    """
    lib = require_library()
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, K+1, V]")
    B, K1, V = target_logits.shape
    K = K1 - 1
    dev = target_logits.device
    _dev(target_logits, "target_logits")
    if target_logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("target_logits must be float32 or bfloat16")
    _dev(draft_probs, "draft_probs", torch.float32, (B, K, V), dev)
    _dev(draft_tokens, "draft_tokens", torch.int32, (B, K), dev)
    _dev(uniforms, "uniforms", torch.float32, (B, K + 1), dev)
    out_tokens = torch.empty((B, K + 1), dtype=torch.int32, device=dev) if out_tokens is None \
        else _dev(out_tokens, "out_tokens", torch.int32, (B, K + 1), dev)
    out_num_accepted = torch.empty(B, dtype=torch.int32, device=dev) if out_num_accepted is None \
        else _dev(out_num_accepted, "out_num_accepted", torch.int32, (B,), dev)
    if out_draft_target_prob is None and want_draft_target_prob:
        out_draft_target_prob = torch.empty((B, K), dtype=torch.float32, device=dev)
    if out_draft_target_prob is not None:
        _dev(out_draft_target_prob, "out_draft_target_prob", torch.float32, (B, K), dev)
    need = spec_verify_workspace_bytes(B, K, V)
    if workspace is None:
        workspace = _workspace(dev, need)
    _dev(workspace, "workspace", device=dev)
    if device_error is not None:
        _dev(device_error, "device_error", torch.int32, (1,), dev)
    st = getattr(lib, _symbol)(_ptr(target_logits), _DTYPES[target_logits.dtype], _ptr(draft_probs),
                                _ptr(draft_tokens), _ptr(uniforms), float(temperature), B, K, V,
                                _ptr(out_tokens), _ptr(out_num_accepted), _ptr(out_draft_target_prob),
                                _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _ptr(device_error), _stream(dev))
    _check(st, _symbol)
    return out_tokens, out_num_accepted, out_draft_target_prob


def noalloc_scratch_bytes() -> int:
    """Size of the fixed scratch array spec_verify_sample_noalloc uses per GPU."""
    return int(require_library().spec_verify_noalloc_scratch_bytes())


def spec_verify_sample_noalloc(target_logits: torch.Tensor, draft_probs: torch.Tensor,
                               draft_tokens: torch.Tensor, uniforms: torch.Tensor,
                               temperature: float,
                               out_tokens: torch.Tensor, out_num_accepted: torch.Tensor,
                               out_draft_target_prob: Optional[torch.Tensor] = None,
                               device_error: Optional[torch.Tensor] = None):
    """spec_verify_sample without a workspace (see spec_verify_sample_noalloc in
    include/spec_verify.h): the library takes its scratch from a fixed device
    array, and the caller passes every output, so the call allocates nothing."""
    lib = require_library()
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, K+1, V]")
    B, K1, V = target_logits.shape
    K = K1 - 1
    dev = target_logits.device
    _dev(target_logits, "target_logits")
    if target_logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("target_logits must be float32 or bfloat16")
    _dev(draft_probs, "draft_probs", torch.float32, (B, K, V), dev)
    _dev(draft_tokens, "draft_tokens", torch.int32, (B, K), dev)
    _dev(uniforms, "uniforms", torch.float32, (B, K + 1), dev)
    _dev(out_tokens, "out_tokens", torch.int32, (B, K + 1), dev)
    _dev(out_num_accepted, "out_num_accepted", torch.int32, (B,), dev)
    if out_draft_target_prob is not None:
        _dev(out_draft_target_prob, "out_draft_target_prob", torch.float32, (B, K), dev)
    if device_error is not None:
        _dev(device_error, "device_error", torch.int32, (1,), dev)
    st = lib.spec_verify_sample_noalloc(
        _ptr(target_logits), _DTYPES[target_logits.dtype], _ptr(draft_probs), _ptr(draft_tokens),
        _ptr(uniforms), float(temperature), B, K, V, _ptr(out_tokens), _ptr(out_num_accepted),
        _ptr(out_draft_target_prob), _ptr(device_error), _stream(dev))
    _check(st, "spec_verify_sample_noalloc")
    return out_tokens, out_num_accepted, out_draft_target_prob


def spec_verify_mixed(target_logits: torch.Tensor, draft_probs: torch.Tensor,
                      draft_tokens: torch.Tensor, uniforms: torch.Tensor,
                      temperatures: torch.Tensor,
                      out_tokens: Optional[torch.Tensor] = None,
                      out_num_accepted: Optional[torch.Tensor] = None,
                      out_draft_target_prob: Optional[torch.Tensor] = None,
                      want_draft_target_prob: bool = False,
                      workspace: Optional[torch.Tensor] = None,
                      device_error: Optional[torch.Tensor] = None,
                      _symbol: str = "spec_verify_mixed"):
    """Verify with a temperature per sequence (0 = greedy); see
    spec_verify_mixed in include/spec_verify.h.

    Returns (out_tokens, num_accepted, draft_target_prob or None).
    """
    lib = require_library()
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, K+1, V]")
    B, K1, V = target_logits.shape
    K = K1 - 1
    dev = target_logits.device
    _dev(target_logits, "target_logits")
    if target_logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("target_logits must be float32 or bfloat16")
    _dev(draft_probs, "draft_probs", torch.float32, (B, K, V), dev)
    _dev(draft_tokens, "draft_tokens", torch.int32, (B, K), dev)
    _dev(uniforms, "uniforms", torch.float32, (B, K + 1), dev)
    _dev(temperatures, "temperatures", torch.float32, (B,), dev)
    out_tokens = torch.empty((B, K + 1), dtype=torch.int32, device=dev) if out_tokens is None \
        else _dev(out_tokens, "out_tokens", torch.int32, (B, K + 1), dev)
    out_num_accepted = torch.empty(B, dtype=torch.int32, device=dev) if out_num_accepted is None \
        else _dev(out_num_accepted, "out_num_accepted", torch.int32, (B,), dev)
    if out_draft_target_prob is None and want_draft_target_prob:
        out_draft_target_prob = torch.empty((B, K), dtype=torch.float32, device=dev)
    if out_draft_target_prob is not None:
        _dev(out_draft_target_prob, "out_draft_target_prob", torch.float32, (B, K), dev)
    need = spec_verify_workspace_bytes(B, K, V)
    if workspace is None:
        workspace = _workspace(dev, need)
    _dev(workspace, "workspace", device=dev)
    if device_error is not None:
        _dev(device_error, "device_error", torch.int32, (1,), dev)
    st = getattr(lib, _symbol)(_ptr(target_logits), _DTYPES[target_logits.dtype],
                               _ptr(draft_probs), _ptr(draft_tokens), _ptr(uniforms),
                               _ptr(temperatures), B, K, V, _ptr(out_tokens),
                               _ptr(out_num_accepted), _ptr(out_draft_target_prob),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _ptr(device_error), _stream(dev))
    _check(st, _symbol)
    return out_tokens, out_num_accepted, out_draft_target_prob


def spec_verify_greedy_early_exit(*args, **kw):
    """spec_verify_greedy computing only the rows up to each sequence's first
    rejection; see spec_verify_greedy_early_exit in include/spec_verify.h.
    Arguments and results as spec_verify_greedy."""
    return spec_verify_greedy(*args, _symbol="spec_verify_greedy_early_exit", **kw)


def spec_verify_sample_early_exit(*args, **kw):
    """spec_verify_sample computing only the rows up to each sequence's first
    rejection; see spec_verify_sample_early_exit in include/spec_verify.h.
    Arguments as spec_verify_sample; draft_target_prob is 0 past num_accepted."""
    return spec_verify_sample(*args, _symbol="spec_verify_sample_early_exit", **kw)


def spec_verify_mixed_early_exit(*args, **kw):
    """spec_verify_mixed computing only the rows up to each sequence's first
    rejection; see spec_verify_mixed_early_exit in include/spec_verify.h.
    Arguments as spec_verify_mixed; draft_target_prob is 0 past num_accepted."""
    return spec_verify_mixed(*args, _symbol="spec_verify_mixed_early_exit", **kw)


# ---------------------------------------------------------------- P-EAGLE
def peagle_build_draft_batch(verify_out_tokens: torch.Tensor, num_accepted: torch.Tensor,
                             draft_tokens: torch.Tensor, start_pos: torch.Tensor,
                             block_table: torch.Tensor, block_size: int,
                             target_hidden: torch.Tensor, h_shared: torch.Tensor,
                             mask_token_id: int, outputs: Optional[dict] = None,
                             want_sample_rows: bool = True,
                             device_error: Optional[torch.Tensor] = None) -> dict:
    """P-EAGLE drafter batch; see peagle_build_draft_batch in include/spec_verify.h.

    Returns a dict of input_ids [B*2K] int32, positions [B*2K] int64,
    slot_mapping [B*2K] int64, hidden [B*2K, H], sample_rows [B, K] int32.
    """
    lib = require_library()
    B, K = draft_tokens.shape
    dev = draft_tokens.device
    H = target_hidden.shape[-1]
    _dev(draft_tokens, "draft_tokens", torch.int32, (B, K), dev)
    _dev(verify_out_tokens, "verify_out_tokens", torch.int32, (B, K + 1), dev)
    _dev(num_accepted, "num_accepted", torch.int32, (B,), dev)
    _dev(start_pos, "start_pos", torch.int64, (B,), dev)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_blocks_per_seq]")
    _dev(block_table, "block_table", torch.int32, device=dev)
    if target_hidden.dtype not in _DTYPES:
        raise TypeError("hidden states must be bfloat16, float16 or float32")
    _dev(target_hidden, "target_hidden", shape=(B * (K + 1), H), device=dev)
    _dev(h_shared, "h_shared", target_hidden.dtype, (H,), dev)
    o = dict(outputs or {})
    n = B * 2 * K
    if "input_ids" not in o:
        o["input_ids"] = torch.empty(n, dtype=torch.int32, device=dev)
    if "positions" not in o:
        o["positions"] = torch.empty(n, dtype=torch.int64, device=dev)
    if "slot_mapping" not in o:
        o["slot_mapping"] = torch.empty(n, dtype=torch.int64, device=dev)
    if "hidden" not in o:
        o["hidden"] = torch.empty((n, H), dtype=target_hidden.dtype, device=dev)
    if "sample_rows" not in o and want_sample_rows:
        o["sample_rows"] = torch.empty((B, K), dtype=torch.int32, device=dev)
    _dev(o["input_ids"], "input_ids", torch.int32, (n,), dev)
    _dev(o["positions"], "positions", torch.int64, (n,), dev)
    _dev(o["slot_mapping"], "slot_mapping", torch.int64, (n,), dev)
    _dev(o["hidden"], "hidden", target_hidden.dtype, (n, H), dev)
    if o.get("sample_rows") is not None:
        _dev(o["sample_rows"], "sample_rows", torch.int32, (B, K), dev)
    if device_error is not None:
        _dev(device_error, "device_error", torch.int32, (1,), dev)
    st = lib.peagle_build_draft_batch(
        _ptr(verify_out_tokens), _ptr(num_accepted), _ptr(draft_tokens), _ptr(start_pos),
        _ptr(block_table), block_table.shape[1], int(block_size), _ptr(target_hidden), _ptr(h_shared),
        _DTYPES[target_hidden.dtype], int(mask_token_id), B, K, H, _ptr(o["input_ids"]),
        _ptr(o["positions"]), _ptr(o["slot_mapping"]), _ptr(o["hidden"]), _ptr(o.get("sample_rows")),
        _ptr(device_error), _stream(dev))
    _check(st, "peagle_build_draft_batch")
    return o


# ---------------------------------------------------------------- drafter outputs
def spec_draft_sample(drafter_logits: torch.Tensor, K: int, temperature: float,
                      uniforms: Optional[torch.Tensor] = None,
                      row_index: Optional[torch.Tensor] = None,
                      temperatures: Optional[torch.Tensor] = None,
                      out_draft_tokens: Optional[torch.Tensor] = None,
                      out_draft_probs: Optional[torch.Tensor] = None,
                      want_draft_probs: bool = True,
                      device_error: Optional[torch.Tensor] = None,
                      out_row_desc: Optional[torch.Tensor] = None,
                      want_row_desc: bool = False):
    """Sample the drafter's prediction rows; see spec_draft_sample in
    include/spec_verify.h.  drafter_logits is [n_rows, V]; B is taken from
    row_index ([B, K]) when given, else n_rows // K.

    Returns (draft_tokens [B, K] int32, draft_probs [B, K, V] fp32 or None),
    plus the row descriptors ([B, K, 4] int32 holding sv_draft_row) as a third
    element when want_row_desc or out_row_desc is given.
    """
    lib = require_library()
    if drafter_logits.dim() != 2:
        raise ValueError("drafter_logits must be [n_rows, V]")
    n_rows, V = drafter_logits.shape
    dev = drafter_logits.device
    _dev(drafter_logits, "drafter_logits")
    if drafter_logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("drafter_logits must be float32 or bfloat16")
    if row_index is not None:
        if row_index.dim() != 2 or row_index.shape[1] != K:
            raise ValueError("row_index must be [B, K]")
        B = row_index.shape[0]
        _dev(row_index, "row_index", torch.int32, (B, K), dev)
    else:
        if K < 1 or n_rows % K:
            raise ValueError("without row_index, n_rows must be a multiple of K")
        B = n_rows // K
    if uniforms is not None:
        _dev(uniforms, "uniforms", torch.float32, (B, K), dev)
    if temperatures is not None:
        _dev(temperatures, "temperatures", torch.float32, (B,), dev)
    out_draft_tokens = torch.empty((B, K), dtype=torch.int32, device=dev) \
        if out_draft_tokens is None else _dev(out_draft_tokens, "out_draft_tokens", torch.int32,
                                             (B, K), dev)
    if out_draft_probs is None and want_draft_probs:
        out_draft_probs = torch.empty((B, K, V), dtype=torch.float32, device=dev)
    if out_draft_probs is not None:
        _dev(out_draft_probs, "out_draft_probs", torch.float32, (B, K, V), dev)
    if device_error is not None:
        _dev(device_error, "device_error", torch.int32, (1,), dev)
    with_desc = want_row_desc or out_row_desc is not None
    if out_row_desc is None and want_row_desc:
        out_row_desc = torch.empty((B, K, 4), dtype=torch.int32, device=dev)
    if out_row_desc is not None:
        _dev(out_row_desc, "out_row_desc", torch.int32, (B, K, 4), dev)
    st = lib.spec_draft_sample(_ptr(drafter_logits), _DTYPES[drafter_logits.dtype], n_rows,
                               _ptr(row_index), _ptr(uniforms), float(temperature),
                               _ptr(temperatures), B, K, V, _ptr(out_draft_tokens),
                               _ptr(out_draft_probs), _ptr(out_row_desc), _ptr(device_error),
                               _stream(dev))
    _check(st, "spec_draft_sample")
    if with_desc:
        return out_draft_tokens, out_draft_probs, out_row_desc
    return out_draft_tokens, out_draft_probs


def _verify_lq(name, target_logits, drafter_logits, drafter_desc, draft_tokens, uniforms,
               temperature, temperatures, drafter_rows, out_tokens, out_num_accepted,
               out_draft_target_prob, want_draft_target_prob, workspace, device_error):
    lib = require_library()
    if target_logits.dim() != 3 or drafter_logits.dim() != 2:
        raise ValueError("target_logits must be [B, K+1, V] and drafter_logits [n_rows, V]")
    B, K1, V = target_logits.shape
    K = K1 - 1
    dev = target_logits.device
    _dev(target_logits, "target_logits")
    if target_logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("target_logits must be float32 or bfloat16")
    _dev(drafter_logits, "drafter_logits", target_logits.dtype, (drafter_logits.shape[0], V), dev)
    _dev(drafter_desc, "drafter_desc", torch.int32, (B, K, 4), dev)
    _dev(draft_tokens, "draft_tokens", torch.int32, (B, K), dev)
    _dev(uniforms, "uniforms", torch.float32, (B, K + 1), dev)
    if temperatures is not None:
        _dev(temperatures, "temperatures", torch.float32, (B,), dev)
    if drafter_rows is not None:
        _dev(drafter_rows, "drafter_rows", torch.int32, (B, K), dev)
    out_tokens = torch.empty((B, K + 1), dtype=torch.int32, device=dev) if out_tokens is None \
        else _dev(out_tokens, "out_tokens", torch.int32, (B, K + 1), dev)
    out_num_accepted = torch.empty(B, dtype=torch.int32, device=dev) if out_num_accepted is None \
        else _dev(out_num_accepted, "out_num_accepted", torch.int32, (B,), dev)
    if out_draft_target_prob is None and want_draft_target_prob:
        out_draft_target_prob = torch.empty((B, K), dtype=torch.float32, device=dev)
    if out_draft_target_prob is not None:
        _dev(out_draft_target_prob, "out_draft_target_prob", torch.float32, (B, K), dev)
    need = spec_verify_workspace_bytes(B, K, V)
    if workspace is None:
        workspace = _workspace(dev, need)
    _dev(workspace, "workspace", device=dev)
    if device_error is not None:
        _dev(device_error, "device_error", torch.int32, (1,), dev)
    head = (_ptr(target_logits), _DTYPES[target_logits.dtype], _ptr(drafter_logits),
            drafter_logits.shape[0], _ptr(drafter_rows), _ptr(drafter_desc), _ptr(draft_tokens),
            _ptr(uniforms))
    tail = (B, K, V, _ptr(out_tokens), _ptr(out_num_accepted), _ptr(out_draft_target_prob),
            _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(device_error),
            _stream(dev))
    if name.startswith("spec_verify_mixed_lq"):
        st = getattr(lib, name)(*head, _ptr(temperatures), *tail)
    else:
        st = getattr(lib, name)(*head, float(temperature), *tail)
    _check(st, name)
    return out_tokens, out_num_accepted, out_draft_target_prob


def spec_verify_sample_lq(target_logits: torch.Tensor, drafter_logits: torch.Tensor,
                          drafter_desc: torch.Tensor, draft_tokens: torch.Tensor,
                          uniforms: torch.Tensor, temperature: float,
                          drafter_rows: Optional[torch.Tensor] = None,
                          out_tokens: Optional[torch.Tensor] = None,
                          out_num_accepted: Optional[torch.Tensor] = None,
                          out_draft_target_prob: Optional[torch.Tensor] = None,
                          want_draft_target_prob: bool = False,
                          workspace: Optional[torch.Tensor] = None,
                          device_error: Optional[torch.Tensor] = None):
    """Sampled verify with q recomputed from the drafter logits and the row
    descriptors of spec_draft_sample; see spec_verify_sample_lq in
    include/spec_verify.h.  Returns (out_tokens, num_accepted, draft_target_prob
    or None)."""
    return _verify_lq("spec_verify_sample_lq", target_logits, drafter_logits, drafter_desc,
                      draft_tokens, uniforms, temperature, None, drafter_rows, out_tokens,
                      out_num_accepted, out_draft_target_prob, want_draft_target_prob,
                      workspace, device_error)


def spec_verify_mixed_lq(target_logits: torch.Tensor, drafter_logits: torch.Tensor,
                         drafter_desc: torch.Tensor, draft_tokens: torch.Tensor,
                         uniforms: torch.Tensor, temperatures: torch.Tensor,
                         drafter_rows: Optional[torch.Tensor] = None,
                         out_tokens: Optional[torch.Tensor] = None,
                         out_num_accepted: Optional[torch.Tensor] = None,
                         out_draft_target_prob: Optional[torch.Tensor] = None,
                         want_draft_target_prob: bool = False,
                         workspace: Optional[torch.Tensor] = None,
                         device_error: Optional[torch.Tensor] = None):
    """Mixed-batch verify (per-sequence temperatures, 0 = greedy) with q
    recomputed from the drafter logits and row descriptors; see
    spec_verify_mixed_lq in include/spec_verify.h.  Returns (out_tokens,
    num_accepted, draft_target_prob or None)."""
    return _verify_lq("spec_verify_mixed_lq", target_logits, drafter_logits, drafter_desc,
                      draft_tokens, uniforms, None, temperatures, drafter_rows, out_tokens,
                      out_num_accepted, out_draft_target_prob, want_draft_target_prob,
                      workspace, device_error)


def spec_verify_sample_lq_early_exit(target_logits, drafter_logits, drafter_desc, draft_tokens,
                                     uniforms, temperature, drafter_rows=None, out_tokens=None,
                                     out_num_accepted=None, out_draft_target_prob=None,
                                     want_draft_target_prob=False, workspace=None,
                                     device_error=None):
    """spec_verify_sample_lq computing only the rows up to each sequence's
    first rejection; see spec_verify_sample_lq_early_exit in
    include/spec_verify.h.  draft_target_prob is 0 past num_accepted."""
    return _verify_lq("spec_verify_sample_lq_early_exit", target_logits, drafter_logits,
                      drafter_desc, draft_tokens, uniforms, temperature, None, drafter_rows,
                      out_tokens, out_num_accepted, out_draft_target_prob,
                      want_draft_target_prob, workspace, device_error)


def spec_verify_mixed_lq_early_exit(target_logits, drafter_logits, drafter_desc, draft_tokens,
                                    uniforms, temperatures, drafter_rows=None, out_tokens=None,
                                    out_num_accepted=None, out_draft_target_prob=None,
                                    want_draft_target_prob=False, workspace=None,
                                    device_error=None):
    """spec_verify_mixed_lq computing only the rows up to each sequence's
    first rejection; see spec_verify_mixed_lq_early_exit in
    include/spec_verify.h.  draft_target_prob is 0 past num_accepted."""
    return _verify_lq("spec_verify_mixed_lq_early_exit", target_logits, drafter_logits,
                      drafter_desc, draft_tokens, uniforms, None, temperatures, drafter_rows,
                      out_tokens, out_num_accepted, out_draft_target_prob,
                      want_draft_target_prob, workspace, device_error)


# ---------------------------------------------------------------- filtered distributions
def _rows(t: torch.Tensor, name: str, device=None, dtype=None) -> int:
    """Checks logit rows [..., V] whose rows may be spaced wider than V (a
    padded vocabulary); returns the elements between rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name} must be float32 or bfloat16")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    V = t.shape[-1]
    if V < 1:
        raise ValueError(f"{name} must have at least one token per row")
    if t.is_contiguous() or t.numel() == 0:
        return V
    step, rows = None, 1
    for d in range(t.dim() - 2, -1, -1):           # the rows are evenly spaced in memory
        if t.shape[d] == 1:
            continue
        if step is None:
            step = t.stride(d)
        elif t.stride(d) != step * rows:
            raise ValueError(f"{name}'s rows must be evenly spaced")
        rows *= t.shape[d]
    if (t.stride(-1) != 1 and V > 1) or (step is not None and step < V):
        raise ValueError(f"{name}'s rows must be contiguous and must not overlap")
    return V if step is None else step


def _settings(B, device, top_ks, top_ps, min_ps):
    """Checks the per-sequence filter settings and returns their pointers."""
    for t, name, dtype in ((top_ks, "top_ks", torch.int32), (top_ps, "top_ps", torch.float32),
                           (min_ps, "min_ps", torch.float32)):
        if t is not None:
            _dev(t, name, dtype, (B,), device)
    return _ptr(top_ks), _ptr(top_ps), _ptr(min_ps)


def spec_filter_workspace_bytes(n_rows: int, V: int) -> int:
    return int(require_library().spec_filter_workspace_bytes(int(n_rows), int(V)))


def _filter_workspace(workspace, n_rows, V, device):
    """The caller's workspace, or one of this call's own from torch's allocator
    (which keeps it until the stream is past the call, also under capture)."""
    if workspace is None:
        return torch.empty(max(16, spec_filter_workspace_bytes(n_rows, V)), dtype=torch.uint8,
                           device=device)
    return _dev(workspace, "workspace", device=device)


def _on(device):
    """The guard under which a call launches: its tensors' device is current."""
    return torch.cuda.device(device)


def spec_draft_sample_filtered(drafter_logits: torch.Tensor, K: int, temperature: float = 1.0,
                               top_ks: Optional[torch.Tensor] = None,
                               top_ps: Optional[torch.Tensor] = None,
                               min_ps: Optional[torch.Tensor] = None,
                               uniforms: Optional[torch.Tensor] = None,
                               row_index: Optional[torch.Tensor] = None,
                               temperatures: Optional[torch.Tensor] = None,
                               out_draft_tokens: Optional[torch.Tensor] = None,
                               out_draft_probs: Optional[torch.Tensor] = None,
                               want_draft_probs: bool = False,
                               out_filter_rows: Optional[torch.Tensor] = None,
                               want_filter_rows: bool = False,
                               workspace: Optional[torch.Tensor] = None,
                               device_error: Optional[torch.Tensor] = None):
    """Sample logit rows under temperature, top-k, top-p and min-p; see
    spec_draft_sample_filtered in include/spec_verify.h.

    drafter_logits [n_rows, V] float32/bfloat16 (rows may be spaced wider than
    V); B is taken from row_index ([B, K]) when given, else n_rows // K.  K = 1
    samples one token per row (a decode step without drafts).  top_ks [B] int32
    (0 = off), top_ps [B] and min_ps [B] float32 (1 and 0 = off) are per
    sequence, None = off for all; temperatures [B] overrides temperature.

    Returns (draft_tokens [B, K] int32, draft_probs [B, K, V] fp32 or None,
    filter_rows [B, K, 8] int32 holding sv_filter_row or None).
    """
    lib = require_library()
    if drafter_logits.dim() != 2:
        raise ValueError("drafter_logits must be [n_rows, V]")
    n_rows, V = drafter_logits.shape
    dev = drafter_logits.device
    stride = _rows(drafter_logits, "drafter_logits")
    if row_index is not None:
        if row_index.dim() != 2 or row_index.shape[1] != K:
            raise ValueError("row_index must be [B, K]")
        B = row_index.shape[0]
        _dev(row_index, "row_index", torch.int32, (B, K), dev)
    else:
        if K < 1 or n_rows % K:
            raise ValueError("without row_index, n_rows must be a multiple of K")
        B = n_rows // K
    if uniforms is not None:
        _dev(uniforms, "uniforms", torch.float32, (B, K), dev)
    if temperatures is not None:
        _dev(temperatures, "temperatures", torch.float32, (B,), dev)
    settings = _settings(B, dev, top_ks, top_ps, min_ps)
    out_draft_tokens = torch.empty((B, K), dtype=torch.int32, device=dev) \
        if out_draft_tokens is None else _dev(out_draft_tokens, "out_draft_tokens", torch.int32,
                                              (B, K), dev)
    if out_draft_probs is None and want_draft_probs:
        out_draft_probs = torch.empty((B, K, V), dtype=torch.float32, device=dev)
    if out_draft_probs is not None:
        _dev(out_draft_probs, "out_draft_probs", torch.float32, (B, K, V), dev)
    if out_filter_rows is None and want_filter_rows:
        out_filter_rows = torch.empty((B, K, 8), dtype=torch.int32, device=dev)
    if out_filter_rows is not None:
        _dev(out_filter_rows, "out_filter_rows", torch.int32, (B, K, 8), dev)
    if device_error is not None:
        _dev(device_error, "device_error", torch.int32, (1,), dev)
    workspace = _filter_workspace(workspace, B * K, V, dev)
    with _on(dev):
        st = lib.spec_draft_sample_filtered(
            _ptr(drafter_logits), _DTYPES[drafter_logits.dtype], n_rows, stride, _ptr(row_index),
            _ptr(uniforms), float(temperature), _ptr(temperatures), *settings, B, K, V,
            _ptr(out_draft_tokens), _ptr(out_draft_probs), _ptr(out_filter_rows), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _ptr(device_error), _stream(dev))
    _check(st, "spec_draft_sample_filtered")
    return out_draft_tokens, out_draft_probs, out_filter_rows


def _verify_filtered(name, target_logits, q_args, draft_tokens, uniforms, temperatures, top_ks,
                     top_ps, min_ps, out_tokens, out_num_accepted, out_draft_target_prob,
                     want_draft_target_prob, workspace, device_error):
    """spec_verify_filtered and _lq: q_args(B, K, V, device) checks the q
    arguments and gives what the library takes for them."""
    lib = require_library()
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, K+1, V]")
    B, K1, V = target_logits.shape
    K = K1 - 1
    dev = target_logits.device
    stride = _rows(target_logits, "target_logits")
    q = q_args(B, K, V, dev)
    _dev(draft_tokens, "draft_tokens", torch.int32, (B, K), dev)
    _dev(uniforms, "uniforms", torch.float32, (B, K + 1), dev)
    _dev(temperatures, "temperatures", torch.float32, (B,), dev)
    settings = _settings(B, dev, top_ks, top_ps, min_ps)
    out_tokens = torch.empty((B, K + 1), dtype=torch.int32, device=dev) if out_tokens is None \
        else _dev(out_tokens, "out_tokens", torch.int32, (B, K + 1), dev)
    out_num_accepted = torch.empty(B, dtype=torch.int32, device=dev) if out_num_accepted is None \
        else _dev(out_num_accepted, "out_num_accepted", torch.int32, (B,), dev)
    if out_draft_target_prob is None and want_draft_target_prob:
        out_draft_target_prob = torch.empty((B, K), dtype=torch.float32, device=dev)
    if out_draft_target_prob is not None:
        _dev(out_draft_target_prob, "out_draft_target_prob", torch.float32, (B, K), dev)
    if device_error is not None:
        _dev(device_error, "device_error", torch.int32, (1,), dev)
    workspace = _filter_workspace(workspace, B * (K + 1), V, dev)
    with _on(dev):
        st = getattr(lib, name)(
            _ptr(target_logits), _DTYPES[target_logits.dtype], stride, *q, _ptr(draft_tokens),
            _ptr(uniforms), _ptr(temperatures), *settings, B, K, V, _ptr(out_tokens),
            _ptr(out_num_accepted), _ptr(out_draft_target_prob), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _ptr(device_error), _stream(dev))
    _check(st, name)
    return out_tokens, out_num_accepted, out_draft_target_prob


def spec_verify_filtered(target_logits: torch.Tensor, draft_probs: torch.Tensor,
                         draft_tokens: torch.Tensor, uniforms: torch.Tensor,
                         temperatures: torch.Tensor, top_ks: Optional[torch.Tensor] = None,
                         top_ps: Optional[torch.Tensor] = None,
                         min_ps: Optional[torch.Tensor] = None,
                         out_tokens: Optional[torch.Tensor] = None,
                         out_num_accepted: Optional[torch.Tensor] = None,
                         out_draft_target_prob: Optional[torch.Tensor] = None,
                         want_draft_target_prob: bool = False,
                         workspace: Optional[torch.Tensor] = None,
                         device_error: Optional[torch.Tensor] = None):
    """Verify against the target's filtered distributions (per-sequence
    temperature, 0 = greedy, top-k, top-p and min-p); see spec_verify_filtered
    in include/spec_verify.h.  target_logits [B, K+1, V] (rows may be spaced
    wider than V), draft_probs [B, K, V] float32; settings as for
    spec_draft_sample_filtered.

    Returns (out_tokens [B, K+1], num_accepted [B], draft_target_prob or None).
    """
    def q_args(B, K, V, dev):
        _dev(draft_probs, "draft_probs", torch.float32, (B, K, V), dev)
        return (_ptr(draft_probs),)

    return _verify_filtered("spec_verify_filtered", target_logits, q_args, draft_tokens, uniforms,
                            temperatures, top_ks, top_ps, min_ps, out_tokens, out_num_accepted,
                            out_draft_target_prob, want_draft_target_prob, workspace, device_error)


def spec_verify_filtered_lq(target_logits: torch.Tensor, drafter_logits: torch.Tensor,
                            filter_rows: torch.Tensor, draft_tokens: torch.Tensor,
                            uniforms: torch.Tensor, temperatures: torch.Tensor,
                            top_ks: Optional[torch.Tensor] = None,
                            top_ps: Optional[torch.Tensor] = None,
                            min_ps: Optional[torch.Tensor] = None,
                            drafter_rows: Optional[torch.Tensor] = None,
                            out_tokens: Optional[torch.Tensor] = None,
                            out_num_accepted: Optional[torch.Tensor] = None,
                            out_draft_target_prob: Optional[torch.Tensor] = None,
                            want_draft_target_prob: bool = False,
                            workspace: Optional[torch.Tensor] = None,
                            device_error: Optional[torch.Tensor] = None):
    """spec_verify_filtered with q from the drafter's logits [n_rows, V] and the
    filter rows ([B, K, 8] int32) of spec_draft_sample_filtered; see
    spec_verify_filtered_lq in include/spec_verify.h."""
    def q_args(B, K, V, dev):
        if drafter_logits.dim() != 2 or drafter_logits.shape[1] != V:
            raise ValueError("drafter_logits must be [n_rows, V]")
        d_stride = _rows(drafter_logits, "drafter_logits", dev, target_logits.dtype)
        _dev(filter_rows, "filter_rows", torch.int32, (B, K, 8), dev)
        if drafter_rows is not None:
            _dev(drafter_rows, "drafter_rows", torch.int32, (B, K), dev)
        return (_ptr(drafter_logits), drafter_logits.shape[0], d_stride, _ptr(drafter_rows),
                _ptr(filter_rows))

    return _verify_filtered("spec_verify_filtered_lq", target_logits, q_args, draft_tokens,
                            uniforms, temperatures, top_ks, top_ps, min_ps, out_tokens,
                            out_num_accepted, out_draft_target_prob, want_draft_target_prob,
                            workspace, device_error)


# ---------------------------------------------------------------- paged cache
def _heads(t: torch.Tensor, name: str, R, D, dtype, device):
    """Checks [R, heads, D] rows with dense heads; returns (heads, elements
    between rows)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or t.shape[0] != R or t.shape[2] != D:
        raise ValueError(f"{name} must be [{R}, heads, {D}], got {tuple(t.shape)}")
    H = t.shape[1]
    if t.numel() and ((D > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != D)):
        raise ValueError(f"{name}'s heads must be dense in each row")
    stride = t.stride(0) if R > 1 else H * D
    if stride < H * D and t.numel():
        raise ValueError(f"{name}'s rows must not overlap")
    return H, max(stride, H * D)


def peagle_append_kv(key: torch.Tensor, value: torch.Tensor, positions: torch.Tensor,
                     slot_mapping: torch.Tensor, key_cache: torch.Tensor,
                     value_cache: torch.Tensor, inv_freq: Optional[torch.Tensor] = None,
                     interleaved: bool = False, rotary_scale: float = 1.0,
                     query: Optional[torch.Tensor] = None,
                     out_query: Optional[torch.Tensor] = None,
                     k_scales: Optional[torch.Tensor] = None,
                     v_scales: Optional[torch.Tensor] = None,
                     device_error: Optional[torch.Tensor] = None):
    """Append keys and values to a paged cache, rotating keys (and queries) by
    their positions; see peagle_append_kv in include/spec_verify.h.

    key, value [R, kv_heads, D] and the optional query [R, q_heads, D] in
    bfloat16, float16 or float32 (rows may be views into one projection);
    positions and slot_mapping [R] int64 as peagle_build_draft_batch writes them
    (slot -1: nothing is written); inv_freq [rotary_dim / 2] float32, None for no
    rotation; caches [num_blocks, block_size, kv_heads, D] of the same type or
    float8_e4m3fn, the last dimension dense, the others with any strides that
    both caches share; k_scales, v_scales [kv_heads] float32 for e4m3 caches.

    Returns the rotated queries (out_query, which may be query itself) or None.
    """
    lib = require_library()
    if not isinstance(key, torch.Tensor) or key.dim() != 3:
        raise ValueError("key must be [R, kv_heads, head_dim]")
    R, Hkv, D = key.shape
    dev, dtype = key.device, key.dtype
    if dtype not in _DTYPES:
        raise TypeError("keys must be bfloat16, float16 or float32")
    _, ks = _heads(key, "key", R, D, dtype, dev)
    Hv, vs = _heads(value, "value", R, D, dtype, dev)
    if Hv != Hkv:
        raise ValueError(f"value must have {Hkv} heads, got {Hv}")
    _dev(positions, "positions", torch.int64, (R,), dev)
    _dev(slot_mapping, "slot_mapping", torch.int64, (R,), dev)
    rot = 0
    if inv_freq is not None:
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be [rotary_dim / 2]")
        _dev(inv_freq, "inv_freq", torch.float32, device=dev)
        rot = 2 * inv_freq.shape[0]
    if key_cache.dim() != 4 or key_cache.shape[2:] != (Hkv, D):
        raise ValueError(f"key_cache must be [num_blocks, block_size, {Hkv}, {D}]")
    if value_cache.shape != key_cache.shape:
        raise ValueError("key_cache and value_cache must have one shape")
    for t, name in ((key_cache, "key_cache"), (value_cache, "value_cache")):
        if not t.is_cuda or t.device != dev:
            raise ValueError(f"{name} must be on {dev}")
        if t.dtype is not dtype and t.dtype is not torch.float8_e4m3fn:
            raise TypeError(f"{name} must be {dtype} or float8_e4m3fn")
    if key_cache.dtype is not value_cache.dtype or key_cache.stride() != value_cache.stride():
        raise ValueError("key_cache and value_cache must have one type and one layout")
    if D > 1 and key_cache.stride(3) != 1:
        raise ValueError("the caches' last dimension must be dense")
    fp8 = key_cache.dtype is torch.float8_e4m3fn
    for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
        if t is not None:
            if not fp8:
                raise ValueError(f"{name} are for float8_e4m3fn caches")
            _dev(t, name, torch.float32, (Hkv,), dev)
    Hq = qs = oqs = 0
    if query is not None:
        if query.dim() != 3:
            raise ValueError("query must be [R, q_heads, head_dim]")
        Hq, qs = _heads(query, "query", R, D, dtype, dev)
        if out_query is None:
            out_query = torch.empty((R, Hq, D), dtype=dtype, device=dev)
        Ho, oqs = _heads(out_query, "out_query", R, D, dtype, dev)
        if Ho != Hq:
            raise ValueError(f"out_query must have {Hq} heads, got {Ho}")
    elif out_query is not None:
        raise ValueError("out_query without query")
    if device_error is not None:
        _dev(device_error, "device_error", torch.int32, (1,), dev)
    nb, bs = key_cache.shape[:2]
    with _on(dev):
        st = lib.peagle_append_kv(
            _ptr(query), _ptr(key), _ptr(value), _DTYPES[dtype], qs, ks, vs, _ptr(positions),
            _ptr(slot_mapping), _ptr(inv_freq), rot, 1 if interleaved else 0, float(rotary_scale),
            R, Hq, Hkv, D, _ptr(key_cache), _ptr(value_cache), SV_E4M3 if fp8 else _DTYPES[dtype],
            nb, bs, key_cache.stride(0), key_cache.stride(1), key_cache.stride(2),
            _ptr(k_scales), _ptr(v_scales), _ptr(out_query), oqs, _ptr(device_error), _stream(dev))
    _check(st, "peagle_append_kv")
    return out_query


# ---------------------------------------------------------------- draft trees
def spec_verify_tree(target_logits: torch.Tensor, parents: torch.Tensor, tokens: torch.Tensor,
                     temperature: float = 0.0, draft_probs: Optional[torch.Tensor] = None,
                     uniforms: Optional[torch.Tensor] = None,
                     out_tokens: Optional[torch.Tensor] = None,
                     out_path: Optional[torch.Tensor] = None,
                     out_num_accepted: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     device_error: Optional[torch.Tensor] = None,
                     _symbol: str = "spec_verify_tree", _temperatures=None):
    """Verify a draft tree per sequence (temperature 0 = greedy); see
    spec_verify_tree in include/spec_verify.h.

    Returns (out_tokens [B, N+1], out_path [B, N+1], num_accepted [B])."""
    lib = require_library()
    mixed = _temperatures is not None
    if mixed:
        temperature = 1.0                  # per-tree temperatures instead
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, N+1, V]")
    B, N1, V = target_logits.shape
    N = N1 - 1
    dev = target_logits.device
    _dev(target_logits, "target_logits")
    if target_logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("target_logits must be float32 or bfloat16")
    _dev(parents, "parents", torch.int32, (B, N), dev)
    _dev(tokens, "tokens", torch.int32, (B, N), dev)
    if temperature > 0:
        _dev(draft_probs, "draft_probs", torch.float32, (B, N + 1, V), dev)
        _dev(uniforms, "uniforms", torch.float32, (B, N + 1), dev)
    out_tokens = torch.empty((B, N + 1), dtype=torch.int32, device=dev) if out_tokens is None \
        else _dev(out_tokens, "out_tokens", torch.int32, (B, N + 1), dev)
    out_path = torch.empty((B, N + 1), dtype=torch.int32, device=dev) if out_path is None \
        else _dev(out_path, "out_path", torch.int32, (B, N + 1), dev)
    out_num_accepted = torch.empty(B, dtype=torch.int32, device=dev) if out_num_accepted is None \
        else _dev(out_num_accepted, "out_num_accepted", torch.int32, (B,), dev)
    need = spec_verify_workspace_bytes(B, N, V)
    if workspace is None:
        workspace = _workspace(dev, need)
    _dev(workspace, "workspace", device=dev)
    if device_error is not None:
        _dev(device_error, "device_error", torch.int32, (1,), dev)
    head = (_ptr(target_logits), _DTYPES[target_logits.dtype],
            _ptr(draft_probs if temperature > 0 else None), _ptr(parents), _ptr(tokens),
            _ptr(uniforms if temperature > 0 else None))
    tail = (B, N, V, _ptr(out_tokens), _ptr(out_path), _ptr(out_num_accepted), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _ptr(device_error), _stream(dev))
    if mixed:
        _dev(_temperatures, "temperatures", torch.float32, (B,), dev)
        st = getattr(lib, _symbol)(*head, _ptr(_temperatures), *tail)
    else:
        st = getattr(lib, _symbol)(*head, float(temperature), *tail)
    _check(st, _symbol)
    return out_tokens, out_path, out_num_accepted


def spec_verify_tree_mixed(target_logits, parents, tokens, temperatures, draft_probs, uniforms,
                           **kw):
    """Verify a mixed batch of draft trees (per-tree temperatures, 0 =
    greedy); see spec_verify_tree_mixed in include/spec_verify.h.  Keyword
    arguments and results as spec_verify_tree."""
    return spec_verify_tree(target_logits, parents, tokens, 1.0, draft_probs, uniforms,
                            _symbol="spec_verify_tree_mixed", _temperatures=temperatures, **kw)


def spec_verify_tree_mixed_early_exit(target_logits, parents, tokens, temperatures,
                                      draft_probs, uniforms, **kw):
    """spec_verify_tree_mixed with the walk computing the statistics of the
    rows it visits only; see spec_verify_tree_mixed_early_exit."""
    return spec_verify_tree(target_logits, parents, tokens, 1.0, draft_probs, uniforms,
                            _symbol="spec_verify_tree_mixed_early_exit",
                            _temperatures=temperatures, **kw)


def spec_verify_tree_lq(target_logits: torch.Tensor, drafter_logits: torch.Tensor,
                        drafter_desc: torch.Tensor, parents: torch.Tensor, tokens: torch.Tensor,
                        uniforms: torch.Tensor, temperature: float,
                        drafter_rows: Optional[torch.Tensor] = None,
                        out_tokens: Optional[torch.Tensor] = None,
                        out_path: Optional[torch.Tensor] = None,
                        out_num_accepted: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None,
                        device_error: Optional[torch.Tensor] = None,
                        _symbol: str = "spec_verify_tree_lq"):
    """Sampled tree verification with q recomputed from the drafter logits
    and the row descriptors of spec_draft_sample; see spec_verify_tree_lq in
    include/spec_verify.h.  drafter_desc is [B, N+1, 4] int32 (sv_draft_row),
    drafter_rows optional [B, N+1].

    Returns (out_tokens [B, N+1], out_path [B, N+1], num_accepted [B])."""
    lib = require_library()
    if target_logits.dim() != 3 or drafter_logits.dim() != 2:
        raise ValueError("target_logits must be [B, N+1, V] and drafter_logits [n_rows, V]")
    B, N1, V = target_logits.shape
    N = N1 - 1
    dev = target_logits.device
    _dev(target_logits, "target_logits")
    if target_logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("target_logits must be float32 or bfloat16")
    _dev(drafter_logits, "drafter_logits", target_logits.dtype, (drafter_logits.shape[0], V), dev)
    _dev(drafter_desc, "drafter_desc", torch.int32, (B, N + 1, 4), dev)
    _dev(parents, "parents", torch.int32, (B, N), dev)
    _dev(tokens, "tokens", torch.int32, (B, N), dev)
    _dev(uniforms, "uniforms", torch.float32, (B, N + 1), dev)
    if drafter_rows is not None:
        _dev(drafter_rows, "drafter_rows", torch.int32, (B, N + 1), dev)
    out_tokens = torch.empty((B, N + 1), dtype=torch.int32, device=dev) if out_tokens is None \
        else _dev(out_tokens, "out_tokens", torch.int32, (B, N + 1), dev)
    out_path = torch.empty((B, N + 1), dtype=torch.int32, device=dev) if out_path is None \
        else _dev(out_path, "out_path", torch.int32, (B, N + 1), dev)
    out_num_accepted = torch.empty(B, dtype=torch.int32, device=dev) if out_num_accepted is None \
        else _dev(out_num_accepted, "out_num_accepted", torch.int32, (B,), dev)
    need = spec_verify_workspace_bytes(B, N, V)
    if workspace is None:
        workspace = _workspace(dev, need)
    _dev(workspace, "workspace", device=dev)
    if device_error is not None:
        _dev(device_error, "device_error", torch.int32, (1,), dev)
    st = getattr(lib, _symbol)(_ptr(target_logits), _DTYPES[target_logits.dtype],
                                 _ptr(drafter_logits), drafter_logits.shape[0],
                                 _ptr(drafter_rows), _ptr(drafter_desc), _ptr(parents),
                                 _ptr(tokens), _ptr(uniforms), float(temperature), B, N, V,
                                 _ptr(out_tokens), _ptr(out_path), _ptr(out_num_accepted),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _ptr(device_error), _stream(dev))
    _check(st, _symbol)
    return out_tokens, out_path, out_num_accepted


def spec_verify_tree_early_exit(*args, **kw):
    """spec_verify_tree with the walk computing the statistics of the rows it
    visits only; see spec_verify_tree_early_exit in include/spec_verify.h.
    Arguments and results as spec_verify_tree."""
    return spec_verify_tree(*args, _symbol="spec_verify_tree_early_exit", **kw)


def spec_verify_tree_lq_early_exit(*args, **kw):
    """spec_verify_tree_lq with the walk computing the statistics of the rows
    it visits only; see spec_verify_tree_lq_early_exit in include/spec_verify.h."""
    return spec_verify_tree_lq(*args, _symbol="spec_verify_tree_lq_early_exit", **kw)


# ---------------------------------------------------------------- acceptance metrics
METRICS_STEPS, METRICS_ROUNDS, METRICS_PROPOSED, METRICS_ACCEPTED, METRICS_EMITTED, \
    METRICS_HIST = range(6)


def accept_metrics_buffer(K: int, device) -> torch.Tensor:
    """A zeroed counter array for spec_accept_metrics (int64 storage of the
    uint64 counters)."""
    n = require_library().spec_accept_metrics_words(int(K))
    if n == 0:
        raise ValueError(f"K={K} out of range")
    return torch.zeros(n, dtype=torch.int64, device=device)


def spec_accept_metrics(num_accepted: torch.Tensor, K: int, metrics: torch.Tensor,
                        device_error: Optional[torch.Tensor] = None):
    """Add one verify call's counts to `metrics`; see spec_accept_metrics in
    include/spec_verify.h."""
    lib = require_library()
    if num_accepted.dim() != 1:
        raise ValueError("num_accepted must be [B]")
    B = num_accepted.shape[0]
    dev = num_accepted.device
    _dev(num_accepted, "num_accepted", torch.int32, (B,), dev)
    _dev(metrics, "metrics", torch.int64, (lib.spec_accept_metrics_words(int(K)),), dev)
    if device_error is not None:
        _dev(device_error, "device_error", torch.int32, (1,), dev)
    _check(lib.spec_accept_metrics(_ptr(num_accepted), B, int(K), _ptr(metrics),
                                   _ptr(device_error), _stream(dev)), "spec_accept_metrics")
    return metrics


def acceptance_summary(metrics: torch.Tensor) -> dict:
    """Host-side view of the counters (synchronises): reads back the integer
    counters that spec_accept_metrics accumulated on the device and divides
    them into the acceptance length, tokens per round and draft acceptance
    rate.  A reporting convenience, not part of the path: every count is
    taken on the GPU, and the three ratios are plain quotients of them."""
    m = [int(x) for x in metrics.cpu().tolist()]
    rounds, proposed, accepted, emitted = (m[METRICS_ROUNDS], m[METRICS_PROPOSED],
                                           m[METRICS_ACCEPTED], m[METRICS_EMITTED])
    return {"steps": m[METRICS_STEPS], "rounds": rounds, "proposed": proposed,
            "accepted": accepted, "emitted": emitted, "hist": m[METRICS_HIST:],
            "acceptance_length": accepted / rounds if rounds else float("nan"),
            "tokens_per_round": emitted / rounds if rounds else float("nan"),
            "draft_acceptance_rate": accepted / proposed if proposed else float("nan")}


# ---------------------------------------------------------------- step graphs
STEP_GREEDY, STEP_SAMPLE, STEP_MIXED = 0, 1, 2


class _StepDesc(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int), ("target_logits", _p), ("logits_dtype", ctypes.c_int),
                ("draft_probs", _p), ("draft_tokens", _p), ("uniforms", _p),
                ("temperature", ctypes.c_float), ("temperatures", _p),
                ("B", ctypes.c_int), ("K", ctypes.c_int), ("V", ctypes.c_int),
                ("out_tokens", _p), ("out_num_accepted", _p), ("out_draft_target_prob", _p),
                ("workspace", _p), ("workspace_bytes", ctypes.c_size_t),
                ("start_pos", _p), ("block_table", _p), ("max_blocks_per_seq", ctypes.c_int),
                ("block_size", ctypes.c_int), ("target_hidden", _p), ("h_shared", _p),
                ("hidden_dtype", ctypes.c_int), ("mask_token_id", ctypes.c_int32),
                ("H", ctypes.c_int), ("out_input_ids", _p), ("out_positions", _p),
                ("out_slot_mapping", _p), ("out_hidden", _p), ("out_sample_rows", _p),
                ("metrics", _p), ("device_error", _p),
                ("drafter_logits", _p), ("n_drafter_rows", ctypes.c_int64),
                ("drafter_rows", _p), ("drafter_desc", _p), ("early_exit", ctypes.c_int)]


class StepGraph:
    """One decode step (verify, then optionally the P-EAGLE build and the
    acceptance metrics) captured as a HIP graph; see sv_step_graph_create in
    include/spec_verify.h.  Every tensor is fixed at capture and kept alive
    by this object; ``launch()`` replays the step on the current stream with
    whatever the tensors hold.

    verify: dict with target_logits, draft_tokens, out_tokens,
      out_num_accepted, workspace, and for sampling draft_probs, uniforms and
      temperature (mode "sample") or temperatures (mode "mixed"); optional
      out_draft_target_prob.  For sampling with q from the drafter logits,
      drafter_logits ([n_rows, V]) and drafter_desc ([B, K, 4] int32, from
      spec_draft_sample) replace draft_probs, with an optional drafter_rows
      ([B, K] int32).
    build: None, or dict with start_pos, block_table, block_size,
      target_hidden, h_shared, mask_token_id and outputs (as returned by
      peagle_build_draft_batch or preallocated).
    metrics: None, or a counter array from accept_metrics_buffer.
    early_exit: capture the _early_exit form of the verify.
    """

    def __init__(self, mode: str, verify: dict, build: Optional[dict] = None,
                 metrics: Optional[torch.Tensor] = None,
                 device_error: Optional[torch.Tensor] = None, early_exit: bool = False):
        lib = require_library()
        z = verify["target_logits"]
        if z.dim() != 3:
            raise ValueError("target_logits must be [B, K+1, V]")
        B, K1, V = z.shape
        K = K1 - 1
        dev = z.device
        d = _StepDesc()
        d.mode = {"greedy": STEP_GREEDY, "sample": STEP_SAMPLE, "mixed": STEP_MIXED}[mode]
        d.early_exit = 1 if early_exit else 0
        keep = [z]

        def ptr(t, name, dtype=None, shape=None):
            if t is None:
                return None
            _dev(t, name, dtype, shape, dev)
            keep.append(t)
            return t.data_ptr()

        d.target_logits = ptr(z, "target_logits")
        d.logits_dtype = _DTYPES[z.dtype]
        d.draft_tokens = ptr(verify["draft_tokens"], "draft_tokens", torch.int32, (B, K))
        zd = verify.get("drafter_logits")
        if zd is not None:
            if mode == "greedy" or verify.get("draft_probs") is not None:
                raise ValueError("drafter_logits replaces draft_probs, for sampling only")
            if zd.dim() != 2 or zd.shape[1] != V or zd.dtype != z.dtype:
                raise ValueError("drafter_logits must be [n_rows, V] in the target's dtype")
            d.drafter_logits = ptr(zd, "drafter_logits")
            d.n_drafter_rows = zd.shape[0]
            d.drafter_rows = ptr(verify.get("drafter_rows"), "drafter_rows", torch.int32, (B, K))
            d.drafter_desc = ptr(verify["drafter_desc"], "drafter_desc", torch.int32, (B, K, 4))
        if mode != "greedy":
            if zd is None:
                d.draft_probs = ptr(verify["draft_probs"], "draft_probs", torch.float32,
                                    (B, K, V))
            d.uniforms = ptr(verify["uniforms"], "uniforms", torch.float32, (B, K + 1))
        if mode == "sample":
            d.temperature = float(verify["temperature"])
        if mode == "mixed":
            d.temperatures = ptr(verify["temperatures"], "temperatures", torch.float32, (B,))
        d.B, d.K, d.V = B, K, V
        d.out_tokens = ptr(verify["out_tokens"], "out_tokens", torch.int32, (B, K + 1))
        d.out_num_accepted = ptr(verify["out_num_accepted"], "out_num_accepted", torch.int32, (B,))
        d.out_draft_target_prob = ptr(verify.get("out_draft_target_prob"), "out_draft_target_prob",
                                      torch.float32, (B, K))
        ws = verify["workspace"]
        d.workspace = ptr(ws, "workspace")
        d.workspace_bytes = ws.numel() * ws.element_size()
        if build is not None:
            h = build["target_hidden"]
            H = h.shape[1]
            o = build["outputs"]
            d.start_pos = ptr(build["start_pos"], "start_pos", torch.int64, (B,))
            bt = build["block_table"]
            d.block_table = ptr(bt, "block_table", torch.int32)
            d.max_blocks_per_seq = bt.shape[1]
            d.block_size = int(build["block_size"])
            d.target_hidden = ptr(h, "target_hidden", None, (B * (K + 1), H))
            d.h_shared = ptr(build["h_shared"], "h_shared", h.dtype, (H,))
            d.hidden_dtype = _DTYPES[h.dtype]
            d.mask_token_id = int(build["mask_token_id"])
            d.H = H
            d.out_input_ids = ptr(o["input_ids"], "input_ids", torch.int32, (B * 2 * K,))
            d.out_positions = ptr(o["positions"], "positions", torch.int64, (B * 2 * K,))
            d.out_slot_mapping = ptr(o["slot_mapping"], "slot_mapping", torch.int64, (B * 2 * K,))
            d.out_hidden = ptr(o["hidden"], "hidden", h.dtype, (B * 2 * K, H))
            d.out_sample_rows = ptr(o.get("sample_rows"), "sample_rows", torch.int32, (B, K))
        if metrics is not None:
            d.metrics = ptr(metrics, "metrics", torch.int64)
        if device_error is not None:
            d.device_error = ptr(device_error, "device_error", torch.int32, (1,))
        self._keep = keep
        self._desc = d
        self._lib = lib
        self._dev = dev
        self._g = ctypes.c_void_p()
        _check(lib.sv_step_graph_create(ctypes.byref(d), ctypes.byref(self._g)),
               "sv_step_graph_create")

    def launch(self):
        _check(self._lib.sv_step_graph_launch(self._g, _stream(self._dev)), "sv_step_graph_launch")

    def close(self):
        if self._g:
            self._lib.sv_step_graph_destroy(self._g)
            self._g = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
