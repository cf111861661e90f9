"""Attention-score vision-token pruning on GB300: Python binding of libtsel.

Every function here marshals torch tensors into the C ABI of ``include/tsel.h``
(device pointers, sizes, the current CUDA stream) and calls the library; all
the work runs in the library's CUDA kernels. PyTorch only provides device
memory and streams. If ``libtsel.so`` has not been built the first call raises;
there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from ._build import LIB_PATH, build

__all__ = [
    "TselError", "load_library", "build",
    "tsel_importance_workspace_size", "tsel_importance", "tsel_importance_noalloc",
    "tsel_select_topk_workspace_size", "tsel_select_topk",
    "tsel_score_select_workspace_size", "tsel_score_select",
    "tsel_select_topk_hist_workspace_size", "tsel_select_topk_hist", "TSEL_SEL_STAGE_TOPK",
    "tsel_gather_compact_workspace_size", "tsel_gather_compact", "tsel_gather_compact_counted",
    "tsel_dynamic_budget", "TSEL_KEEP_FROM_DEVICE",
    "tsel_keep_count", "tsel_read_device_status", "tsel_clear_device_status",
    "tsel_importance_redo_pairs", "tsel_select_path_counts", "tsel_importance_one_launch",
    "tsel_status_string", "tsel_last_error", "tsel_probe_ex2",
    "tsel_rope_frequencies", "tsel_rope_table", "tsel_rope",
    "TselCache", "tsel_cache_new", "tsel_cache_workspace_size", "tsel_cache_write", "tsel_cache_read",
    "tsel_cache_compact", "tsel_cache_resize_workspace_size", "tsel_cache_resize", "tsel_cache_fork",
    "tsel_prefix_attention_workspace_size", "tsel_prefix_attention",
    "tsel_tree_attention_workspace_size", "tsel_tree_attention", "TSEL_DEV_PARENTS",
    "tsel_prompt_attention_workspace_size", "tsel_prompt_attention", "TSEL_ATT_CAUSAL",
    "TSEL_ROPE_ADJACENT", "TSEL_ROPE_INVERSE", "TSEL_ROPE_SECTIONED", "TSEL_ROPE_INTERLEAVED", "TSEL_ROPE_PER_AXIS",
    "TSEL_DEV_SEQLENS", "TSEL_DEV_REQUESTS", "TSEL_DEV_KEEP_IDX", "TSEL_DEV_TIMEOUT", "TSEL_DEV_NAN",
    "TSEL_DEV_PAGES", "TSEL_DEV_POSITIONS",
    "TSEL_IMP_LSE_PROVIDED", "TSEL_IMP_FP8_E4M3", "TSEL_IMP_SCORE_SUM", "TSEL_IMP_ROWREF_FIXED", "TSEL_IMP_ROWREF_MOVING", "TSEL_IMP_TWO_PASS", "TSEL_IMP_TEST_STALL", "TSEL_IMP_STAGE_PREP", "TSEL_IMP_STAGE_PASS1", "TSEL_IMP_STAGE_PASS2",
]

TSEL_OK = 0
TSEL_ERR_INVALID_VALUE = 1
TSEL_ERR_UNSUPPORTED = 2
TSEL_ERR_WORKSPACE = 3
TSEL_ERR_CUDA = 4
TSEL_ERR_DEVICE_CHECK = 5

TSEL_DEV_SEQLENS = 0x1
TSEL_DEV_REQUESTS = 0x2
TSEL_DEV_KEEP_IDX = 0x4
TSEL_DEV_TIMEOUT = 0x8
TSEL_DEV_NAN = 0x10
TSEL_DEV_PAGES = 0x20
TSEL_DEV_POSITIONS = 0x40
TSEL_DEV_PARENTS = 0x80

TSEL_KEEP_FROM_DEVICE = -1

TSEL_IMP_LSE_PROVIDED = 0x1
TSEL_IMP_FP8_E4M3 = 0x2
TSEL_IMP_SCORE_SUM = 0x4
TSEL_IMP_ROWREF_FIXED = 0x8
TSEL_IMP_ROWREF_MOVING = 0x20
TSEL_IMP_TWO_PASS = 0x40
TSEL_IMP_TEST_STALL = 0x10000
TSEL_IMP_STAGE_PREP = 0x100
TSEL_IMP_STAGE_PASS1 = 0x200
TSEL_IMP_STAGE_PASS2 = 0x400
TSEL_SEL_STAGE_TOPK = 0x800

TSEL_ROPE_ADJACENT = 0x1
TSEL_ROPE_INVERSE = 0x2
TSEL_ROPE_SECTIONED = 0
TSEL_ROPE_INTERLEAVED = 1
TSEL_ROPE_PER_AXIS = 2

TSEL_ATT_CAUSAL = 0x1

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}   # TSEL_BF16, _FP16, _FP32

_c_int, _c_i64, _c_size, _c_float, _c_uint, _p = (ctypes.c_int, ctypes.c_int64, ctypes.c_size_t,
                                                   ctypes.c_float, ctypes.c_uint, ctypes.c_void_p)

_SIGNATURES = {
    "tsel_importance_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "tsel_importance": (_c_int, [_p, _c_i64, _p, _c_i64, _p, _p, _c_int, _c_int, _c_int, _c_int,
                                 _c_int, _c_int, _c_int, _c_int, _c_float, _c_uint, _p, _p, _p,
                                 _c_size, _p]),
    "tsel_select_topk_workspace_size": (_c_size, [_c_int]),
    "tsel_select_topk": (_c_int, [_p, _c_int, _p, _c_int, _p, _c_int, _p, _p, _p, _c_size, _p]),
    "tsel_gather_compact_workspace_size": (_c_size, []),
    "tsel_gather_compact": (_c_int, [_p, _c_i64, _c_int, _c_int, _p, _c_int, _p, _c_int, _c_int,
                                     _p, _c_int, _p, _p, _p, _p, _p, _c_size, _p]),
    "tsel_gather_compact_counted": (_c_int, [_p, _c_i64, _c_int, _c_int, _p, _c_int, _p, _c_int,
                                             _c_int, _p, _p, _c_int, _p, _p, _p, _p, _p, _c_size,
                                             _p]),
    "tsel_dynamic_budget": (_c_int, [_p, _c_int, _p, _c_int, _c_int, _c_int, _c_int, _p, _p, _p,
                                     _c_size, _p]),
    "tsel_keep_count": (_c_int, [_c_int, _c_int]),
    "tsel_importance_one_launch": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                            _c_uint]),
    "tsel_read_device_status": (_c_int, [_p, ctypes.POINTER(ctypes.c_uint32), _p]),
    "tsel_clear_device_status": (_c_int, [_p, _p]),
    "tsel_importance_redo_pairs": (_c_int, [_p, ctypes.POINTER(ctypes.c_int32), _p]),
    "tsel_select_path_counts": (_c_int, [_p, ctypes.POINTER(ctypes.c_int32), _p]),
    "tsel_status_string": (ctypes.c_char_p, [_c_int]),
    "tsel_last_error": (ctypes.c_char_p, []),
    "tsel_probe_ex2": (_c_int, [_c_int, _c_int, _p, _p]),
    "tsel_score_select_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "tsel_score_select": (_c_int, [_p, _c_i64, _p, _c_i64, _p, _p, _c_int, _c_int, _c_int, _c_int,
                                   _c_int, _c_int, _c_int, _c_int, _c_float, _c_uint, _p, _p,
                                   _p, _c_int, _p, _c_int, _p, _p, _p, _c_size, _p]),
    "tsel_select_topk_hist_workspace_size": (_c_size, [_c_int]),
    "tsel_select_topk_hist": (_c_int, [_p, _c_int, _p, _c_int, _p, _c_int, _p, _p, _p, _c_size,
                                       _p]),
    "tsel_importance_noalloc": (_c_int, [_p, _c_i64, _p, _c_i64, _p, _p, _c_int, _c_int, _c_int,
                                         _c_int, _c_int, _c_int, _c_int, _c_int, _c_float, _p, _p,
                                         _p, _p]),
    "tsel_rope_frequencies": (_c_int, [ctypes.c_double, _p, _c_int, _c_int, _p, _p]),
    "tsel_rope_table": (_c_int, [_p, _p, _c_int, _p]),
    "tsel_cache_workspace_size": (_c_size, []),
    "tsel_rope": (_c_int, [_p, _c_i64, _p, _c_i64, _p, _c_int, _p, _c_int, _c_int, _c_int, _c_int,
                           _c_int, _c_int, _c_uint, _p, _c_i64, _p, _c_i64, _p, _c_size, _p]),
    "tsel_cache_write": (_c_int, [_p, _c_i64, _p, _c_i64, _p, _c_int, _p, _c_int, _p, _c_int,
                                  _c_int, _c_int, _c_int, _c_uint, _p, _p, _p, _p, _c_int, _c_int,
                                  _p, _c_size, _p]),
    "tsel_cache_read": (_c_int, [_p, _p, _p, _p, _c_int, _c_int, _p, _c_int, _c_int, _c_int,
                                 _c_int, _p, _c_i64, _p, _c_i64, _p, _c_size, _p]),
    "tsel_cache_compact": (_c_int, [_p, _p, _p, _p, _c_int, _c_int, _p, _c_i64, _c_int, _p, _c_i64, _c_int, _p, _p, _p, _p,
                                    _c_int, _c_int, _c_int, _c_int, _c_int, _p, _p, _c_size, _p]),
    "tsel_cache_resize_workspace_size": (_c_size, [_c_int] * 2),
    "tsel_cache_resize": (_c_int, [_p, _c_int, _c_int, _p, _c_i64, _c_int, _c_int, _p, _p, _p, _c_size, _p]),
    "tsel_cache_fork": (_c_int, [_p, _p, _p, _p, _c_int, _c_int, _c_int, _c_int, _p, _p, _c_i64, _c_int, _c_int, _p, _p, _p,
                                 _c_int, _p, _c_size, _p]),
    "tsel_prefix_attention_workspace_size": (_c_size, [_c_int] * 8),
    "tsel_prefix_attention": (_c_int, [_p, _c_i64, _p, _c_int, _c_int, _c_int, _p, _p, _p, _p,
                                       _c_int, _c_int, _p, _p, _c_int, _p, _c_i64, _p, _c_int,
                                       _c_int, _c_int, _c_int, _c_int, _c_float, _p, _c_i64, _p,
                                       _p, _c_size, _p]),
    "tsel_tree_attention_workspace_size": (_c_size, [_c_int] * 8),
    "tsel_tree_attention": (_c_int, [_p, _c_i64, _p, _c_int, _c_int, _c_int, _p, _p, _p, _p, _p,
                                     _c_int, _c_int, _p, _p, _c_int, _p, _c_i64, _p, _c_int,
                                     _c_int, _c_int, _c_int, _c_int, _c_float, _p, _c_i64, _p,
                                     _p, _c_size, _p]),
    "tsel_prompt_attention_workspace_size": (_c_size, [_c_int] * 7),
    "tsel_prompt_attention": (_c_int, [_p, _c_i64, _p, _c_i64, _p, _c_i64, _p, _p, _c_int, _c_int, _c_int, _c_int,
                                       _c_int, _c_int, _c_int, _c_int, _c_int, _c_float, _c_uint, _p, _c_i64, _p,
                                       _p, _c_size, _p]),
}

_lib: Optional[ctypes.CDLL] = None


class TselError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} [status {status}]")
        self.status = status


def load_library() -> ctypes.CDLL:
    """Loads the in-tree libtsel.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libtsel.so is not built at {LIB_PATH}: call "
                               "attention_score_vision_gb300.build() (nvcc, sm_103a) first")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(status: int) -> None:
    if status != TSEL_OK:
        lib = load_library()
        name = lib.tsel_status_string(status).decode()
        detail = lib.tsel_last_error().decode()
        raise TselError(status, f"{name}: {detail}")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream, device) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: torch.Tensor, dtype, name: str) -> None:
    if t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA {dtype} tensor")


def _new_workspace(nbytes: int, device) -> torch.Tensor:
    # zeroed so the device status word starts clear
    return torch.zeros(max(nbytes, 1024), dtype=torch.uint8, device=device)


def _check_qk(q: torch.Tensor, k: torch.Tensor, cu_seqlens_q: torch.Tensor,
              cu_seqlens_k: torch.Tensor, allow_fp8: bool):
    """Checks the importance inputs the C ABI cannot see (dtypes, devices, the
    [rows, heads, head_dim] layout the TMA maps are built from); returns
    (Tq, H, d, Tk, Hkv, fp8)."""
    fp8_types = (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8))
    fp8 = allow_fp8 and q.dtype in fp8_types and k.dtype in fp8_types
    if fp8:
        if not (q.is_cuda and k.is_cuda):
            raise TypeError("q and k must be CUDA tensors")
    else:
        _need(q, torch.bfloat16, "q")
        _need(k, torch.bfloat16, "k")
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q")
    _need(cu_seqlens_k, torch.int32, "cu_seqlens_k")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [rows, heads, head_dim] tensors")
    tq, H, d = q.shape
    tk, Hkv, dk = k.shape
    if dk != d:
        raise ValueError("q and k head_dim differ")
    for t, name in ((q, "q"), (k, "k")):
        if t.stride(2) != 1 or t.stride(1) != d:
            raise ValueError(f"{name} must have contiguous [heads, head_dim] rows")
    if cu_seqlens_q.numel() != cu_seqlens_k.numel():
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    for t in (k, cu_seqlens_q, cu_seqlens_k):
        if t.device != q.device:
            raise ValueError("q, k and cu_seqlens must be on the same device")
    return tq, H, d, tk, Hkv, fp8


# ---------------------------------------------------------------------------
# Importance
# ---------------------------------------------------------------------------

def tsel_importance_workspace_size(num_seg: int, total_q: int, total_k: int, num_heads: int) -> int:
    return int(load_library().tsel_importance_workspace_size(num_seg, total_q, total_k, num_heads))


def tsel_importance(q: torch.Tensor, k: torch.Tensor, cu_seqlens_q: torch.Tensor,
                    cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int, *,
                    softmax_scale: float = 0.0, flags: int = 0,
                    lse: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, want_lse: bool = True,
                    stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Mean attention received per key token; returns (scores [Tk], lse [H, Tq] or None).

    q: bf16 [Tq, H, d] (rows may be strided, head dim contiguous);
    k: bf16 [Tk, Hkv, d]; cu_seqlens_*: int32 [G+1] on the same device.
    With flags containing TSEL_IMP_LSE_PROVIDED, `lse` (fp32 [H, Tq], natural
    log) is an input and only the column pass runs. uint8 / float8_e4m3fn q and
    k are E4M3 inputs; softmax_scale then includes their dequantisation scales.
    """
    tq, H, d, tk, Hkv, fp8 = _check_qk(q, k, cu_seqlens_q, cu_seqlens_k, allow_fp8=True)
    if fp8:
        flags |= TSEL_IMP_FP8_E4M3   # E4M3 bytes; softmax_scale must carry the dequant scales
    G = cu_seqlens_k.numel() - 1
    dev = q.device
    if scores is None:
        scores = torch.empty(tk, dtype=torch.float32, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((H, tq), dtype=torch.float32, device=dev)
    nbytes = tsel_importance_workspace_size(G, tq, tk, H)
    if workspace is None:
        workspace = _new_workspace(nbytes, dev)
    lib = load_library()
    with torch.cuda.device(dev):   # the library works on the current device
        st = lib.tsel_importance(_ptr(q), q.stride(0), _ptr(k), k.stride(0), _ptr(cu_seqlens_q),
                                 _ptr(cu_seqlens_k), G, tq, tk, int(max_seqlen_q),
                                 int(max_seqlen_k), H, Hkv, d, float(softmax_scale), int(flags),
                                 _ptr(lse), _ptr(scores), _ptr(workspace), workspace.numel(),
                                 _stream(stream, dev))
    _check(st)
    return scores, lse


def tsel_importance_noalloc(q: torch.Tensor, k: torch.Tensor, cu_seqlens_q: torch.Tensor,
                            cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int, *,
                            softmax_scale: float = 0.0, lse: Optional[torch.Tensor] = None,
                            scores: Optional[torch.Tensor] = None,
                            device_status: Optional[torch.Tensor] = None, want_lse: bool = True,
                            stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """tsel_importance with the library's static scratch array instead of a
    workspace (for callers that cannot allocate device memory). Output
    tensors passed in are used as they are; calls on one device must not
    overlap on the GPU."""
    tq, H, d, tk, Hkv, _ = _check_qk(q, k, cu_seqlens_q, cu_seqlens_k, allow_fp8=False)
    if device_status is not None:
        _need(device_status, torch.int32, "device_status")
        if device_status.device != q.device:
            raise ValueError("device_status must be on q's device")
    G = cu_seqlens_k.numel() - 1
    dev = q.device
    if scores is None:
        scores = torch.empty(tk, dtype=torch.float32, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((H, tq), dtype=torch.float32, device=dev)
    # the static scratch array is looked up on the current device: make it q's
    with torch.cuda.device(dev):
        st = load_library().tsel_importance_noalloc(
            _ptr(q), q.stride(0), _ptr(k), k.stride(0), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), G,
            tq, tk, int(max_seqlen_q), int(max_seqlen_k), H, Hkv, d, float(softmax_scale),
            _ptr(lse), _ptr(scores), _ptr(device_status), _stream(stream, dev))
    _check(st)
    return scores, lse


def tsel_score_select_workspace_size(num_seg: int, total_q: int, total_k: int, num_heads: int,
                                     num_req: int) -> int:
    return int(load_library().tsel_score_select_workspace_size(num_seg, total_q, total_k,
                                                                num_heads, num_req))


def tsel_score_select(q: torch.Tensor, k: torch.Tensor, cu_seqlens_q: torch.Tensor,
                      cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int,
                      req_tok_offsets: torch.Tensor, keep_per_req: torch.Tensor, total_keep: int,
                      *, softmax_scale: float = 0.0, flags: int = 0,
                      lse: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None,
                      keep_idx: Optional[torch.Tensor] = None,
                      cu_keep: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, want_lse: bool = True,
                      stream=None):
    """tsel_importance + tsel_select_topk in one call (the top-B starts from the
    score histograms the column pass builds); returns (scores, lse, keep_idx, cu_keep)."""
    tq, H, d, tk, Hkv, fp8 = _check_qk(q, k, cu_seqlens_q, cu_seqlens_k, allow_fp8=True)
    if fp8:
        flags |= TSEL_IMP_FP8_E4M3
    _need(req_tok_offsets, torch.int32, "req_tok_offsets")
    _need(keep_per_req, torch.int32, "keep_per_req")
    G = cu_seqlens_k.numel() - 1
    R = keep_per_req.numel()
    dev = q.device
    if scores is None:
        scores = torch.empty(tk, dtype=torch.float32, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((H, tq), dtype=torch.float32, device=dev)
    if keep_idx is None:
        cap = tk if int(total_keep) == TSEL_KEEP_FROM_DEVICE else int(total_keep)
        keep_idx = torch.empty(cap, dtype=torch.int32, device=dev)
    if cu_keep is None:
        cu_keep = torch.empty(R + 1, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = _new_workspace(tsel_score_select_workspace_size(G, tq, tk, H, R), dev)
    with torch.cuda.device(dev):
        st = load_library().tsel_score_select(
            _ptr(q), q.stride(0), _ptr(k), k.stride(0), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), G,
            tq, tk, int(max_seqlen_q), int(max_seqlen_k), H, Hkv, d, float(softmax_scale),
            int(flags), _ptr(lse), _ptr(scores), _ptr(req_tok_offsets), R, _ptr(keep_per_req),
            int(total_keep), _ptr(keep_idx), _ptr(cu_keep), _ptr(workspace), workspace.numel(),
            _stream(stream, dev))
    _check(st)
    return scores, lse, keep_idx, cu_keep


# ---------------------------------------------------------------------------
# Top-B
# ---------------------------------------------------------------------------

def tsel_select_topk_workspace_size(num_req: int) -> int:
    return int(load_library().tsel_select_topk_workspace_size(num_req))


def tsel_select_topk(scores: torch.Tensor, req_tok_offsets: torch.Tensor,
                     keep_per_req: torch.Tensor, total_keep: int, *,
                     keep_idx: Optional[torch.Tensor] = None, cu_keep: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Pooled top-B per request; returns (keep_idx int32 [total_keep], cu_keep int32 [R+1]).

    total_keep = TSEL_KEEP_FROM_DEVICE takes budgets computed on the device
    (tsel_dynamic_budget): keep_idx then has room for every token and
    cu_keep[R] holds the kept count."""
    _need(scores, torch.float32, "scores")
    _need(req_tok_offsets, torch.int32, "req_tok_offsets")
    _need(keep_per_req, torch.int32, "keep_per_req")
    R = keep_per_req.numel()
    dev = scores.device
    if keep_idx is None:
        cap = scores.numel() if int(total_keep) == TSEL_KEEP_FROM_DEVICE else int(total_keep)
        keep_idx = torch.empty(cap, dtype=torch.int32, device=dev)
    if cu_keep is None:
        cu_keep = torch.empty(R + 1, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = _new_workspace(tsel_select_topk_workspace_size(R), dev)
    st = load_library().tsel_select_topk(_ptr(scores), scores.numel(), _ptr(req_tok_offsets), R,
                                         _ptr(keep_per_req), int(total_keep), _ptr(keep_idx),
                                         _ptr(cu_keep), _ptr(workspace), workspace.numel(),
                                         _stream(stream, dev))
    _check(st)
    return keep_idx, cu_keep


def tsel_select_topk_hist_workspace_size(num_req: int) -> int:
    return int(load_library().tsel_select_topk_hist_workspace_size(num_req))


def tsel_select_topk_hist(scores: torch.Tensor, req_tok_offsets: torch.Tensor,
                          keep_per_req: torch.Tensor, total_keep: int, *,
                          keep_idx: Optional[torch.Tensor] = None,
                          cu_keep: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None,
                          stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """tsel_select_topk started from per-request score histograms (built by one
    extra launch); same results. Returns (keep_idx, cu_keep)."""
    _need(scores, torch.float32, "scores")
    _need(req_tok_offsets, torch.int32, "req_tok_offsets")
    _need(keep_per_req, torch.int32, "keep_per_req")
    R = keep_per_req.numel()
    dev = scores.device
    if keep_idx is None:
        cap = scores.numel() if int(total_keep) == TSEL_KEEP_FROM_DEVICE else int(total_keep)
        keep_idx = torch.empty(cap, dtype=torch.int32, device=dev)
    if cu_keep is None:
        cu_keep = torch.empty(R + 1, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = _new_workspace(tsel_select_topk_hist_workspace_size(R), dev)
    with torch.cuda.device(dev):
        st = load_library().tsel_select_topk_hist(
            _ptr(scores), scores.numel(), _ptr(req_tok_offsets), R, _ptr(keep_per_req),
            int(total_keep), _ptr(keep_idx), _ptr(cu_keep), _ptr(workspace), workspace.numel(),
            _stream(stream, dev))
    _check(st)
    return keep_idx, cu_keep


def tsel_dynamic_budget(scores: torch.Tensor, req_tok_offsets: torch.Tensor, mass_permille: int,
                        min_permille: int = 0, max_permille: int = 1000, *,
                        keep_per_req: Optional[torch.Tensor] = None,
                        total_keep: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None,
                        stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-request budgets from the scores (fewest top tokens holding mass_permille of
    the request's score quanta, bounded); returns (keep_per_req int32 [R], total int32 [1])."""
    _need(scores, torch.float32, "scores")
    _need(req_tok_offsets, torch.int32, "req_tok_offsets")
    R = req_tok_offsets.numel() - 1
    dev = scores.device
    if keep_per_req is None:
        keep_per_req = torch.empty(max(R, 0), dtype=torch.int32, device=dev)
    if total_keep is None:
        total_keep = torch.empty(1, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = _new_workspace(tsel_select_topk_workspace_size(R), dev)
    st = load_library().tsel_dynamic_budget(_ptr(scores), scores.numel(), _ptr(req_tok_offsets), R,
                                            int(mass_permille), int(min_permille), int(max_permille),
                                            _ptr(keep_per_req), _ptr(total_keep), _ptr(workspace),
                                            workspace.numel(), _stream(stream, dev))
    _check(st)
    return keep_per_req, total_keep


# ---------------------------------------------------------------------------
# Compaction
# ---------------------------------------------------------------------------

def tsel_gather_compact_workspace_size() -> int:
    return int(load_library().tsel_gather_compact_workspace_size())


def tsel_gather_compact(hidden: torch.Tensor, pos: Optional[torch.Tensor], cu_seqlens_k: torch.Tensor,
                        keep_idx: torch.Tensor, *, out_hidden: Optional[torch.Tensor] = None,
                        out_pos: Optional[torch.Tensor] = None, out_img_id: Optional[torch.Tensor] = None,
                        out_cu_seqlens: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None):
    """Compacts kept rows; returns (out_hidden, out_pos, out_img_id, out_cu_seqlens)."""
    _need(cu_seqlens_k, torch.int32, "cu_seqlens_k")
    _need(keep_idx, torch.int32, "keep_idx")
    if hidden.dim() != 2 or hidden.stride(1) != 1 or not hidden.is_cuda:
        raise ValueError("hidden must be a CUDA [T, D] tensor with contiguous rows")
    tk, D = hidden.shape
    K = keep_idx.numel()
    G = cu_seqlens_k.numel() - 1
    dev = hidden.device
    P = 0 if pos is None else pos.shape[1]
    if pos is not None:
        _need(pos, torch.int32, "pos")
        if not pos.is_contiguous() or pos.shape[0] != tk:
            raise ValueError("pos must be a contiguous int32 [T, P] tensor")
    if out_hidden is None:
        out_hidden = torch.empty((K, D), dtype=hidden.dtype, device=dev)
    if out_pos is None and P > 0:
        out_pos = torch.empty((K, P), dtype=torch.int32, device=dev)
    if out_img_id is None:
        out_img_id = torch.empty(K, dtype=torch.int32, device=dev)
    if out_cu_seqlens is None:
        out_cu_seqlens = torch.empty(G + 1, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = _new_workspace(tsel_gather_compact_workspace_size(), dev)
    st = load_library().tsel_gather_compact(
        _ptr(hidden), hidden.stride(0), D, hidden.element_size(), _ptr(pos), P, _ptr(cu_seqlens_k),
        G, tk, _ptr(keep_idx), K, _ptr(out_hidden), _ptr(out_pos), _ptr(out_img_id),
        _ptr(out_cu_seqlens), _ptr(workspace), workspace.numel(), _stream(stream, dev))
    _check(st)
    return out_hidden, out_pos, out_img_id, out_cu_seqlens


def tsel_gather_compact_counted(hidden: torch.Tensor, pos: Optional[torch.Tensor],
                                cu_seqlens_k: torch.Tensor, keep_idx: torch.Tensor,
                                num_kept: torch.Tensor, max_kept: int, *,
                                out_hidden: Optional[torch.Tensor] = None,
                                out_pos: Optional[torch.Tensor] = None,
                                out_img_id: Optional[torch.Tensor] = None,
                                out_cu_seqlens: Optional[torch.Tensor] = None,
                                workspace: Optional[torch.Tensor] = None, stream=None):
    """tsel_gather_compact with the kept count read on the device (num_kept: int32
    device scalar, e.g. cu_keep[R:]); outputs have room for max_kept rows, of which
    the first *num_kept are written."""
    _need(cu_seqlens_k, torch.int32, "cu_seqlens_k")
    _need(keep_idx, torch.int32, "keep_idx")
    _need(num_kept, torch.int32, "num_kept")
    if hidden.dim() != 2 or hidden.stride(1) != 1 or not hidden.is_cuda:
        raise ValueError("hidden must be a CUDA [T, D] tensor with contiguous rows")
    tk, D = hidden.shape
    K = int(max_kept)
    if keep_idx.numel() < K:
        raise ValueError("keep_idx has fewer than max_kept entries")
    G = cu_seqlens_k.numel() - 1
    dev = hidden.device
    P = 0 if pos is None else pos.shape[1]
    if pos is not None:
        _need(pos, torch.int32, "pos")
        if not pos.is_contiguous() or pos.shape[0] != tk:
            raise ValueError("pos must be a contiguous int32 [T, P] tensor")
    if out_hidden is None:
        out_hidden = torch.empty((K, D), dtype=hidden.dtype, device=dev)
    if out_pos is None and P > 0:
        out_pos = torch.empty((K, P), dtype=torch.int32, device=dev)
    if out_img_id is None:
        out_img_id = torch.empty(K, dtype=torch.int32, device=dev)
    if out_cu_seqlens is None:
        out_cu_seqlens = torch.empty(G + 1, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = _new_workspace(tsel_gather_compact_workspace_size(), dev)
    st = load_library().tsel_gather_compact_counted(
        _ptr(hidden), hidden.stride(0), D, hidden.element_size(), _ptr(pos), P, _ptr(cu_seqlens_k),
        G, tk, _ptr(keep_idx), _ptr(num_kept), K, _ptr(out_hidden), _ptr(out_pos), _ptr(out_img_id),
        _ptr(out_cu_seqlens), _ptr(workspace), workspace.numel(), _stream(stream, dev))
    _check(st)
    return out_hidden, out_pos, out_img_id, out_cu_seqlens


# ---------------------------------------------------------------------------
# Rotary positions with several axes
# ---------------------------------------------------------------------------

# The calls below are made once per layer and decoding step, where the host's
# share counts. Every question to a tensor costs a tenth of a microsecond or two,
# so the checks ask few of them and compare devices by index, and the device is
# switched and the stream looked up in the cheapest way there is.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_U8, _I32, _I64, _F32 = torch.uint8, torch.int32, torch.int64, torch.float32


def _call(fn, index: int, stream, *args) -> None:
    """fn(*args, stream) on device `index` (the library works on the current device)."""
    if stream is None and _raw_stream is not None:
        handle = _raw_stream(index)
    else:
        handle = _stream(stream, index)
    if torch.cuda.current_device() == index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            st = fn(*args, handle)
    if st != TSEL_OK:
        _check(st)


def _rows(t: torch.Tensor, name: str, index: int, dtype, shape=None) -> int:
    """Checks a [rows, heads, head_dim] tensor; returns its row stride (0: dense)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    if t.is_contiguous():
        return 0
    n, h, d = t.shape
    if (d > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != d):
        raise ValueError(f"{name} must have contiguous [heads, head_dim] rows")
    if n <= 1:
        return 0
    if t.stride(0) <= 0:   # expanded: 0 would mean dense
        raise ValueError(f"{name} must not be an expanded tensor")
    return t.stride(0)


def _first(t: torch.Tensor, name: str):
    """(shape, dtype, device index) of the tensor that the others have to match."""
    shape, dtype, index = t.shape, t.dtype, t.get_device()
    if index < 0 or dtype not in _DTYPES:
        raise TypeError(f"{name} must be a CUDA bf16, fp16 or fp32 tensor")
    if len(shape) != 3:
        raise ValueError(f"{name} must be a [rows, heads, head_dim] tensor")
    return shape, dtype, index


def _sizes(bits: int) -> None:
    """Refuses sizes (or-ed together) that a C int does not hold: a foreign call
    takes their low 32 bits."""
    if bits >> 31:
        raise ValueError("a size is negative or past 2^31 - 1")


def _vector(t: torch.Tensor, dtype, name: str, index: int, numel: Optional[int] = None) -> int:
    """Checks a dense tensor; returns its pointer."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be a CUDA {dtype} tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} entries")
    return t.data_ptr()


def _rope_args(pos, table, total: int, index: int):
    """(pos pointer, pos_dim, table pointer, pairs) of a rotation."""
    if table is None:
        return None, 0, None, 0
    if pos is None:
        raise ValueError("a rope table needs positions")
    pos_p = _vector(pos, _I32, "pos", index)
    shape = pos.shape
    if len(shape) != 2 or shape[0] != total:
        raise ValueError("pos must be an int32 [tokens, axes] tensor")
    return pos_p, shape[1], _vector(table, _I64, "table", index), table.numel()


def _new(stream, make, *args, device, **kw):
    """make(*args, device=device, **kw) with memory of `stream`: what a call
    allocates is cleared, used and freed in the order of the stream it runs on."""
    if stream is None:
        return make(*args, device=device, **kw)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return make(*args, device=device, **kw)


def _like(t: torch.Tensor, stream) -> torch.Tensor:
    """A dense tensor of t's shape and type."""
    if stream is None and t.is_contiguous():
        return torch.empty_like(t)   # the cheapest allocation there is
    return _new(stream, torch.empty, t.shape, dtype=t.dtype, device=t.device)


def _written(*outs) -> None:
    """Tells autograd that a call writes into tensors it was given (or None)."""
    given = [t for t in outs if t is not None]
    if any(t.requires_grad for t in given) and torch.is_grad_enabled():
        raise ValueError("an output that requires a gradient cannot be written where autograd records")
    torch.autograd.graph.increment_version(given)


def _workspace(workspace: Optional[torch.Tensor], nbytes: int, index: int, stream) -> torch.Tensor:
    if workspace is None:
        return _new(stream, _new_workspace, nbytes, device=torch.device("cuda", index))
    if workspace.get_device() != index:
        raise ValueError(f"workspace must be on cuda:{index}")
    if not workspace.is_contiguous():   # its numel() would not be the bytes behind its pointer
        raise ValueError("workspace must be contiguous")
    return workspace


def _int32s(values: list, name: str) -> list:
    if any(not -2 ** 31 <= x < 2 ** 31 for x in values):   # ctypes keeps the low 32 bits
        raise ValueError(f"{name} past 32 bits")
    return values


def tsel_rope_frequencies(base: float, sections: Sequence[int],
                          layout: int = TSEL_ROPE_SECTIONED) -> Tuple[list, list]:
    """Frequencies (radians per position step) and axes of the rotated pairs, axis a
    having sections[a] of them; see tsel_rope_frequencies in include/tsel.h."""
    sections = [int(x) for x in sections]
    n, total = len(sections), sum(sections)
    sec = (ctypes.c_int32 * max(n, 1))(*_int32s(sections, "sections"))
    freq, axis = (ctypes.c_double * 128)(), (ctypes.c_int32 * 128)()   # the library takes no more pairs
    _check(load_library().tsel_rope_frequencies(float(base), sec, n, int(layout), freq, axis))
    return list(freq)[:total], list(axis)[:total]


def tsel_rope_table(inv_freq: Sequence[float], axis: Sequence[int], device="cuda") -> torch.Tensor:
    """The device table (int64 [pairs]) of a rotation, built once from its
    frequencies and axes (tsel_rope_frequencies, or any others)."""
    n = len(inv_freq)
    if len(axis) != n:
        raise ValueError("inv_freq and axis must have the same length")
    freq = (ctypes.c_double * max(n, 1))(*[float(x) for x in inv_freq])
    ax = (ctypes.c_int32 * max(n, 1))(*_int32s([int(x) for x in axis], "axis"))
    table = torch.empty(n, dtype=torch.int64)
    _check(load_library().tsel_rope_table(freq, ax, n, _ptr(table) if n else None))
    return table.to(device)


class _Rotation(torch.autograd.Function):
    """tsel_rope on the tape: the gradient of a rotation is the rotation back."""

    @staticmethod
    def forward(ctx, q, k, pos, table, flags, workspace, stream):
        q_out, k_out = tsel_rope(q, k, pos, table, flags=flags, workspace=workspace, stream=stream)
        ctx.save_for_backward(pos, table)
        ctx.flags, ctx.workspace = flags ^ TSEL_ROPE_INVERSE, workspace
        ctx.set_materialize_grads(False)
        # each output depends on its own input alone
        ctx.mark_non_differentiable(*[t for t, need in zip((q_out, k_out), ctx.needs_input_grad) if t is not None and not need])
        return q_out, k_out

    @staticmethod
    def backward(ctx, *grads):
        pos, table = ctx.saved_tensors
        turned = [None, None]
        # a gradient may come expanded or transposed
        given = [i for i in (0, 1) if ctx.needs_input_grad[i] and grads[i] is not None]
        if given:
            g = [grads[i].contiguous() for i in given] + [None]
            back = tsel_rope(g[0], g[1], pos, table, flags=ctx.flags, workspace=ctx.workspace)
            for i, t in zip(given, back):
                turned[i] = t
        return (*turned, None, None, None, None, None)


def tsel_rope(q: torch.Tensor, k: Optional[torch.Tensor], pos: torch.Tensor, table: torch.Tensor, *,
              flags: int = 0, q_out: Optional[torch.Tensor] = None,
              k_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Rotates q [T, H, d] and k [T, Hkv, d] (or None) by positions pos int32 [T, axes];
    returns (q_out, k_out), which may be q and k themselves. With
    TSEL_ROPE_INVERSE it turns gradients of the outputs into those of the inputs.

    Where autograd records (grad mode, and q or k requires a gradient) the
    outputs carry gradients; they are then new tensors, q_out and k_out are
    refused. The backward pass runs on the stream that was current in the forward
    call; to capture it into a graph, let no eager graph of the same leaves live."""
    shape, dtype, index = _first(q, "q")
    qs = _rows(q, "q", index, dtype)
    total, H, d = shape
    Hkv = ks = kos = 0
    if k is not None:
        ks = _rows(k, "k", index, dtype)
        k_shape = k.shape
        if len(k_shape) != 3 or k_shape[0] != total or k_shape[2] != d:
            raise ValueError("q and k must have the same rows and head_dim")
        Hkv = k_shape[1]
    elif k_out is not None:
        raise ValueError("k_out without k")
    pos_p, pos_dim, table_p, pairs = _rope_args(pos, table, total, index)
    _sizes(total | H | Hkv | d | pos_dim | pairs)
    qos = 0 if q_out is None else _rows(q_out, "q_out", index, dtype, shape)
    if k_out is not None:
        kos = _rows(k_out, "k_out", index, dtype, k_shape)
    if torch.is_grad_enabled() and (q.requires_grad or (k is not None and k.requires_grad)):
        if q_out is not None or k_out is not None:
            raise ValueError("q_out and k_out cannot be written where autograd records q or k")
        return _Rotation.apply(q, k, pos, table, flags, workspace, stream)
    if q_out is not None or k_out is not None:
        _written(q_out, k_out)
    workspace = _workspace(workspace, 1024, index, stream)
    if q_out is None:
        q_out = _like(q, stream)
    if k is not None and k_out is None:
        k_out = _like(k, stream)
    _call(load_library().tsel_rope, index, stream, q.data_ptr(), qs, _ptr(k), ks, pos_p, pos_dim,
          table_p, pairs, total, H, Hkv, d, _DTYPES[dtype], flags, q_out.data_ptr(), qos,
          _ptr(k_out), kos, workspace.data_ptr(), workspace.numel())
    return q_out, k_out


# ---------------------------------------------------------------------------
# Quantised paged cache
# ---------------------------------------------------------------------------

class TselCache(NamedTuple):
    """A paged cache: E4M3 codes uint8 [pages, Hkv, page_size, d] and scale
    exponents uint8 [pages, Hkv, page_size] of K and V."""
    k_pages: torch.Tensor
    v_pages: torch.Tensor
    k_exps: torch.Tensor
    v_exps: torch.Tensor


def tsel_cache_new(num_pages: int, page_size: int, num_kv_heads: int, head_dim: int,
                   device="cuda") -> TselCache:
    """A zeroed cache."""
    shape = (int(num_pages), int(num_kv_heads), int(page_size))
    codes = [torch.zeros(shape + (int(head_dim),), dtype=torch.uint8, device=device) for _ in range(2)]
    return TselCache(*codes, *[torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2)])


def _cache_args(cache: TselCache, index: int):
    """(pointers and sizes of the C calls, Hkv, d) of a cache."""
    kp, vp, ke, ve = cache
    shape = kp.shape
    if len(shape) != 4:
        raise ValueError("k_pages must be a uint8 [pages, heads, page_size, head_dim] tensor")
    pages, heads, page_size, d = shape
    if vp.shape != shape or ke.shape != shape[:3] or ve.shape != shape[:3]:
        raise ValueError("the cache's tensors do not match one another")
    return (_vector(kp, _U8, "k_pages", index), _vector(vp, _U8, "v_pages", index),
            _vector(ke, _U8, "k_exps", index), _vector(ve, _U8, "v_exps", index), pages, page_size), heads, d


def tsel_cache_workspace_size() -> int:
    return int(load_library().tsel_cache_workspace_size())


def tsel_cache_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: TselCache, *,
                     pos: Optional[torch.Tensor] = None, table: Optional[torch.Tensor] = None,
                     flags: int = 0, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantises k and v [T, Hkv, d] into the cache's slots (int32 [T], negative:
    skipped); with a rope table and positions k is rotated on its way."""
    shape, dtype, index = _first(k, "k")
    ks = _rows(k, "k", index, dtype)
    vs = _rows(v, "v", index, dtype, shape)
    total, Hkv, d = shape
    cache_p, ch, cd = _cache_args(cache, index)
    if ch != Hkv or cd != d:
        raise ValueError("k and v do not match the cache's heads and head_dim")
    slots_p = _vector(slots, _I32, "slots", index, total)
    pos_p, pos_dim, table_p, pairs = _rope_args(pos, table, total, index)
    _sizes(total | Hkv | d | pos_dim | pairs | cache_p[4] | cache_p[5])
    workspace = _workspace(workspace, 1024, index, stream)
    _call(load_library().tsel_cache_write, index, stream, k.data_ptr(), ks, v.data_ptr(), vs, pos_p,
          pos_dim, table_p, pairs, slots_p, total, Hkv, d, _DTYPES[dtype], flags, *cache_p,
          workspace.data_ptr(), workspace.numel())


def tsel_cache_read(cache: TselCache, slots: torch.Tensor, *, dtype=torch.bfloat16,
                    k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Reads slots (int32 [T], negative: zeros) back as k and v [T, Hkv, d] of dtype."""
    index = cache.k_pages.get_device()
    if index < 0:
        raise TypeError("the cache must be on a CUDA device")
    cache_p, Hkv, d = _cache_args(cache, index)
    slots_p = _vector(slots, _I32, "slots", index)
    if dtype not in _DTYPES:
        raise TypeError("dtype must be bf16, fp16 or fp32")
    shape = (slots.numel(), Hkv, d)
    _sizes(shape[0] | Hkv | d | cache_p[4] | cache_p[5])
    kos = 0 if k_out is None else _rows(k_out, "k_out", index, dtype, shape)
    vos = 0 if v_out is None else _rows(v_out, "v_out", index, dtype, shape)
    if k_out is not None or v_out is not None:
        _written(k_out, v_out)
    workspace = _workspace(workspace, 1024, index, stream)
    if k_out is None:
        k_out = _new(stream, torch.empty, shape, dtype=dtype, device=slots.device)
    if v_out is None:
        v_out = _like(k_out, stream)
    _call(load_library().tsel_cache_read, index, stream, *cache_p, slots_p, shape[0], Hkv, d,
          _DTYPES[dtype], k_out.data_ptr(), kos, v_out.data_ptr(), vos, workspace.data_ptr(),
          workspace.numel())
    return k_out, v_out


# ---------------------------------------------------------------------------
# Pages of the cache
# ---------------------------------------------------------------------------

def _table(t: torch.Tensor, name: str, index: int, rows: Optional[int] = None):
    """Checks a page table, int32 [rows, pages] with contiguous rows; returns
    (pointer, row stride, rows, pages)."""
    if t.dtype is not _I32:
        raise TypeError(f"{name} must be a CUDA torch.int32 tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}")
    shape = t.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be an int32 [requests, pages] tensor with contiguous rows")
    stride = t.stride(0) if shape[0] > 1 else shape[1]
    if stride < shape[1]:
        raise ValueError(f"{name} rows must not overlap")
    return t.data_ptr(), stride, shape[0], shape[1]


def tsel_cache_compact(cache: TselCache, page_table: torch.Tensor, keep_idx: torch.Tensor, cu_keep: torch.Tensor,
                       max_keep: int, *, starts: Optional[torch.Tensor] = None, bases: Optional[torch.Tensor] = None,
                       dst_table: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Moves the cached rows of kept tokens together; returns the new lengths int32 [R],
    -1 for a request that is refused.

    Token k of request r's kept ones goes from position starts[r] + keep_idx[cu_keep[r] + k]
    - bases[r] of its pages (page_table int32 [R, pages]) to position starts[r] + k of
    the pages of dst_table, or of its own (None: in place). keep_idx ascends in each
    request, e.g. accepted nodes of a drafted tree with starts = the length before it, or
    tsel_select_topk's tokens with bases = its request offsets."""
    index = cache.k_pages.get_device()
    if index < 0:
        raise TypeError("the cache must be on a CUDA device")
    cache_p, Hkv, d = _cache_args(cache, index)
    R = cu_keep.numel() - 1
    if R < 0:
        raise ValueError("cu_keep must have at least one entry")
    table_p, table_s, _, pages = _table(page_table, "page_table", index, R)
    to_p, to_s, to_pages = None, 0, 0
    if dst_table is not None:
        to_p, to_s, _, to_pages = _table(dst_table, "dst_table", index, R)
        if to_p == table_p:
            raise ValueError("dst_table is page_table: give None to move in place")
    keep_p = _vector(keep_idx, _I32, "keep_idx", index)
    cu_p = _vector(cu_keep, _I32, "cu_keep", index)
    starts_p = None if starts is None else _vector(starts, _I32, "starts", index, R)
    bases_p = None if bases is None else _vector(bases, _I32, "bases", index, R)
    total, most = keep_idx.numel(), int(max_keep)
    _sizes(R | total | most | pages | to_pages | Hkv | d | cache_p[4] | cache_p[5])
    if new_lens is not None:
        if _vector(new_lens, _I32, "new_lens", index, R) == starts_p and R:
            raise ValueError("new_lens must not be starts")
        _written(new_lens)
    workspace = _workspace(workspace, 1024, index, stream)
    if new_lens is None:
        new_lens = _new(stream, torch.empty, R, dtype=_I32, device=cu_keep.device)
    _call(load_library().tsel_cache_compact, index, stream, *cache_p, table_p, table_s, pages, to_p, to_s, to_pages,
          starts_p, bases_p, keep_p, cu_p, R, total, most, Hkv, d, new_lens.data_ptr(), workspace.data_ptr(),
          workspace.numel())
    return new_lens


def tsel_cache_resize_workspace_size(num_rows: int, pages_per_row: int) -> int:
    """Bytes of workspace of tsel_cache_resize and tsel_cache_fork."""
    sizes = [int(num_rows), int(pages_per_row)]
    if any(n >> 31 for n in sizes):   # negative, or more than a C int holds
        return 0
    return int(load_library().tsel_cache_resize_workspace_size(*sizes))


def tsel_cache_resize(refs: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor, new_lens: torch.Tensor,
                      page_size: int, *, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gives pages to the rows of page_table (int32 [rows, pages]) that grow from lens to
    new_lens (int32 [rows], negative: left alone) and takes them back from those that
    shrink. refs int32 [num_pages] counts the rows that hold a page; the lowest free
    pages go to rows in order. A row that ends inside a page which others hold too
    (after tsel_cache_fork) does not grow from there; a fork of it does. page_table, refs
    and lens are written."""
    index = refs.get_device()
    if index < 0:
        raise TypeError("refs must be a CUDA torch.int32 tensor")
    refs_p = _vector(refs, _I32, "refs", index)
    table_p, stride, rows, pages = _table(page_table, "page_table", index)
    lens_p = _vector(lens, _I32, "lens", index, rows)
    new_p = _vector(new_lens, _I32, "new_lens", index, rows)
    num_pages, page_size = refs.numel(), int(page_size)
    _sizes(num_pages | rows | pages | page_size)
    nbytes = 0 if workspace is not None else tsel_cache_resize_workspace_size(rows, pages)
    workspace = _workspace(workspace, nbytes, index, stream)
    _call(load_library().tsel_cache_resize, index, stream, refs_p, num_pages, page_size, table_p, stride, rows, pages,
          lens_p, new_p, workspace.data_ptr(), workspace.numel())


def tsel_cache_fork(cache: TselCache, refs: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
                    parents: torch.Tensor, children: torch.Tensor, *, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    """Rows children[i] of page_table start from the cached tokens of rows parents[i]
    (int32 [n], children ascending and of length 0): whole pages are shared, the
    rows of a last page that is not full are copied into a free one. cache, refs (int32
    [num_pages]), page_table and lens are written."""
    index = cache.k_pages.get_device()
    if index < 0:
        raise TypeError("the cache must be on a CUDA device")
    cache_p, Hkv, d = _cache_args(cache, index)
    refs_p = _vector(refs, _I32, "refs", index, cache_p[4])
    table_p, stride, rows, pages = _table(page_table, "page_table", index)
    lens_p = _vector(lens, _I32, "lens", index, rows)
    parents_p = _vector(parents, _I32, "parents", index)
    n = parents.numel()
    children_p = _vector(children, _I32, "children", index, n)
    _sizes(n | rows | pages | Hkv | d | cache_p[4] | cache_p[5])
    nbytes = 0 if workspace is not None else tsel_cache_resize_workspace_size(rows, pages)
    workspace = _workspace(workspace, nbytes, index, stream)
    _call(load_library().tsel_cache_fork, index, stream, *cache_p, Hkv, d, refs_p, table_p, stride, rows, pages, lens_p,
          parents_p, children_p, n, workspace.data_ptr(), workspace.numel())


# ---------------------------------------------------------------------------
# Attention over a shared prefix
# ---------------------------------------------------------------------------

def tsel_prefix_attention_workspace_size(num_req: int, total_q: int, max_seqlen_q: int,
                                         num_heads: int, num_kv_heads: int, head_dim: int,
                                         max_prefix_len: int, max_suffix_len: int) -> int:
    sizes = [int(n) for n in (num_req, total_q, max_seqlen_q, num_heads, num_kv_heads, head_dim, max_prefix_len, max_suffix_len)]
    if any(n >> 31 for n in sizes):   # negative, or more than a C int holds
        return 0
    return int(load_library().tsel_prefix_attention_workspace_size(*sizes))


def tsel_prefix_attention(q: torch.Tensor, cu_seqlens_q: torch.Tensor, max_seqlen_q: int,
                          cache: TselCache, prefix_pages: Optional[torch.Tensor],
                          prefix_len: Optional[torch.Tensor], max_prefix_len: int,
                          page_table: Optional[torch.Tensor], suffix_lens: Optional[torch.Tensor],
                          max_suffix_len: int, *, softmax_scale: float = 0.0,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          want_lse: bool = True, workspace: Optional[torch.Tensor] = None,
                          stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention of a batch over a prefix that all requests share and each one's own
    suffix, both in the cache; returns (out [Tq, H, d], lse fp32 [H, Tq] or None).

    q bf16 or fp16 [Tq, H, d]; cu_seqlens_q int32 [R+1]; prefix_pages int32 and
    prefix_len int32 [1] (None with max_prefix_len 0); page_table int32
    [R, pages] and suffix_lens int32 [R] (None with max_suffix_len 0). A
    request's last query rows are its last suffix tokens (causal). Rows past
    cu_seqlens_q[R] are left as they are in a given out or lse. The results carry
    no gradients."""
    return _attend_cache(q, cu_seqlens_q, max_seqlen_q, None, cache, prefix_pages, prefix_len, max_prefix_len, page_table,
                         suffix_lens, max_suffix_len, softmax_scale, out, lse, want_lse, workspace, stream)


def _attend_cache(q, cu_seqlens_q, max_seqlen_q, parents, cache, prefix_pages, prefix_len, max_prefix_len, page_table,
                  suffix_lens, max_suffix_len, softmax_scale, out, lse, want_lse, workspace, stream):
    """Both attentions over the cache: of trees where parents are given."""
    shape, dtype, index = _first(q, "q")
    if dtype is _F32:
        raise TypeError("q must be bf16 or fp16")
    qs = _rows(q, "q", index, dtype)
    tq, H, d = shape
    cache_p, Hkv, cd = _cache_args(cache, index)
    page_size = cache_p[5]
    if cd != d:
        raise ValueError("q does not match the cache's head_dim")
    cu_p = _vector(cu_seqlens_q, _I32, "cu_seqlens_q", index)
    R = cu_seqlens_q.numel() - 1
    if R < 0:
        raise ValueError("cu_seqlens_q must have at least one entry")
    max_q, max_p, max_s = int(max_seqlen_q), int(max_prefix_len), int(max_suffix_len)
    parents_p = None if parents is None else _vector(parents, _I32, "parents", index, tq)
    _sizes(tq | H | Hkv | d | R | max_q | max_p | max_s | cache_p[4] | page_size)
    prefix_p = len_p = table_p = suffix_p = None
    if max_p > 0:
        if prefix_pages is None or prefix_len is None:
            raise ValueError("max_prefix_len > 0 needs prefix_pages and prefix_len")
        prefix_p = _vector(prefix_pages, _I32, "prefix_pages", index)
        len_p = _vector(prefix_len, _I32, "prefix_len", index, 1)
        if prefix_pages.numel() * page_size < max_p:
            raise ValueError("prefix_pages holds fewer than max_prefix_len keys")
    table_stride = 0
    if max_s > 0 and R > 0:
        if page_table is None or suffix_lens is None:
            raise ValueError("max_suffix_len > 0 needs page_table and suffix_lens")
        if page_table.dtype is not _I32:
            raise TypeError("page_table must be a CUDA torch.int32 tensor")
        if page_table.get_device() != index:
            raise ValueError(f"page_table must be on cuda:{index}")
        t_shape = page_table.shape
        if len(t_shape) != 2 or t_shape[0] != R or (t_shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("page_table must be an int32 [requests, pages] tensor with contiguous rows")
        table_stride = page_table.stride(0) if R > 1 else t_shape[1]
        if table_stride < t_shape[1]:
            raise ValueError("page_table rows must not overlap")
        if t_shape[1] * page_size < max_s:
            raise ValueError("page_table rows hold fewer than max_suffix_len keys")
        table_p = page_table.data_ptr()
        suffix_p = _vector(suffix_lens, _I32, "suffix_lens", index, R)
    os_ = 0 if out is None else _rows(out, "out", index, dtype, shape)
    if lse is not None:
        _vector(lse, _F32, "lse", index, H * tq)
    if out is not None or lse is not None:
        _written(out, lse)
    size = tsel_prefix_attention_workspace_size if parents is None else tsel_tree_attention_workspace_size
    nbytes = 0 if workspace is not None else size(R, tq, max_q, H, Hkv, d, max_p, max_s)
    workspace = _workspace(workspace, nbytes, index, stream)
    if out is None:
        out = _like(q, stream)
    if lse is None and want_lse:
        lse = _new(stream, torch.empty, (H, tq), dtype=_F32, device=q.device)
    tree = () if parents is None else (parents_p,)
    _call(load_library().tsel_prefix_attention if parents is None else load_library().tsel_tree_attention, index, stream,
          q.data_ptr(), qs, cu_p, R, tq, max_q, *tree, *cache_p, prefix_p, len_p, max_p, table_p, table_stride, suffix_p, max_s, H, Hkv, d,
          _DTYPES[dtype], softmax_scale, out.data_ptr(), os_, _ptr(lse), workspace.data_ptr(),
          workspace.numel())
    return out, lse


def tsel_tree_attention_workspace_size(num_req: int, total_q: int, max_nodes: int, num_heads: int, num_kv_heads: int,
                                       head_dim: int, max_prefix_len: int, max_suffix_len: int) -> int:
    sizes = [int(n) for n in (num_req, total_q, max_nodes, num_heads, num_kv_heads, head_dim, max_prefix_len, max_suffix_len)]
    if any(n >> 31 for n in sizes):   # negative, or more than a C int holds
        return 0
    return int(load_library().tsel_tree_attention_workspace_size(*sizes))


def tsel_tree_attention(q: torch.Tensor, cu_seqlens_q: torch.Tensor, max_nodes: int, parents: torch.Tensor,
                        cache: TselCache, prefix_pages: Optional[torch.Tensor], prefix_len: Optional[torch.Tensor],
                        max_prefix_len: int, page_table: Optional[torch.Tensor], suffix_lens: Optional[torch.Tensor],
                        max_suffix_len: int, *, softmax_scale: float = 0.0, out: Optional[torch.Tensor] = None,
                        lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                        workspace: Optional[torch.Tensor] = None,
                        stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """tsel_prefix_attention of drafted tokens that form a tree in each request; returns
    (out [Tq, H, d], lse fp32 [H, Tq] or None).

    parents int32 [Tq]: each node's parent as an index into its request's nodes, or -1
    for a root. A request's last suffix keys are those of its nodes (at most 64), in
    order; a node sees the prefix, the suffix before the tree, its ancestors and itself.
    The results carry no gradients."""
    if parents is None:
        raise ValueError("parents must be an int32 [tokens] tensor")
    return _attend_cache(q, cu_seqlens_q, max_nodes, parents, cache, prefix_pages, prefix_len, max_prefix_len, page_table,
                         suffix_lens, max_suffix_len, softmax_scale, out, lse, want_lse, workspace, stream)


# ---------------------------------------------------------------------------
# Attention over whole prompts
# ---------------------------------------------------------------------------

def tsel_prompt_attention_workspace_size(num_seg: int, total_q: int, max_seqlen_q: int, max_seqlen_k: int,
                                         num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    sizes = [int(n) for n in (num_seg, total_q, max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_dim)]
    if any(n >> 31 for n in sizes):   # negative, or more than a C int holds
        return 0
    return int(load_library().tsel_prompt_attention_workspace_size(*sizes))


def tsel_prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                          cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int, *,
                          softmax_scale: float = 0.0, flags: int = 0, out: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                          workspace: Optional[torch.Tensor] = None,
                          stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention of packed sequences; returns (out [Tq, H, d], lse fp32 [H, Tq] or None).

    q bf16 or fp16 [Tq, H, d], k and v [Tk, Hkv, d] (rows may be strided, e.g. views
    of a packed QKV tensor); cu_seqlens_q and cu_seqlens_k int32 [G+1]. With
    TSEL_ATT_CAUSAL in flags the last row of a segment sees all its keys and every
    row before it one fewer. lse is what tsel_importance takes with
    TSEL_IMP_LSE_PROVIDED. Rows past cu_seqlens_q[G] are left as they are in a given
    out or lse. The results carry no gradients."""
    shape, dtype, index = _first(q, "q")
    if dtype is _F32:
        raise TypeError("q must be bf16 or fp16")
    qs = _rows(q, "q", index, dtype)
    tq, H, d = shape
    ks = _rows(k, "k", index, dtype)
    k_shape = k.shape
    if len(k_shape) != 3 or k_shape[2] != d:
        raise ValueError("k does not match q's head_dim")
    vs = _rows(v, "v", index, dtype, k_shape)
    tk, Hkv, _ = k_shape
    cu_q = _vector(cu_seqlens_q, _I32, "cu_seqlens_q", index)
    n = cu_seqlens_q.numel()
    if n < 1:
        raise ValueError("cu_seqlens_q must have at least one entry")
    cu_k = _vector(cu_seqlens_k, _I32, "cu_seqlens_k", index, n)
    max_q, max_k = int(max_seqlen_q), int(max_seqlen_k)
    _sizes(tq | tk | H | Hkv | d | max_q | max_k)
    os_ = 0 if out is None else _rows(out, "out", index, dtype, shape)
    if lse is not None:
        _vector(lse, _F32, "lse", index, H * tq)
    if out is not None or lse is not None:
        _written(out, lse)
    nbytes = 0 if workspace is not None else tsel_prompt_attention_workspace_size(n - 1, tq, max_q, max_k, H, Hkv, d)
    workspace = _workspace(workspace, nbytes, index, stream)
    if out is None:
        out = _like(q, stream)
    if lse is None and want_lse:
        lse = _new(stream, torch.empty, (H, tq), dtype=_F32, device=q.device)
    _call(load_library().tsel_prompt_attention, index, stream, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs,
          cu_q, cu_k, n - 1, tq, tk, max_q, max_k, H, Hkv, d, _DTYPES[dtype], softmax_scale, flags, out.data_ptr(),
          os_, _ptr(lse), workspace.data_ptr(), workspace.numel())
    return out, lse


# ---------------------------------------------------------------------------
# Helpers
# ---------------------------------------------------------------------------

def tsel_importance_one_launch(num_seg: int, total_q: int, total_k: int, max_seqlen_q: int,
                               max_seqlen_k: int, num_heads: int, head_dim: int,
                               flags: int = 0) -> int:
    """1 if tsel_importance takes the one-launch path for these sizes and flags
    on the current device, 0 if the scheduled two-pass launches, -1 on a CUDA
    error."""
    return int(load_library().tsel_importance_one_launch(
        int(num_seg), int(total_q), int(total_k), int(max_seqlen_q), int(max_seqlen_k),
        int(num_heads), int(head_dim), int(flags)))


def tsel_keep_count(n_tokens: int, keep_permille: int) -> int:
    return int(load_library().tsel_keep_count(int(n_tokens), int(keep_permille)))


def tsel_read_device_status(workspace: torch.Tensor, stream=None) -> int:
    """Device status bits of a workspace (synchronises the stream)."""
    bits = ctypes.c_uint32(0)
    st = load_library().tsel_read_device_status(_ptr(workspace), ctypes.byref(bits),
                                                _stream(stream, workspace.device))
    if st not in (TSEL_OK, TSEL_ERR_DEVICE_CHECK):
        _check(st)
    return int(bits.value)


def tsel_importance_redo_pairs(workspace: torch.Tensor, stream=None) -> int:
    """(head, query pair)s the last importance call on `workspace` redid with a
    moving reference (synchronises the stream)."""
    n = ctypes.c_int32(0)
    _check(load_library().tsel_importance_redo_pairs(_ptr(workspace), ctypes.byref(n),
                                                     _stream(stream, workspace.device)))
    return int(n.value)


def tsel_select_path_counts(workspace: torch.Tensor, stream=None) -> list:
    """Top-B requests per threshold path on `workspace` since it was zeroed:
    [radix rounds, histogram + rounds, histogram + candidates, candidates
    rejected, ranked in the one-launch importance kernel] (synchronises the
    stream)."""
    c = (ctypes.c_int32 * 5)()
    _check(load_library().tsel_select_path_counts(_ptr(workspace), c,
                                                  _stream(stream, workspace.device)))
    return [int(x) for x in c]


def tsel_clear_device_status(workspace: torch.Tensor, stream=None) -> None:
    _check(load_library().tsel_clear_device_status(_ptr(workspace), _stream(stream, workspace.device)))


def tsel_status_string(status: int) -> str:
    return load_library().tsel_status_string(int(status)).decode()


def tsel_last_error() -> str:
    return load_library().tsel_last_error().decode()


def tsel_probe_ex2(blocks: int, iters: int, sink: torch.Tensor, stream=None) -> None:
    """Enqueues the MUFU exp2 throughput probe (blocks*512*iters*8 exp2).
    sink[blocks*512:] receives block 0's SM cycles and nanoseconds (two
    int64 words), whose ratio is the SM clock during the probe."""
    _need(sink, torch.float32, "sink")
    if sink.numel() < blocks * 512 + 4:
        raise ValueError("sink needs blocks*512 + 4 floats")
    _check(load_library().tsel_probe_ex2(int(blocks), int(iters), _ptr(sink),
                                         _stream(stream, sink.device)))
