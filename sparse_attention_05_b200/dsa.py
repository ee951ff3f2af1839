"""Thin Python binding of the C ABI in include/dsa.h (libdsa.so).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. Tensors are PyTorch CUDA tensors (device memory and streams come from
PyTorch); each call is enqueued on the current PyTorch stream unless a stream
is given. There is no CPU or PyTorch fallback: a missing library raises.
"""

from __future__ import annotations

import ctypes
import dataclasses
import math
import os
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdsa.so")

DSA_KV_CONTIGUOUS = 0
DSA_KV_PAGED = 1

H_IDX, D_IDX, HEADS, D_QK, D_V, MAX_K = 64, 128, 128, 576, 512, 2048

STATUS = {
    0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_UNSUPPORTED_SHAPE", 3: "DSA_ERR_CUDA",
    4: "DSA_ERR_DEVICE_TIMEOUT", 5: "DSA_ERR_BOUNDS", 6: "DSA_ERR_WORKSPACE",
}


class DSAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


class KvDescC(ctypes.Structure):
    _fields_ = [
        ("layout", ctypes.c_int32), ("batch", ctypes.c_int32), ("max_ctx", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("block_table", ctypes.c_void_p),
        ("seqlens", ctypes.c_void_p),
    ]


class QDescC(ctypes.Structure):
    _fields_ = [("num_q", ctypes.c_int32), ("q_per_seq", ctypes.c_int32),
                ("row_begin", ctypes.c_int32), ("row_count", ctypes.c_int32),
                ("q_start", ctypes.c_void_p)]


class RopeDescC(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("layout", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("rot_begin", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("magnitude", ctypes.c_float),
                ("num_rows", ctypes.c_int64), ("x_row_stride", ctypes.c_int64),
                ("x_head_stride", ctypes.c_int64), ("out_row_stride", ctypes.c_int64),
                ("out_head_stride", ctypes.c_int64)]


_P = ctypes.c_void_p
_lib = None

# name -> (restype, argtypes): mirrors include/dsa.h
SIGNATURES = {
    "dsa_indexer_scores": (ctypes.c_int, [_P, _P, _P, _P, ctypes.POINTER(KvDescC),
                                          ctypes.POINTER(QDescC), _P, ctypes.c_int64, _P]),
    "dsa_topk": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.POINTER(KvDescC),
                                ctypes.POINTER(QDescC), ctypes.c_int32, _P, _P]),
    "dsa_topk_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(KvDescC), ctypes.POINTER(QDescC),
                                                  ctypes.c_int32]),
    "dsa_topk_ws": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.POINTER(KvDescC),
                                   ctypes.POINTER(QDescC), ctypes.c_int32, _P, ctypes.c_size_t,
                                   _P, _P]),
    "dsa_sparse_mla_fwd": (ctypes.c_int, [_P, _P, ctypes.POINTER(KvDescC), ctypes.POINTER(QDescC),
                                          _P, ctypes.c_int32, ctypes.c_float, _P, _P, _P]),
    "dsa_sparse_mla_fwd_ws": (ctypes.c_int, [_P, _P, ctypes.POINTER(KvDescC),
                                             ctypes.POINTER(QDescC), _P, ctypes.c_int32,
                                             ctypes.c_float, _P, ctypes.c_size_t, _P, _P, _P]),
    "dsa_sparse_mla_workspace_size": (ctypes.c_size_t, []),
    "dsa_indexer_kl": (ctypes.c_int, [_P, _P, ctypes.POINTER(KvDescC), ctypes.POINTER(QDescC),
                                      _P, ctypes.c_int32, ctypes.c_float, _P, _P, ctypes.c_int64,
                                      _P, _P]),
    "dsa_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(KvDescC), ctypes.POINTER(QDescC),
                                             ctypes.c_int32]),
    "dsa_forward": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.POINTER(KvDescC),
                                   ctypes.POINTER(QDescC), ctypes.c_int32, ctypes.c_float, _P,
                                   ctypes.c_size_t, _P, _P, _P, _P]),
    "dsa_forward_noalloc": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.POINTER(KvDescC),
                                           ctypes.POINTER(QDescC), ctypes.c_int32, ctypes.c_float,
                                           _P, _P, _P, _P]),
    "dsa_mla_up_project": (ctypes.c_int, [_P, _P, _P, ctypes.POINTER(KvDescC), _P, _P, _P,
                                          ctypes.c_int64, _P]),
    "dsa_selection_mask": (ctypes.c_int, [_P, ctypes.c_int32, ctypes.POINTER(KvDescC),
                                          ctypes.POINTER(QDescC), _P, ctypes.c_int64, _P]),
    "dsa_masked_mha": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_int64, ctypes.POINTER(KvDescC),
                                      ctypes.POINTER(QDescC), _P, ctypes.c_int64, ctypes.c_int32,
                                      ctypes.c_float, _P, _P, _P]),
    "dsa_mha_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(KvDescC), ctypes.POINTER(QDescC),
                                                 ctypes.c_int32]),
    "dsa_mha_prefill": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(KvDescC),
                                       ctypes.POINTER(QDescC), ctypes.c_int32, ctypes.c_float, _P,
                                       ctypes.c_size_t, _P, _P, _P, _P]),
    "dsa_fused_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(KvDescC), ctypes.POINTER(QDescC),
                                                   ctypes.c_int32]),
    "dsa_select_fused": (ctypes.c_int, [_P, _P, _P, _P, ctypes.POINTER(KvDescC),
                                        ctypes.POINTER(QDescC), ctypes.c_int32, ctypes.c_int32, _P,
                                        ctypes.c_size_t, _P, _P]),
    "dsa_forward_fused": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.POINTER(KvDescC),
                                         ctypes.POINTER(QDescC), ctypes.c_int32, ctypes.c_float,
                                         ctypes.c_int32, _P, ctypes.c_size_t, _P, _P, _P, _P]),
    "dsa_rope": (ctypes.c_int, [_P, _P, _P, ctypes.POINTER(RopeDescC), _P, _P]),
    "dsa_rope_bwd": (ctypes.c_int, [_P, _P, _P, ctypes.POINTER(RopeDescC), _P, _P]),
    "dsa_cache_append": (ctypes.c_int, [_P, ctypes.c_int64, _P, ctypes.c_int64, _P, _P,
                                        ctypes.c_float, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.POINTER(KvDescC), ctypes.POINTER(QDescC), _P, _P,
                                        _P, _P]),
    "dsa_attn_mass_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(KvDescC),
                                                       ctypes.POINTER(QDescC), ctypes.c_int32]),
    "dsa_attn_mass": (ctypes.c_int, [_P, _P, ctypes.POINTER(KvDescC), ctypes.POINTER(QDescC), _P,
                                     ctypes.c_int32, ctypes.c_float, _P, _P, ctypes.c_int64, _P,
                                     ctypes.c_size_t, _P]),
    "dsa_evict_select": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.POINTER(KvDescC),
                                        ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P,
                                        _P]),
    "dsa_cache_compact": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_int64, ctypes.POINTER(KvDescC),
                                         _P, ctypes.c_int32, _P, ctypes.POINTER(KvDescC), _P, _P,
                                         _P, _P, ctypes.c_int64, _P]),
    "dsa_get_device_error": (ctypes.c_int, [_P]),
    "dsa_set_wait_timeout_ns": (ctypes.c_uint64, [ctypes.c_uint64]),
    "dsa_selftest_wait_timeout": (ctypes.c_int, [_P]),
    "dsa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
}


def lib() -> ctypes.CDLL:
    """Load libdsa.so (built in-tree by ``sparse_attention_05_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libdsa.so not built ({LIB_PATH}); run "
                               "python -m sparse_attention_05_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != 0:
        raise DSAError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the DSA library must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the DSA library must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


@dataclasses.dataclass
class KvLayout:
    """Geometry of the per-token caches (dsa_kv_desc_t)."""
    batch: int
    max_ctx: int
    seqlens: Optional[torch.Tensor] = None         # int32 [batch] on the device
    block_table: Optional[torch.Tensor] = None     # int32 [batch, max_pages] (paged)
    page_size: int = 64
    num_pages: int = 0

    @property
    def paged(self) -> bool:
        return self.block_table is not None

    def c(self) -> KvDescC:
        seqlens = None if self.seqlens is None else _ptr(self.seqlens).value
        if self.block_table is None:
            return KvDescC(DSA_KV_CONTIGUOUS, self.batch, self.max_ctx, 0, 0, 0, None, seqlens)
        return KvDescC(DSA_KV_PAGED, self.batch, self.max_ctx, self.page_size, self.num_pages,
                       self.block_table.shape[1], _ptr(self.block_table).value, seqlens)

    @staticmethod
    def of(problem) -> "KvLayout":
        """Geometry of a synth.Problem whose tensors live on the GPU."""
        return KvLayout(batch=problem.batch, max_ctx=problem.max_ctx, seqlens=problem.seqlens,
                        block_table=problem.block_table if problem.paged else None,
                        page_size=problem.page_size,
                        num_pages=problem.k_idx.shape[0] if problem.paged else 0)


def _qdesc(num_q: int, q_per_seq: int, rows: Optional[Tuple[int, int]] = None,
           q_start: Optional[torch.Tensor] = None) -> QDescC:
    """rows = (row_begin, row_count) window within each sequence (None = all);
    q_start = int32 [batch + 1] device offsets of a ragged batch's query rows
    (sequence b owns rows q_start[b] .. q_start[b+1] - 1; q_per_seq = the largest
    count), None for a uniform batch."""
    r0, rc = rows if rows is not None else (0, 0)
    if q_start is not None and (q_start.dtype != torch.int32 or q_start.dim() != 1):
        raise ValueError("q_start must be a 1-D int32 tensor of batch + 1 offsets")
    return QDescC(num_q, q_per_seq, r0, rc, _ptr(q_start).value if q_start is not None else None)


def round_up(x: int, m: int) -> int:
    return (x + m - 1) // m * m


def _window(kv: KvLayout, q_per_seq: int, rows) -> int:
    """Rows per sequence covered by the window."""
    r0, rc = rows if rows is not None else (0, 0)
    return rc if rc else q_per_seq - r0


def dsa_indexer_scores(q_idx, w, k_idx, k_scale, kv: KvLayout, q_per_seq: int,
                       scores: Optional[torch.Tensor] = None, rows=None,
                       stream=None, q_start=None) -> torch.Tensor:
    """Scores [batch * window_rows, ld] (window rows stored compactly)."""
    T = q_idx.shape[0]
    if scores is None:
        scores = torch.empty(kv.batch * _window(kv, q_per_seq, rows), round_up(kv.max_ctx, 128),
                             dtype=torch.float32, device=q_idx.device)
    kvd, qd = kv.c(), _qdesc(T, q_per_seq, rows, q_start)
    _check(lib().dsa_indexer_scores(_ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(k_scale),
                                    ctypes.byref(kvd), ctypes.byref(qd), _ptr(scores),
                                    scores.shape[1], _stream(stream)), "dsa_indexer_scores")
    return scores


def dsa_topk(scores, kv: KvLayout, q_per_seq: int, k: int,
             idx: Optional[torch.Tensor] = None, rows=None, stream=None, q_start=None,
             num_q: Optional[int] = None) -> torch.Tensor:
    """Selected positions [T, k] (rows outside the window are left untouched). A
    ragged batch (q_start) needs ``idx`` or ``num_q`` for T."""
    if q_start is None:
        T = kv.batch * q_per_seq
    elif num_q is not None:
        T = num_q
    elif idx is not None:
        T = idx.shape[0]
    else:
        raise ValueError("dsa_topk on a ragged batch needs idx or num_q")
    if idx is None:
        idx = torch.empty(T, k, dtype=torch.int32, device=scores.device)
    kvd, qd = kv.c(), _qdesc(T, q_per_seq, rows, q_start)
    _check(lib().dsa_topk(_ptr(scores), scores.shape[1], ctypes.byref(kvd), ctypes.byref(qd), k,
                          _ptr(idx), _stream(stream)), "dsa_topk")
    return idx


def dsa_topk_workspace_size(kv: KvLayout, num_q: int, q_per_seq: int, k: int, rows=None,
                            q_start=None) -> int:
    kvd, qd = kv.c(), _qdesc(num_q, q_per_seq, rows, q_start)
    return int(lib().dsa_topk_workspace_size(ctypes.byref(kvd), ctypes.byref(qd), k))


def dsa_topk_ws(scores, kv: KvLayout, q_per_seq: int, k: int, workspace=None,
                idx: Optional[torch.Tensor] = None, rows=None, stream=None, q_start=None,
                num_q: Optional[int] = None) -> torch.Tensor:
    """dsa_topk with scratch for sweeping long rows with several CTAs (include/dsa.h);
    ``workspace`` is a 256-B aligned device tensor (a fresh one of
    dsa_topk_workspace_size() bytes when None). Same selection as dsa_topk."""
    if q_start is None:
        T = kv.batch * q_per_seq
    elif num_q is not None:
        T = num_q
    elif idx is not None:
        T = idx.shape[0]
    else:
        raise ValueError("dsa_topk_ws on a ragged batch needs idx or num_q")
    if idx is None:
        idx = torch.empty(T, k, dtype=torch.int32, device=scores.device)
    if workspace is None:
        workspace = torch.empty(max(256, dsa_topk_workspace_size(kv, T, q_per_seq, k, rows,
                                                                 q_start)),
                                dtype=torch.uint8, device=scores.device)
    kvd, qd = kv.c(), _qdesc(T, q_per_seq, rows, q_start)
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().dsa_topk_ws(_ptr(scores), scores.shape[1], ctypes.byref(kvd), ctypes.byref(qd),
                             k, _ptr(workspace), nbytes, _ptr(idx), _stream(stream)),
           "dsa_topk_ws")
    return idx


def dsa_sparse_mla_fwd(q, kv_cache, kv: KvLayout, q_per_seq: int, idx, scale: float,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       rows=None, stream=None, q_start=None) -> Tuple[torch.Tensor, torch.Tensor]:
    T = q.shape[0]
    if out is None:
        out = torch.empty(T, HEADS, D_V, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(T, HEADS, dtype=torch.float32, device=q.device)
    kvd, qd = kv.c(), _qdesc(T, q_per_seq, rows, q_start)
    _check(lib().dsa_sparse_mla_fwd(_ptr(q), _ptr(kv_cache), ctypes.byref(kvd), ctypes.byref(qd),
                                    _ptr(idx), idx.shape[1], float(scale), _ptr(out), _ptr(lse),
                                    _stream(stream)), "dsa_sparse_mla_fwd")
    return out, lse


def dsa_sparse_mla_workspace_size() -> int:
    return int(lib().dsa_sparse_mla_workspace_size())


def dsa_sparse_mla_fwd_ws(q, kv_cache, kv: KvLayout, q_per_seq: int, idx, scale: float,
                          workspace: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          rows=None, stream=None, q_start=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """dsa_sparse_mla_fwd with scratch for splitting the rows of a partly filled
    last wave (include/dsa.h); ``workspace`` is any 256-B aligned device tensor
    (a fresh one of dsa_sparse_mla_workspace_size() bytes when None)."""
    T = q.shape[0]
    if workspace is None:
        workspace = torch.empty(dsa_sparse_mla_workspace_size(), dtype=torch.uint8,
                                device=q.device)
    if out is None:
        out = torch.empty(T, HEADS, D_V, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(T, HEADS, dtype=torch.float32, device=q.device)
    kvd, qd = kv.c(), _qdesc(T, q_per_seq, rows, q_start)
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().dsa_sparse_mla_fwd_ws(_ptr(q), _ptr(kv_cache), ctypes.byref(kvd),
                                       ctypes.byref(qd), _ptr(idx), idx.shape[1], float(scale),
                                       _ptr(workspace), nbytes, _ptr(out), _ptr(lse),
                                       _stream(stream)), "dsa_sparse_mla_fwd_ws")
    return out, lse


def dsa_indexer_kl(q, kv_cache, kv: KvLayout, q_per_seq: int, idx, scale: float, lse, scores,
                   kl: Optional[torch.Tensor] = None, rows=None, stream=None, q_start=None) -> torch.Tensor:
    """KL(p || softmax(I)) per row of the window (include/dsa.h): idx [T][k], lse
    [T][128] from dsa_sparse_mla_fwd, scores [batch * window rows][ld]."""
    T = q.shape[0]
    if kl is None:
        kl = torch.empty(kv.batch * _window(kv, q_per_seq, rows), dtype=torch.float32,
                         device=q.device)
    kvd, qd = kv.c(), _qdesc(T, q_per_seq, rows, q_start)
    _check(lib().dsa_indexer_kl(_ptr(q), _ptr(kv_cache), ctypes.byref(kvd), ctypes.byref(qd),
                                _ptr(idx), idx.shape[1], float(scale), _ptr(lse), _ptr(scores),
                                scores.shape[1], _ptr(kl), _stream(stream)), "dsa_indexer_kl")
    return kl


def dsa_workspace_size(kv: KvLayout, num_q: int, q_per_seq: int, k: int, rows=None,
                       q_start=None) -> int:
    kvd, qd = kv.c(), _qdesc(num_q, q_per_seq, rows, q_start)
    return int(lib().dsa_workspace_size(ctypes.byref(kvd), ctypes.byref(qd), k))


def dsa_forward(q_idx, w, k_idx, k_scale, q, kv_cache, kv: KvLayout, q_per_seq: int, k: int,
                scale: float, workspace: Optional[torch.Tensor] = None,
                idx_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, rows=None, stream=None, q_start=None):
    T = q.shape[0]
    if workspace is None:
        nbytes = dsa_workspace_size(kv, T, q_per_seq, k, rows, q_start)
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty(T, HEADS, D_V, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(T, HEADS, dtype=torch.float32, device=q.device)
    kvd, qd = kv.c(), _qdesc(T, q_per_seq, rows, q_start)
    _check(lib().dsa_forward(_ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(k_scale), _ptr(q),
                             _ptr(kv_cache), ctypes.byref(kvd), ctypes.byref(qd), k, float(scale),
                             _ptr(workspace), workspace.numel(), _ptr(idx_out), _ptr(out),
                             _ptr(lse), _stream(stream)), "dsa_forward")
    return out, lse, idx_out


def dsa_forward_noalloc(q_idx, w, k_idx, k_scale, q, kv_cache, kv: KvLayout, q_per_seq: int,
                        k: int, scale: float, idx_out: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        rows=None, stream=None, q_start=None):
    """dsa_forward on the library's own fixed scratch array: the caller passes
    inputs and outputs only (see include/dsa.h for the limits)."""
    T = q.shape[0]
    if out is None:
        out = torch.empty(T, HEADS, D_V, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(T, HEADS, dtype=torch.float32, device=q.device)
    kvd, qd = kv.c(), _qdesc(T, q_per_seq, rows, q_start)
    _check(lib().dsa_forward_noalloc(_ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(k_scale), _ptr(q),
                                     _ptr(kv_cache), ctypes.byref(kvd), ctypes.byref(qd), k,
                                     float(scale), _ptr(idx_out), _ptr(out), _ptr(lse),
                                     _stream(stream)), "dsa_forward_noalloc")
    return out, lse, idx_out


# ---- fused indexer -> top-k (no stored score rows) -------------------------------------


def dsa_fused_workspace_size(kv: KvLayout, num_q: int, q_per_seq: int, k: int, rows=None,
                             q_start=None) -> int:
    kvd, qd = kv.c(), _qdesc(num_q, q_per_seq, rows, q_start)
    return int(lib().dsa_fused_workspace_size(ctypes.byref(kvd), ctypes.byref(qd), k))


def dsa_select_fused(q_idx, w, k_idx, k_scale, kv: KvLayout, q_per_seq: int, k: int,
                     cand_cap: int = 0, idx=None, workspace=None, rows=None, stream=None, q_start=None):
    """Selected positions [T, k] without stored score rows (include/dsa.h)."""
    T = q_idx.shape[0]
    if idx is None:
        idx = torch.empty(T, k, dtype=torch.int32, device=q_idx.device)
    if workspace is None:
        nbytes = dsa_fused_workspace_size(kv, T, q_per_seq, k, rows, q_start)
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q_idx.device)
    kvd, qd = kv.c(), _qdesc(T, q_per_seq, rows, q_start)
    _check(lib().dsa_select_fused(_ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(k_scale),
                                  ctypes.byref(kvd), ctypes.byref(qd), k, int(cand_cap),
                                  _ptr(workspace), workspace.numel(), _ptr(idx), _stream(stream)),
           "dsa_select_fused")
    return idx


def dsa_forward_fused(q_idx, w, k_idx, k_scale, q, kv_cache, kv: KvLayout, q_per_seq: int,
                      k: int, scale: float, cand_cap: int = 0, workspace=None, idx_out=None,
                      out=None, lse=None, rows=None, stream=None, q_start=None):
    T = q.shape[0]
    if workspace is None:
        nbytes = dsa_fused_workspace_size(kv, T, q_per_seq, k, rows, q_start)
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty(T, HEADS, D_V, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(T, HEADS, dtype=torch.float32, device=q.device)
    kvd, qd = kv.c(), _qdesc(T, q_per_seq, rows, q_start)
    _check(lib().dsa_forward_fused(_ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(k_scale), _ptr(q),
                                   _ptr(kv_cache), ctypes.byref(kvd), ctypes.byref(qd), k,
                                   float(scale), int(cand_cap), _ptr(workspace),
                                   workspace.numel(), _ptr(idx_out), _ptr(out), _ptr(lse),
                                   _stream(stream)), "dsa_forward_fused")
    return out, lse, idx_out


# ---- MLA in MHA mode (masked-MHA emulation of DSA for short prefill) -------------------

MHA_DN, MHA_DR, MHA_DV = 128, 64, 128


def mha_ctx_pad(kv: KvLayout) -> int:
    """Key slots per (sequence, head) of the decompressed keys and values."""
    return round_up(kv.max_ctx, 128)


def dsa_mla_up_project(kv_cache, w_uk, w_uv, kv: KvLayout, k_nope=None, k_rope=None, v=None,
                       stream=None):
    """Decompressed MHA-mode keys / values (include/dsa.h): k_nope [B,128,ctx_pad,128],
    k_rope [B,ctx_pad,64], v [B,128,ctx_pad,128], all bf16."""
    cp = mha_ctx_pad(kv)
    dev = kv_cache.device
    if k_nope is None:
        k_nope = torch.empty(kv.batch, HEADS, cp, MHA_DN, dtype=torch.bfloat16, device=dev)
    if k_rope is None:
        k_rope = torch.empty(kv.batch, cp, MHA_DR, dtype=torch.bfloat16, device=dev)
    if v is None:
        v = torch.empty(kv.batch, HEADS, cp, MHA_DV, dtype=torch.bfloat16, device=dev)
    kvd = kv.c()
    _check(lib().dsa_mla_up_project(_ptr(kv_cache), _ptr(w_uk), _ptr(w_uv), ctypes.byref(kvd),
                                    _ptr(k_nope), _ptr(k_rope), _ptr(v), k_nope.shape[2],
                                    _stream(stream)), "dsa_mla_up_project")
    return k_nope, k_rope, v


def dsa_selection_mask(idx, kv: KvLayout, q_per_seq: int, mask=None, rows=None, stream=None,
                       q_start=None):
    """Selection bits [T, mask_ld] uint32 (stored as int32) of the window's rows."""
    T, k = idx.shape
    if mask is None:
        mask = torch.zeros(T, mha_ctx_pad(kv) // 32, dtype=torch.int32, device=idx.device)
    kvd, qd = kv.c(), _qdesc(T, q_per_seq, rows, q_start)
    _check(lib().dsa_selection_mask(_ptr(idx), k, ctypes.byref(kvd), ctypes.byref(qd),
                                    _ptr(mask), mask.shape[1], _stream(stream)),
           "dsa_selection_mask")
    return mask


def dsa_masked_mha(q_mha, k_nope, k_rope, v, kv: KvLayout, q_per_seq: int, scale: float,
                   mask=None, k: int = 0, out=None, lse=None, rows=None, stream=None, q_start=None):
    """Masked MHA (include/dsa.h): out [T,128,128] bf16, lse [T,128] fp32."""
    T = q_mha.shape[0]
    if out is None:
        out = torch.empty(T, HEADS, MHA_DV, dtype=torch.bfloat16, device=q_mha.device)
    if lse is None:
        lse = torch.empty(T, HEADS, dtype=torch.float32, device=q_mha.device)
    kvd, qd = kv.c(), _qdesc(T, q_per_seq, rows, q_start)
    _check(lib().dsa_masked_mha(_ptr(q_mha), _ptr(k_nope), _ptr(k_rope), _ptr(v),
                                k_nope.shape[2], ctypes.byref(kvd), ctypes.byref(qd), _ptr(mask),
                                mask.shape[1] if mask is not None else 0, int(k), float(scale),
                                _ptr(out), _ptr(lse), _stream(stream)), "dsa_masked_mha")
    return out, lse


def dsa_mha_workspace_size(kv: KvLayout, num_q: int, q_per_seq: int, k: int, rows=None,
                           q_start=None) -> int:
    kvd, qd = kv.c(), _qdesc(num_q, q_per_seq, rows, q_start)
    return int(lib().dsa_mha_workspace_size(ctypes.byref(kvd), ctypes.byref(qd), k))


def dsa_mha_prefill(q_idx, w, k_idx, k_scale, q_mha, kv_cache, w_uk, w_uv, kv: KvLayout,
                    q_per_seq: int, k: int, scale: float, workspace=None, idx_out=None,
                    out=None, lse=None, rows=None, stream=None, q_start=None):
    """Short-prefill DSA in MHA mode: indexer -> top-k -> masks -> up-projection ->
    masked MHA, one call (include/dsa.h)."""
    T = q_mha.shape[0]
    if workspace is None:
        nbytes = dsa_mha_workspace_size(kv, T, q_per_seq, k, rows, q_start)
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q_mha.device)
    if out is None:
        out = torch.empty(T, HEADS, MHA_DV, dtype=torch.bfloat16, device=q_mha.device)
    if lse is None:
        lse = torch.empty(T, HEADS, dtype=torch.float32, device=q_mha.device)
    kvd, qd = kv.c(), _qdesc(T, q_per_seq, rows, q_start)
    _check(lib().dsa_mha_prefill(_ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(k_scale), _ptr(q_mha),
                                 _ptr(kv_cache), _ptr(w_uk), _ptr(w_uv), ctypes.byref(kvd),
                                 ctypes.byref(qd), k, float(scale), _ptr(workspace),
                                 workspace.numel(), _ptr(idx_out), _ptr(out), _ptr(lse),
                                 _stream(stream)), "dsa_mha_prefill")
    return out, lse, idx_out


# ---- filling, weighing and trimming the two caches --------------------------------------

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_HALF, _INTERLEAVED, _NONE = 0, 1, 2
D_ROPE = 64


def rope_freqs(rot_dim: int, base: float = 10000.0, scaling: Optional[str] = None,
               factor: float = 1.0, original_ctx: int = 4096, beta_fast: float = 32.0,
               beta_slow: float = 1.0, device=None) -> Tuple[torch.Tensor, float]:
    """Radians per position of each pair (fp64 [rot_dim / 2]), for ``dsa_rope`` and
    ``dsa_cache_append``, and the schedule's factor m on queries and keys. With
    theta_i = base^(-2i / rot_dim):
      None      theta_i
      "linear"  theta_i / factor (position interpolation)
      "ntk"     the same for base * factor^(rot_dim / (rot_dim - 2))
      "yarn"    g_i theta_i + (1 - g_i) theta_i / factor, g_i rising linearly from 0 at
                beta_slow to 1 at beta_fast turns over original_ctx positions, and
                m = 0.1 ln(factor) + 1 (YaRN, arXiv 2309.00071, section 3)
    m scales the whole logit by m^2. Heads that rotate in all their dims may have it from
    the calls' ``magnitude``; MLA's and the indexer's rotate in a part of theirs, so there
    ``magnitude`` stays 1 and the attention's scale becomes scale * m**2 (the indexer's
    selection does not depend on it).
    Any other schedule is a tensor of one's own."""
    if rot_dim < 2 or rot_dim % 2 or base <= 0 or factor <= 0 or original_ctx < 1:
        raise ValueError("rope_freqs: rot_dim must be even and base, factor, original_ctx positive")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"rope_freqs: unknown scaling {scaling!r}")
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("rope_freqs: ntk scaling needs rot_dim >= 4")
        base = base * factor ** (rot_dim / (rot_dim - 2.0))
    theta = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    magnitude = 1.0
    if scaling == "linear":
        theta = [t / factor for t in theta]
    elif scaling == "yarn":
        if beta_fast <= beta_slow:
            raise ValueError("rope_freqs: beta_fast must exceed beta_slow")
        turns = [original_ctx * t / (2.0 * math.pi) for t in theta]
        g = [min(1.0, max(0.0, (r - beta_slow) / (beta_fast - beta_slow))) for r in turns]
        theta = [gi * t + (1.0 - gi) * t / factor for gi, t in zip(g, theta)]
        magnitude = 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
    return torch.tensor(theta, dtype=torch.float64, device=device), magnitude


def _need(name: str, t: torch.Tensor, dtype, shape, device: int) -> int:
    """Address of a contiguous tensor of this type, shape (None: any) and device."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _device(t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError("tensors passed to the DSA library must be CUDA tensors")
    return t.get_device()


def _kv_desc(kv: KvLayout, device: int, q_start: Optional[torch.Tensor] = None) -> KvDescC:
    """kv.c() with its tensors' types, sizes and device checked (and q_start's size)."""
    lens, table = kv.seqlens, kv.block_table
    if lens is not None:
        lens = _need("seqlens", lens, torch.int32, (kv.batch,), device)
    if q_start is not None:
        _need("q_start", q_start, torch.int32, (kv.batch + 1,), device)
    if table is None:
        return KvDescC(DSA_KV_CONTIGUOUS, kv.batch, kv.max_ctx, 0, 0, 0, None, lens)
    if table.dim() != 2 or table.shape[0] != kv.batch:
        raise ValueError("block_table must be [batch, max_pages]")
    return KvDescC(DSA_KV_PAGED, kv.batch, kv.max_ctx, kv.page_size, kv.num_pages, table.shape[1],
                   _need("block_table", table, torch.int32, None, device), lens)


def _rows_shape(kv: KvLayout):
    return (kv.batch, kv.max_ctx) if kv.block_table is None else (kv.num_pages, kv.page_size)


def _cache_ptrs(kv: KvLayout, kv_cache, k_idx, k_scale, device: int):
    """The three cache arrays of one geometry, checked."""
    n = _rows_shape(kv)
    return (_need("kv_cache", kv_cache, torch.bfloat16, (*n, D_QK), device),
            _need("k_idx", k_idx, torch.uint8, (*n, D_IDX), device),
            _need("k_scale", k_scale, torch.float32, n, device))


def _call(name: str, device: int, stream, *args) -> None:
    """The library call on the device of its tensors, on ``stream`` or that device's
    current one."""
    f = getattr(lib(), name)
    st = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
    if device == torch.cuda.current_device():
        status = f(*args, st)
    else:
        with torch.cuda.device(device):
            status = f(*args, st)
    if status:
        raise DSAError(status, name)


def _new(shape, dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """A tensor for the call to write, allocated for the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _rope(where, x, positions, freqs, out, rot_begin, interleaved, magnitude, stream):
    if x.dtype not in _DTYPES:
        raise ValueError(f"x must be bfloat16, float16 or float32, got {x.dtype}")
    if (x.requires_grad or out is not None and out.requires_grad) and torch.is_grad_enabled():
        raise ValueError(f"{where} records no gradient: pass detached tensors, and take the "
                         "gradient from dsa_rope_bwd")
    dev = _device(x)
    given = out is not None
    if not given:
        out = _new(x.shape, x.dtype, x, stream)
    elif out.shape != x.shape or out.dtype is not x.dtype or out.get_device() != dev:
        raise ValueError("out must have x's shape, type and device")
    shape, xs, os = x.shape, x.stride(), out.stride()
    if len(shape) == 3:
        rows, heads, dim = shape
        x_head, out_head = xs[1], os[1]
    elif len(shape) == 2:
        (rows, dim), heads = shape, 1
        x_head = out_head = dim
    else:
        raise ValueError("x must be [rows, dim] or [rows, heads, dim]")
    if dim > 1 and (xs[-1] != 1 or os[-1] != 1):
        raise ValueError("the last axis of x and out must be contiguous")
    if freqs.dim() != 1:
        raise ValueError("freqs must be one-dimensional")
    d = RopeDescC(_DTYPES[x.dtype], _INTERLEAVED if interleaved else _HALF, heads, dim, rot_begin,
                  2 * freqs.shape[0], magnitude, rows, xs[0], x_head, os[0], out_head)
    if heads and rows:
        _call(where, dev, stream, x.data_ptr(),
              _need("positions", positions, torch.int32, (rows,), dev),
              _need("freqs", freqs, torch.float64, None, dev), ctypes.byref(d), out.data_ptr())
        if given and not out.is_inference():  # autograd may have saved what it held
            torch.autograd.graph.increment_version(out)
    return out


def dsa_rope(x, positions, freqs, out=None, rot_begin: int = 0, interleaved: bool = False,
             magnitude: float = 1.0, stream=None) -> torch.Tensor:
    """Rotary positions on dims [rot_begin, rot_begin + 2 len(freqs)) of every head of x
    [rows, dim] or [rows, heads, dim] (strided views allowed); ``out=x`` works in place.
    positions int32 [rows]; magnitude a factor on those dims (include/dsa.h, ``rope_freqs``).
    No gradient is recorded (a tensor that requires one is refused outside no_grad):
    ``dsa_rope_bwd`` is its backward pass."""
    return _rope("dsa_rope", x, positions, freqs, out, rot_begin, interleaved, magnitude, stream)


def dsa_rope_bwd(dout, positions, freqs, dx=None, rot_begin: int = 0, interleaved: bool = False,
                 magnitude: float = 1.0, stream=None) -> torch.Tensor:
    """The gradient of ``dsa_rope``'s input from that of its output; ``dx=dout`` works in
    place. Where the forward read one row or head for several (a broadcast input), dx has
    each one's part, to be summed."""
    return _rope("dsa_rope_bwd", dout, positions, freqs, dx, rot_begin, interleaved, magnitude,
                 stream)


def dsa_cache_append(latent_new, k_new, kv_cache, k_idx, k_scale, kv: KvLayout, q_per_seq: int,
                     freqs, positions=None, interleaved: bool = True,
                     idx_interleaved: Optional[bool] = False, magnitude: float = 1.0, rows=None,
                     stream=None, q_start=None) -> None:
    """The new tokens into both caches (include/dsa.h): latent_new bf16 [T, 576] (the last
    64 dims not yet rotated) and k_new bf16 [T, 128], each row's elements consecutive. Token
    t goes to the slot of query row t; its rotary position is that slot, or positions[t].
    ``interleaved`` is the pairing of the latent's rope dims, ``idx_interleaved`` that of the
    key's first 64 dims (None: the key is not rotated)."""
    T, dev = latent_new.shape[0], _device(kv_cache)
    for name, x, dim in (("latent_new", latent_new, D_QK), ("k_new", k_new, D_IDX)):
        if x.dtype is not torch.bfloat16 or x.shape != (T, dim) or x.get_device() != dev:
            raise ValueError(f"{name} must be a bfloat16 [T, {dim}] tensor on cuda:{dev}")
        if x.stride(1) != 1:
            raise ValueError(f"the last axis of {name} must be contiguous")
    kvd, qd = _kv_desc(kv, dev, q_start), _qdesc(T, q_per_seq, rows, q_start)
    _call("dsa_cache_append", dev, stream, latent_new.data_ptr(),
          latent_new.stride(0) if T > 1 else D_QK, k_new.data_ptr(),
          k_new.stride(0) if T > 1 else D_IDX,
          None if positions is None else _need("positions", positions, torch.int32, (T,), dev),
          _need("freqs", freqs, torch.float64, (D_ROPE // 2,), dev), magnitude,
          _INTERLEAVED if interleaved else _HALF,
          _NONE if idx_interleaved is None else _INTERLEAVED if idx_interleaved else _HALF,
          ctypes.byref(kvd), ctypes.byref(qd), *_cache_ptrs(kv, kv_cache, k_idx, k_scale, dev))


def dsa_attn_mass_workspace_size(kv: KvLayout, num_q: int, q_per_seq: int, k: int, rows=None,
                                 q_start=None) -> int:
    kvd, qd = kv.c(), _qdesc(num_q, q_per_seq, rows, q_start)
    return int(lib().dsa_attn_mass_workspace_size(ctypes.byref(kvd), ctypes.byref(qd), k))


def _mass_ptr(name, mass, kv: KvLayout, dev: int) -> int:
    if mass.dim() != 2 or mass.shape[0] != kv.batch or mass.shape[1] < kv.max_ctx:
        raise ValueError(f"{name} must be [batch, >= max_ctx]")
    return _need(name, mass, torch.float32, None, dev)


def dsa_attn_mass(q, kv_cache, kv: KvLayout, q_per_seq: int, idx, scale: float, lse, mass,
                  workspace: Optional[torch.Tensor] = None, rows=None, stream=None,
                  q_start=None) -> torch.Tensor:
    """The head mean of the window's attention weights added to mass [batch, >= max_ctx], by
    slot (include/dsa.h): idx [T, k] and lse [T, 128] as the forward used and wrote them;
    ``workspace`` is a 256-B aligned device tensor (a fresh one when None, none for one row a
    sequence)."""
    T, k, dev = q.shape[0], idx.shape[1], _device(q)
    kvd, qd = _kv_desc(kv, dev, q_start), _qdesc(T, q_per_seq, rows, q_start)
    ref, qref = ctypes.byref(kvd), ctypes.byref(qd)
    args = (_need("q", q, torch.bfloat16, (T, HEADS, D_QK), dev),
            _need("kv_cache", kv_cache, torch.bfloat16, (*_rows_shape(kv), D_QK), dev), ref, qref,
            _need("idx", idx, torch.int32, (T, k), dev), k, scale,
            _need("lse", lse, torch.float32, (T, HEADS), dev), _mass_ptr("mass", mass, kv, dev),
            mass.shape[1])
    nbytes = 0
    if workspace is None:
        need = lib().dsa_attn_mass_workspace_size(ref, qref, k)
        if need:
            workspace, nbytes = _new(need, torch.uint8, q, stream), need
    else:
        if workspace.get_device() != dev:
            raise ValueError(f"workspace is on {workspace.device}, not on cuda:{dev}")
        nbytes = workspace.numel() * workspace.element_size()
    _call("dsa_attn_mass", dev, stream, *args, _ptr(workspace), nbytes)
    return mass


def dsa_evict_select(mass, kv: KvLayout, keep: int, sink: int = 0, recent: int = 0,
                     kept: Optional[torch.Tensor] = None,
                     new_lens: Optional[torch.Tensor] = None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The slots that stay when each sequence is trimmed to ``keep`` tokens (include/dsa.h):
    (kept int32 [batch, keep] ascending and padded with -1, new_lens int32 [batch])."""
    dev = _device(mass)
    if kept is None:
        kept = _new((kv.batch, max(keep, 0)), torch.int32, mass, stream)
    if new_lens is None:
        new_lens = _new(kv.batch, torch.int32, mass, stream)
    kvd = _kv_desc(kv, dev)
    _call("dsa_evict_select", dev, stream, _mass_ptr("mass", mass, kv, dev), mass.shape[1],
          ctypes.byref(kvd), keep, sink, recent,
          _need("kept", kept, torch.int32, (kv.batch, keep), dev),
          _need("new_lens", new_lens, torch.int32, (kv.batch,), dev))
    return kept, new_lens


def dsa_cache_compact(kv_cache, k_idx, k_scale, kv: KvLayout, kept, new_lens,
                      mass: Optional[torch.Tensor] = None, dst: Optional[KvLayout] = None,
                      dst_kv_cache=None, dst_k_idx=None, dst_k_scale=None, dst_mass=None,
                      stream=None) -> None:
    """Moves the tokens that stay together (include/dsa.h), in place, or into the slots of
    ``dst``: other cache arrays, or the same ones with pages that no source sequence uses."""
    dev = _device(kv_cache)
    kvd = _kv_desc(kv, dev)
    if kept.dim() != 2 or kept.shape[0] != kv.batch:
        raise ValueError("kept must be [batch, keep]")
    m = None if mass is None else _mass_ptr("mass", mass, kv, dev)
    dm, dstd = None, None
    if dst is None:
        to = (dst_kv_cache, dst_k_idx, dst_k_scale)
        if to != (None, None, None) or dst_mass is not None:
            raise ValueError("dst arrays need a dst layout")
    else:
        if dst.batch != kv.batch:
            raise ValueError("dst must have the source's batch")
        if (mass is None) != (dst_mass is None):
            raise ValueError("mass and dst_mass go together")
        to = _cache_ptrs(dst, dst_kv_cache, dst_k_idx, dst_k_scale, dev)
        dm = None if dst_mass is None else _mass_ptr("dst_mass", dst_mass, dst, dev)
        dstc = _kv_desc(dst, dev)
        dstd = ctypes.byref(dstc)
    _call("dsa_cache_compact", dev, stream, *_cache_ptrs(kv, kv_cache, k_idx, k_scale, dev), m,
          0 if m is None else mass.shape[1], ctypes.byref(kvd),
          _need("kept", kept, torch.int32, None, dev), kept.shape[1],
          _need("new_lens", new_lens, torch.int32, (kv.batch,), dev), dstd, *to, dm,
          0 if dm is None else dst_mass.shape[1])


def dsa_get_device_error(stream=None) -> int:
    return int(lib().dsa_get_device_error(_stream(stream)))


def dsa_set_wait_timeout_ns(ns: int) -> int:
    return int(lib().dsa_set_wait_timeout_ns(ns))


def dsa_selftest_wait_timeout(stream=None) -> int:
    return int(lib().dsa_selftest_wait_timeout(_stream(stream)))


def dsa_status_string(status: int) -> str:
    return lib().dsa_status_string(status).decode()
