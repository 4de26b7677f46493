"""lightning_indexer_top_gb300 -- lightning-indexer sparse attention on GB300.

A thin ctypes binding over ``liblidx.so`` (C ABI in ``include/lidx.h``).  The
functions here only marshal torch tensors into pointers, sizes and the current
CUDA stream; every step of the computation runs in the library's kernels.
There is no CPU fallback: if the library is missing or fails to load, every
call raises.

Build with ``lightning_indexer_top_gb300.build()`` (nvcc, sm_103a).
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

from ._build import LIB as _LIB_PATH
from ._build import build  # noqa: F401

__all__ = [
    "Batch", "LidxError", "build", "load", "idx_hadamard", "idx_score", "idx_block_pool", "idx_block_pool_update",
    "idx_quantize_rows", "idx_score_q8", "inline_scales",
    "idx_topk", "sparse_attn_decode", "sparse_attn_prefill", "idx_workspace_size",
    "idx_device_status", "topk_capacity", "sparse_attn_decode_noalloc", "idx_score_topk", "idx_block_score_topk", "sparse_decode_step", "sparse_decode_step_fused",
    "dense_attn", "dense_attn_workspace_size", "idx_page_copy", "idx_page_update", "idx_page_compact",
    "idx_page_workspace_size",
]

IDX_OK, IDX_ERR_INVALID_ARG, IDX_ERR_UNSUPPORTED, IDX_ERR_CUDA, IDX_ERR_TIMEOUT, IDX_ERR_DEVICE_BOUNDS, IDX_ERR_INEXACT = range(7)
IDX_F32, IDX_F16, IDX_BF16 = 0, 1, 2
IDX_POS_CLEAN = 2**31 - 1   # stale_pos value: no edit
IDX_OP_SCORE, IDX_OP_TOPK, IDX_OP_ATTN_DECODE, IDX_OP_ATTN_PREFILL, IDX_OP_SCORE_TOPK, IDX_OP_DECODE_STEP = 0, 1, 2, 3, 4, 5

_DTYPES = {torch.float32: IDX_F32, torch.float16: IDX_F16, torch.bfloat16: IDX_BF16}


class LidxError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"lidx status {status}: {msg}")
        self.status = status


class _Batch(ctypes.Structure):
    _fields_ = [
        ("n_seq", ctypes.c_int32),
        ("n_q_per_seq", ctypes.c_int32),
        ("n_kv", ctypes.c_void_p),
        ("kv_start", ctypes.c_void_p),
        ("kv_seq_stride", ctypes.c_int64),
        ("q_pos", ctypes.c_void_p),
        ("max_n_kv", ctypes.c_int32),
        ("page_table", ctypes.c_void_p),
        ("page_table_stride", ctypes.c_int64),
        ("page_size", ctypes.c_int32),
    ]


class _Mods(ctypes.Structure):
    _fields_ = [
        ("softcap", ctypes.c_float),
        ("slopes", ctypes.c_void_p),
        ("window", ctypes.c_int32),
        ("prefix_len", ctypes.c_void_p),
        ("doc_start", ctypes.c_void_p),
        ("prefix_end", ctypes.c_void_p),
    ]


class _PageCache(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("row_stride_bytes", ctypes.c_int64),
        ("row_bytes", ctypes.c_int64),
    ]


IDX_MAX_PAGE_CACHES = 8

_lib = None


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load liblidx.so (once) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run lightning_indexer_top_gb300.build() first")
    lib = ctypes.CDLL(path)
    P, I32, I64, F, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    sigs = {
        "idx_hadamard": [P, P, I32, I64, I32, I64, P],
        "idx_score": [P, I32, P, I32, I32, P, I32, I64, I64, _Batch, I32, P, I64, P, SZ, P],
        "idx_block_pool": [P, I32, I64, I64, _Batch, I32, I32, P, I64, P],
        "idx_block_pool_update": [P, I32, I64, I64, _Batch, P, P, I32, I32, P, I64, P],
        "idx_quantize_rows": [P, I32, I64, I32, I64, P, I64, P, P],
        "idx_score_q8": [P, I32, P, I32, I32, P, I64, P, I64, _Batch, I32, P, I64, P, SZ, P],
        "idx_topk": [P, I64, _Batch, I32, I32, P, I64, P, P, SZ, P],
        "idx_score_topk": [P, I32, P, I32, I32, P, I32, I64, I64, _Batch, I32, P, I64, P, I64, P, P, SZ, P],
        "idx_block_score_topk": [P, I32, P, I32, I32, P, I32, I64, I64, _Batch, P, P, I32, P, I64, I32, P, I64, P,
                                 I64, P, P],
        "sparse_attn_decode": [P, I32, I32, I32, I32, I32, P, P, I64, I64, I64, _Batch, P, I64, P, F,
                               P, I32, P, SZ, P],
        "sparse_attn_prefill": [P, I32, I32, I32, I32, I32, P, P, I64, I64, I64, _Batch, P, I64, P, F,
                                P, I32, P, SZ, P],
        "sparse_attn_decode_noalloc": [P, I32, I32, I32, I32, I32, P, I64, I64, _Batch, P, I64, P, F, P, I32, P],
        "sparse_decode_step": [P, I32, P, I32, I32, P, I32, I64, I64, _Batch, I32, P, I64, P, I64, P,
                               P, I32, I32, I32, I32, I32, P, P, I64, I64, I64, F, P, I32, P, SZ, P],
        "idx_workspace_size": [I32, I64, I32, I32, I32, I32],
        "sparse_decode_step_fused": [I64, I32, I32, I32, I64],
        "dense_attn": [P, I32, I32, I32, I32, I32, P, P, I64, I64, I64, _Batch, ctypes.POINTER(_Mods), F, P, P, P, SZ,
                       P],
        "dense_attn_workspace_size": [I32, I32, I32, I32, I32, I32, I32, I32],
        "idx_page_copy": [ctypes.POINTER(_PageCache), I32, I32, I32, P, P, I32, P],
        "idx_page_update": [P, I64, I32, I32, P, P, P, I32, I32, I32, P, P, I64, I32, P, ctypes.POINTER(_PageCache), I32,
                            P, SZ, P],
        "idx_page_compact": [P, I64, I32, I32, P, I32, I32, P, P, I64, P, P, ctypes.POINTER(_PageCache), I32, P, SZ, P],
        "idx_page_workspace_size": [I32, I32],
        "idx_last_error": [],
        "idx_device_status": [I32],
    }
    for name, args in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    for name in ("idx_workspace_size", "dense_attn_workspace_size", "idx_page_workspace_size"):
        getattr(lib, name).restype = ctypes.c_size_t
    lib.idx_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != IDX_OK:
        raise LidxError(status, load().idx_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# the current stream of a device as an address, without the Stream object around it (2 us less a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> int:
    """The current stream of a tensor's device."""
    if _raw_stream is None:     # (not part of torch's public interface)
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(device.index)


def _dtype(t: torch.Tensor) -> int:
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("lidx operates on CUDA tensors only")


@dataclass
class Batch:
    """Batch geometry (see idx_batch in include/lidx.h).

    n_kv:      int32 CUDA tensor [B], cached tokens per sequence.
    n_q_per_seq: query rows per sequence (decode: 1).
    max_n_kv:  host bound on every n_kv[b].
    kv_start:  optional int32 CUDA tensor [B]: cache row of position 0.
    kv_seq_stride: rows between sequences when kv_start is None.
    q_pos:     optional int32 CUDA tensor [B*T]: causal position per query row.
    page_table: optional int32 CUDA tensor [B, pages]: physical page of each logical page
               (position j of sequence b is cache row page_table[b, j // page_size] * page_size
               + j % page_size); kv_start / kv_seq_stride are then unused.
    """

    n_kv: torch.Tensor
    n_q_per_seq: int
    max_n_kv: int
    kv_start: Optional[torch.Tensor] = None
    kv_seq_stride: int = 0
    q_pos: Optional[torch.Tensor] = None
    page_table: Optional[torch.Tensor] = None
    page_size: int = 0

    @property
    def n_seq(self) -> int:
        return int(self.n_kv.numel())

    @property
    def n_rows(self) -> int:
        return self.n_seq * self.n_q_per_seq

    def c(self) -> _Batch:
        ptrs = []
        for t in (self.n_kv, self.kv_start, self.q_pos, self.page_table):
            if t is not None and (t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous()):
                raise ValueError("batch arrays must be contiguous int32 CUDA tensors")
            ptrs.append(None if t is None else t.data_ptr())
        pt_stride = self.page_table.shape[-1] if self.page_table is not None else 0
        return _Batch(self.n_seq, self.n_q_per_seq, ptrs[0], ptrs[1], self.kv_seq_stride, ptrs[2], self.max_n_kv,
                      ptrs[3], pt_stride, self.page_size if self.page_table is not None else 0)


IDX_DEFAULT_TOP_K = 2048   # top_k = -1: the model's configured indexer top_k


def topk_capacity(top_k: int, block_size: int = 0) -> int:
    """Row capacity idx_topk writes: top_k, or floor(top_k/C)*C + C - 1 in block mode (-1: the default)."""
    if top_k == -1:
        top_k = IDX_DEFAULT_TOP_K
    if block_size > 1:
        return (top_k // block_size) * block_size + block_size - 1
    return top_k


def idx_hadamard(x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotate the rows (last dim) of x by the orthonormal Hadamard matrix into `out`
    (in place when out is None or is x)."""
    out = x if out is None else out
    _need_cuda(x, out)
    if not x.is_contiguous() or not out.is_contiguous() or out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("x and out must be contiguous tensors of the same shape and dtype")
    d = x.shape[-1]
    rows = x.numel() // d
    _check(load().idx_hadamard(_ptr(x), _ptr(out), _dtype(x), rows, d, d, _stream(x.device)))
    return out


def idx_workspace_size(op: int, n_rows: int, max_n_kv: int, top_k: int, n_q_heads: int = 0, dv: int = 0) -> int:
    return int(load().idx_workspace_size(op, n_rows, max_n_kv, top_k, n_q_heads, dv))


def idx_score(q: torch.Tensor, w: torch.Tensor, k: torch.Tensor, batch: Batch, *, block_size: int = 0,
              scores: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Indexer scores [B*T, keys] f32.  q [B*T, H, d]; w [B*T, H] f32; k [rows, d] (key cache
    or pooled keys when block_size > 1)."""
    _need_cuda(q, w, k, scores, workspace)
    rows, H, d = q.shape
    assert rows == batch.n_rows and w.shape == (rows, H) and w.dtype == torch.float32
    assert q.is_contiguous() and w.is_contiguous() and k.stride(-1) == 1
    keys = batch.max_n_kv // block_size if block_size > 1 else batch.max_n_kv
    if scores is None:
        scores = torch.empty(rows, max(keys, 1), device=q.device, dtype=torch.float32)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().idx_score(_ptr(q), _dtype(q), _ptr(w), H, d, _ptr(k), _dtype(k), k.stride(0),
                            k.shape[0], batch.c(), block_size, _ptr(scores), scores.stride(0),
                            _ptr(workspace), ws_bytes, _stream(q.device)))
    return scores


def idx_block_pool(k_raw: torch.Tensor, batch: Batch, block_size: int, *, pool_seq_stride: Optional[int] = None,
                   pooled: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Mean-pooled complete blocks, f32 [B, pool_seq_stride, d]."""
    _need_cuda(k_raw, pooled)
    d = k_raw.shape[-1]
    if pool_seq_stride is None:
        pool_seq_stride = max(batch.max_n_kv // block_size, 1)
    if pooled is None:
        pooled = torch.zeros(batch.n_seq, pool_seq_stride, d, device=k_raw.device, dtype=torch.float32)
    _check(load().idx_block_pool(_ptr(k_raw), _dtype(k_raw), k_raw.stride(0), k_raw.shape[0], batch.c(),
                                 block_size, d, _ptr(pooled), pool_seq_stride, _stream(k_raw.device)))
    return pooled


def idx_quantize_rows(x: torch.Tensor, *, q8: Optional[torch.Tensor] = None,
                      scale: Optional[torch.Tensor] = None, inline_scale: bool = False):
    """Per-row int8 codes and f32 scales of key rows [n, d]: x ~= scale[:, None] * q8.

    inline_scale: each row's scale is stored in bytes d .. d+3 of its code row (rows of
    ceil((d + 4) / 16) * 16 bytes); returns (rows [n, that width] int8, None)."""
    _need_cuda(x, q8, scale)
    n, d = x.shape[0], x.shape[-1]
    if inline_scale:
        if q8 is None:
            q8 = torch.empty(n, (d + 4 + 15) // 16 * 16, device=x.device, dtype=torch.int8)
        _check(load().idx_quantize_rows(_ptr(x), _dtype(x), n, d, x.stride(0), _ptr(q8), q8.stride(0), None,
                                        _stream(x.device)))
        return q8, None
    if q8 is None:
        q8 = torch.empty(n, (d + 15) // 16 * 16, device=x.device, dtype=torch.int8)[:, :d]
    if scale is None:
        scale = torch.empty(n, device=x.device, dtype=torch.float32)
    _check(load().idx_quantize_rows(_ptr(x), _dtype(x), n, d, x.stride(0), _ptr(q8), q8.stride(0), _ptr(scale),
                                    _stream(x.device)))
    return q8, scale


def inline_scales(rows: torch.Tensor, d: int) -> torch.Tensor:
    """The f32 scales stored inline (bytes d .. d+3) in int8 code rows written with inline_scale."""
    return rows[:, d:d + 4].contiguous().view(torch.float32).view(-1)


def idx_score_q8(q: torch.Tensor, w: torch.Tensor, k8: torch.Tensor, k_scale: Optional[torch.Tensor],
                 batch: Batch, *, scores: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Indexer scores over an int8 key cache with per-row scales (f32 [rows, keys]);
    k_scale None: the scales are inline in the rows (idx_quantize_rows(..., inline_scale=True))."""
    _need_cuda(q, w, k8, k_scale, scores)
    H, d = q.shape[-2], q.shape[-1]
    rows = batch.n_rows
    if scores is None:
        scores = torch.empty(rows, max(batch.max_n_kv, 1), device=q.device, dtype=torch.float32)
    _check(load().idx_score_q8(_ptr(q), _dtype(q), _ptr(w), H, d, _ptr(k8), k8.stride(0), _ptr(k_scale),
                               k8.shape[0], batch.c(), 0, _ptr(scores), scores.stride(0), None, 0,
                               _stream(q.device)))
    return scores


def idx_block_pool_update(k_raw: torch.Tensor, batch: Batch, block_size: int, pooled: torch.Tensor, *,
                          n_pooled: Optional[torch.Tensor] = None, stale_pos: Optional[torch.Tensor] = None,
                          pool_seq_stride: Optional[int] = None) -> torch.Tensor:
    """(Re)pool only the blocks from min(n_pooled[b], stale_pos[b] // C) on, in place in ``pooled``.

    n_pooled / stale_pos: device int32 [n_seq] or None (0 / no edit); IDX_POS_CLEAN marks no edit.
    """
    _need_cuda(k_raw, pooled, n_pooled, stale_pos)
    d = k_raw.shape[-1]
    if pool_seq_stride is None:
        pool_seq_stride = pooled.shape[1] if pooled.dim() == 3 else max(batch.max_n_kv // block_size, 1)
    for t in (n_pooled, stale_pos):
        if t is not None and (t.dtype != torch.int32 or t.numel() < batch.n_seq or not t.is_contiguous()):
            raise ValueError("n_pooled / stale_pos must be contiguous int32 with one entry per sequence")
    _check(load().idx_block_pool_update(_ptr(k_raw), _dtype(k_raw), k_raw.stride(0), k_raw.shape[0], batch.c(),
                                        _ptr(n_pooled), _ptr(stale_pos), block_size, d, _ptr(pooled),
                                        pool_seq_stride, _stream(k_raw.device)))
    return pooled


def idx_topk(scores: torch.Tensor, batch: Batch, top_k: int, *, block_size: int = 0,
             idx: Optional[torch.Tensor] = None, n_sel: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None):
    """Selected positions (ascending, -1 padded) and their count per row."""
    _need_cuda(scores, idx, n_sel, workspace)
    rows = batch.n_rows
    cap = topk_capacity(top_k, block_size)
    if idx is None:
        idx = torch.empty(rows, cap, device=scores.device, dtype=torch.int32)
    if n_sel is None:
        n_sel = torch.empty(rows, device=scores.device, dtype=torch.int32)
    if workspace is None and block_size <= 1:
        need = idx_workspace_size(IDX_OP_TOPK, rows, batch.max_n_kv, top_k)
        if need:
            workspace = torch.empty(need, device=scores.device, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().idx_topk(_ptr(scores), scores.stride(0), batch.c(), top_k, block_size, _ptr(idx),
                           idx.stride(0), _ptr(n_sel), _ptr(workspace), ws_bytes, _stream(scores.device)))
    return idx, n_sel


def _attn(fn_name, q, k, v, batch, idx, n_sel, scale, out, out_dtype, workspace, n_kv_heads, dv):
    _need_cuda(q, k, v, idx, n_sel, out, workspace)
    rows, Hq, dk = q.shape
    assert rows == batch.n_rows and q.is_contiguous()
    if v is None:
        hkv, dv = 1, (dv if dv is not None else 512)
        kv_row_stride = k.stride(0)
        v_row_stride = 0
    else:
        hkv = n_kv_heads if n_kv_heads is not None else k.shape[1]
        dv = v.shape[-1]
        kv_row_stride = k.stride(0)
        v_row_stride = v.stride(0)
    if out is None:
        out = torch.empty(rows, Hq, dv, device=q.device, dtype=out_dtype)
    if workspace is None:
        op = IDX_OP_ATTN_PREFILL if fn_name == "sparse_attn_prefill" else IDX_OP_ATTN_DECODE
        need = idx_workspace_size(op, rows, batch.max_n_kv, idx.stride(0), Hq, dv)
        if need:
            workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    fn = getattr(load(), fn_name)
    _check(fn(_ptr(q), _dtype(q), Hq, hkv, dk, dv, _ptr(k), _ptr(v), kv_row_stride, v_row_stride,
              k.shape[0], batch.c(), _ptr(idx), idx.stride(0), _ptr(n_sel), float(scale), _ptr(out),
              _dtype(out), _ptr(workspace), ws_bytes, _stream(q.device)))
    return out


def sparse_attn_decode(q, k, v, batch, idx, n_sel, scale, *, out=None, out_dtype=torch.float32,
                       workspace=None, n_kv_heads=None, dv=None):
    """Attention over the selected keys.  q [B*T, Hq, dk]; k [rows, Hkv, dk] (or the MLA latent
    [rows, 576] with v=None and dv=512); v [rows, Hkv, dv] or None."""
    return _attn("sparse_attn_decode", q, k, v, batch, idx, n_sel, scale, out, out_dtype, workspace,
                 n_kv_heads, dv)


def sparse_attn_prefill(q, k, v, batch, idx, n_sel, scale, *, out=None, out_dtype=torch.float32,
                        workspace=None, n_kv_heads=None, dv=None):
    """Same function as sparse_attn_decode, tuned for many query rows."""
    return _attn("sparse_attn_prefill", q, k, v, batch, idx, n_sel, scale, out, out_dtype, workspace,
                 n_kv_heads, dv)


def idx_block_score_topk(q: torch.Tensor, w: torch.Tensor, k_raw: torch.Tensor, batch: Batch, block_size: int,
                         pooled: torch.Tensor, top_k: int, *, n_pooled: Optional[torch.Tensor] = None,
                         stale_pos: Optional[torch.Tensor] = None, pool_seq_stride: Optional[int] = None,
                         scores: Optional[torch.Tensor] = None, idx: Optional[torch.Tensor] = None,
                         n_sel: Optional[torch.Tensor] = None):
    """The indexer of a block-pooled decode step in one call: (scores, idx, n_sel) exactly as
    idx_block_pool_update + idx_score over ``pooled`` + idx_topk in block mode give them; ``pooled``
    is updated in place."""
    _need_cuda(q, w, k_raw, pooled, n_pooled, stale_pos, scores, idx, n_sel)
    rows, H, d = q.shape
    assert rows == batch.n_rows and w.shape == (rows, H) and w.dtype == torch.float32
    assert q.is_contiguous() and w.is_contiguous() and k_raw.stride(-1) == 1
    assert pooled.dtype == torch.float32 and pooled.is_contiguous()
    if pool_seq_stride is None:
        pool_seq_stride = pooled.shape[1] if pooled.dim() == 3 else max(batch.max_n_kv // block_size, 1)
    for t in (n_pooled, stale_pos):
        if t is not None and (t.dtype != torch.int32 or t.numel() < batch.n_seq or not t.is_contiguous()):
            raise ValueError("n_pooled / stale_pos must be contiguous int32 with one entry per sequence")
    kk = 2048 if top_k == -1 else top_k
    if scores is None:
        scores = torch.empty(rows, max(batch.max_n_kv // block_size, 1), device=q.device, dtype=torch.float32)
    if idx is None:
        idx = torch.empty(rows, topk_capacity(kk, block_size), device=q.device, dtype=torch.int32)
    if n_sel is None:
        n_sel = torch.empty(rows, device=q.device, dtype=torch.int32)
    _check(load().idx_block_score_topk(_ptr(q), _dtype(q), _ptr(w), H, d, _ptr(k_raw), _dtype(k_raw), k_raw.stride(0),
                                       k_raw.shape[0], batch.c(), _ptr(n_pooled), _ptr(stale_pos), block_size,
                                       _ptr(pooled), pool_seq_stride, top_k, _ptr(scores), scores.stride(0), _ptr(idx),
                                       idx.stride(0), _ptr(n_sel), _stream(q.device)))
    return scores, idx, n_sel


def idx_score_topk(q: torch.Tensor, w: torch.Tensor, k: torch.Tensor, batch: Batch, top_k: int, *,
                   scores: Optional[torch.Tensor] = None, idx: Optional[torch.Tensor] = None,
                   n_sel: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """The fused indexer + selection (token keys): (scores, idx, n_sel) exactly as idx_score followed
    by idx_topk would give them."""
    _need_cuda(q, w, k, scores, idx, n_sel, workspace)
    rows, H, d = q.shape
    assert rows == batch.n_rows and w.shape == (rows, H) and w.dtype == torch.float32
    assert q.is_contiguous() and w.is_contiguous() and k.stride(-1) == 1
    kk = 2048 if top_k == -1 else top_k
    if scores is None:
        scores = torch.empty(rows, max(batch.max_n_kv, 1), device=q.device, dtype=torch.float32)
    if idx is None:
        idx = torch.empty(rows, kk, device=q.device, dtype=torch.int32)
    if n_sel is None:
        n_sel = torch.empty(rows, device=q.device, dtype=torch.int32)
    if workspace is None:
        need = idx_workspace_size(IDX_OP_SCORE_TOPK, rows, batch.max_n_kv, top_k)
        if need:
            workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().idx_score_topk(_ptr(q), _dtype(q), _ptr(w), H, d, _ptr(k), _dtype(k), k.stride(0), k.shape[0],
                                 batch.c(), top_k, _ptr(scores), scores.stride(0), _ptr(idx), idx.stride(0),
                                 _ptr(n_sel), _ptr(workspace), ws_bytes, _stream(q.device)))
    return scores, idx, n_sel


def sparse_decode_step(q: torch.Tensor, w: torch.Tensor, k: torch.Tensor, batch: Batch, top_k: int,
                       q_attn: torch.Tensor, k_attn: torch.Tensor, v_attn: Optional[torch.Tensor], scale: float, *,
                       dv: Optional[int] = None, scores: Optional[torch.Tensor] = None,
                       idx: Optional[torch.Tensor] = None, n_sel: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                       workspace: Optional[torch.Tensor] = None):
    """One decode step: idx_score_topk then sparse_attn_decode (one launch for few short rows).
    Returns (scores, idx, n_sel, out)."""
    _need_cuda(q, w, k, q_attn, k_attn, v_attn, scores, idx, n_sel, out, workspace)
    rows, H, d = q.shape
    assert rows == batch.n_rows and w.shape == (rows, H) and w.dtype == torch.float32
    assert q.is_contiguous() and w.is_contiguous() and k.stride(-1) == 1 and q_attn.is_contiguous()
    _, Hq, dk = q_attn.shape
    if v_attn is None:
        hkv, dv = 1, (dv if dv is not None else 512)
        v_row_stride = 0
    else:
        hkv, dv = k_attn.shape[1], v_attn.shape[-1]
        v_row_stride = v_attn.stride(0)
    kk = 2048 if top_k == -1 else top_k
    if scores is None:
        scores = torch.empty(rows, max(batch.max_n_kv, 1), device=q.device, dtype=torch.float32)
    if idx is None:
        idx = torch.empty(rows, kk, device=q.device, dtype=torch.int32)
    if n_sel is None:
        n_sel = torch.empty(rows, device=q.device, dtype=torch.int32)
    if out is None:
        out = torch.empty(rows, Hq, dv, device=q.device, dtype=out_dtype)
    if workspace is None:
        need = idx_workspace_size(IDX_OP_DECODE_STEP, rows, batch.max_n_kv, top_k, Hq, dv)
        if need:
            workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().sparse_decode_step(_ptr(q), _dtype(q), _ptr(w), H, d, _ptr(k), _dtype(k), k.stride(0), k.shape[0],
                                     batch.c(), top_k, _ptr(scores), scores.stride(0), _ptr(idx), idx.stride(0),
                                     _ptr(n_sel), _ptr(q_attn), _dtype(q_attn), Hq, hkv, dk, dv, _ptr(k_attn),
                                     _ptr(v_attn), k_attn.stride(0), v_row_stride, k_attn.shape[0], float(scale),
                                     _ptr(out), _dtype(out), _ptr(workspace), ws_bytes, _stream(q.device)))
    return scores, idx, n_sel, out


def sparse_decode_step_fused(n_rows: int, n_q_per_seq: int, max_n_kv: int, top_k: int, idx_row_stride: int) -> bool:
    """Whether sparse_decode_step runs as one launch for these sizes on the current device."""
    return bool(load().sparse_decode_step_fused(n_rows, n_q_per_seq, max_n_kv, top_k, idx_row_stride))


def sparse_attn_decode_noalloc(q, latent, batch, idx, n_sel, scale, *, out=None, out_dtype=torch.bfloat16):
    """The 128-head MLA decode attention without a workspace, for callers that cannot
    allocate device memory: its key-split scratch is a static array inside the library
    (see include/lidx.h).  Calls that overlap on the GPU must be serialised."""
    _need_cuda(q, latent, idx, n_sel, out)
    rows, Hq, dk = q.shape
    assert rows == batch.n_rows and q.is_contiguous()
    if out is None:
        out = torch.empty(rows, Hq, 512, device=q.device, dtype=out_dtype)
    _check(load().sparse_attn_decode_noalloc(_ptr(q), _dtype(q), Hq, 1, dk, 512, _ptr(latent), latent.stride(0),
                                             latent.shape[0], batch.c(), _ptr(idx), idx.stride(0), _ptr(n_sel),
                                             float(scale), _ptr(out), _dtype(out), _stream(q.device)))
    return out


class _On:
    """Makes `device` current for a call."""

    def __init__(self, device):
        self.prev, self.idx = torch.cuda.current_device(), device.index

    def __enter__(self):
        if self.prev != self.idx:
            torch.cuda.set_device(self.idx)

    def __exit__(self, *exc):
        if self.prev != self.idx:
            torch.cuda.set_device(self.prev)


def _all_on(device, *ts):
    for t in ts:
        if t is not None and t.device != device:
            _need_cuda(t)
            raise ValueError(f"tensors on {device} and {t.device}: lidx works on one device per call")


def _i32(name: str, t: torch.Tensor, n: int):
    if t.dtype is not torch.int32 or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of at least {n} entries")
    return t.data_ptr()


def dense_attn_workspace_size(dtype: torch.dtype, n_seq: int, n_q_per_seq: int, max_n_kv: int, n_q_heads: int,
                              n_kv_heads: int, dk: int, dv: int) -> int:
    """Bytes of workspace with which dense_attn splits the keys as it would like to."""
    return int(load().dense_attn_workspace_size(_DTYPES[dtype], n_seq, n_q_per_seq, max_n_kv, n_q_heads, n_kv_heads,
                                                dk, dv))


def dense_attn(q: torch.Tensor, k: torch.Tensor, v: Optional[torch.Tensor], batch: Batch, scale: float, *,
               softcap: float = 0.0, slopes: Optional[torch.Tensor] = None, window: int = 0,
               prefix_len: Optional[torch.Tensor] = None, doc_start: Optional[torch.Tensor] = None,
               prefix_end: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, dv: Optional[int] = None) -> torch.Tensor:
    """Attention of a chunk of new tokens (batch.n_q_per_seq rows per sequence, 1 = decode) over every key
    its rows see in a contiguous or paged cache.  q [B*T, Hq, dk]; k [rows, Hkv, dk] and v [rows, Hkv, dv],
    or the MLA latent [rows, dk] with v=None (dv columns of it, 512 unless given).  Returns out
    [B*T, Hq, dv] of q's dtype; lse, if given (f32 [B*T, Hq]), gets the log of the rows' softmax sums.

    Row r sees positions up to batch.q_pos[r] (none if that is negative: a padding row, whose out is
    zero), or up to prefix_len[b] or prefix_end[r] where that is further; not before doc_start[r]; with window,
    at most that many positions up to its own.  (prefix_len is the sequence's and runs on into later documents;
    documents with prefixes of their own take prefix_end, the position behind that of the row's document.)  softcap c > 0: scores x become c * tanh(x / c); slopes (f32 [Hq]):
    minus slopes[h] * |q_pos[r] - j| for key j."""
    dev = q.device
    _need_cuda(q)
    _all_on(dev, k, v, out, lse, workspace, batch.n_kv, batch.q_pos, batch.page_table, batch.kv_start)
    b = batch.c()
    rows = b.n_seq * b.n_q_per_seq
    # (kv_start is not read beside a page table)
    where, n = (batch.kv_start, b.n_seq) if batch.page_table is None else (batch.page_table, b.n_seq * b.page_table_stride)
    if batch.q_pos is not None and batch.q_pos.numel() < rows or where is not None and where.numel() < n:
        raise ValueError("q_pos, kv_start or page_table has fewer entries than the batch")
    if q.dim() != 3 or q.shape[0] != rows or not q.is_contiguous():
        raise ValueError("q must be a contiguous [n_seq * n_q_per_seq, heads, dk] tensor")
    _, Hq, dk = q.shape
    if v is None:
        if k.dim() == 3 and k.shape[1] == 1:
            k = k[:, 0]
        if k.dim() != 2 or k.shape[1] < dk or k.stride(1) != 1:
            raise ValueError("the latent cache must be [rows, dk] with contiguous rows")
        hkv, dv, v_row_stride, v_ptr = 1, (512 if dv is None else dv), 0, None
    else:
        if k.dim() != 3 or v.dim() != 3:
            raise ValueError("k and v must be [rows, kv heads, dk] and [rows, kv heads, dv]")
        n, hkv, d = k.shape
        nv, hkv_v, d_v = v.shape
        if n != nv or hkv != hkv_v or d != dk:
            raise ValueError("k and v must be [rows, kv heads, dk] and [rows, kv heads, dv]")
        if dv is not None and dv != d_v:
            raise ValueError("dv differs from v's last dimension")
        dv = d_v
        ks, vs = k.stride(), v.stride()
        if ks[2] != 1 or vs[2] != 1 or (hkv > 1 and (ks[1] != dk or vs[1] != dv)):
            raise ValueError("the heads of a cache row must be contiguous")
        # an empty cache has no address; v's tells the latent form apart and is not read
        v_row_stride, v_ptr = vs[0], v.data_ptr() or q.data_ptr()
    dt = _dtype(q)
    if k.dtype is not q.dtype or (v is not None and v.dtype is not q.dtype):
        raise ValueError("q, k and v must have the same dtype")
    mods = None
    if not -2**31 <= window < 2**31:
        raise ValueError("window must be below 2**31")
    if softcap and not ctypes.c_float(softcap).value:
        raise ValueError("softcap is 0 in float32, which is no cap")
    if softcap or window or not (slopes is prefix_len is doc_start is prefix_end is None):
        _all_on(dev, slopes, prefix_len, doc_start, prefix_end)
        if slopes is not None and (slopes.dtype is not torch.float32 or not slopes.is_contiguous() or
                                   slopes.numel() != Hq):
            raise ValueError("slopes must be a contiguous float32 tensor with one entry per query head")
        mods = _Mods(softcap, None if slopes is None else slopes.data_ptr(), window,
                     None if prefix_len is None else _i32("prefix_len", prefix_len, b.n_seq),
                     None if doc_start is None else _i32("doc_start", doc_start, rows),
                     None if prefix_end is None else _i32("prefix_end", prefix_end, rows))
    if out is None:
        out = torch.empty((rows, Hq, dv), device=dev, dtype=q.dtype)
    elif out.shape != (rows, Hq, dv) or out.dtype is not q.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous [rows, heads, dv] tensor of q's dtype")
    if lse is not None and (lse.shape != (rows, Hq) or lse.dtype is not torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [rows, heads] tensor")
    lib = load()
    with _On(dev):
        if workspace is None:
            need = lib.dense_attn_workspace_size(dt, b.n_seq, b.n_q_per_seq, b.max_n_kv, Hq, hkv, dk, dv)
            if need:
                workspace = torch.empty(need, device=dev, dtype=torch.uint8)
        _check(lib.dense_attn(q.data_ptr(), dt, Hq, hkv, dk, dv, k.data_ptr(), v_ptr, k.stride(0), v_row_stride, k.shape[0],
                              b, mods, scale, out.data_ptr(), None if lse is None else lse.data_ptr(), *_space(workspace),
                              _stream(dev)))
    return out


def _space(workspace: Optional[torch.Tensor]):
    """(address, bytes) of a workspace."""
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous():
        raise ValueError("a workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _page_caches(caches, page_size: int, device):
    """(ctypes array of cache descriptions, pages in each) of caches sharing page numbers."""
    n = len(caches)
    if not 1 <= n <= IDX_MAX_PAGE_CACHES:
        raise ValueError(f"1 to {IDX_MAX_PAGE_CACHES} caches share a page table")
    if page_size < 1:
        raise ValueError("page_size < 1")
    flat = []
    n_pages = -1
    for c in caches:
        if c.device != device:
            _all_on(device, c)
        rows, *shape = c.shape
        stride, *inner = c.stride()
        if n_pages < 0:
            n_pages = rows // page_size
        elif rows // page_size != n_pages:
            raise ValueError("the caches must hold the same number of pages")
        width = 1
        for d, st in zip(reversed(shape), reversed(inner)):
            if d != 1 and st != width:
                raise ValueError("the elements of a cache row must be contiguous")
            width *= d
        if stride < width:
            if rows > 1:
                raise ValueError("the rows of a cache must not overlap")
            stride = width
        size = c.element_size()
        flat.append((c.data_ptr(), stride * size, width * size))
    return (_PageCache * n)(*flat), n_pages


def idx_page_workspace_size(n_seq: int, n_pages: int) -> int:
    return int(load().idx_page_workspace_size(n_seq, n_pages))


def idx_page_copy(caches, page_size: int, src: torch.Tensor, dst: torch.Tensor) -> None:
    """Copies page src[i] to page dst[i] in every cache (tensors whose dim 0 is the cache row), in place.
    The pages of dst must differ from one another and from those of src; entries below 0 are skipped."""
    dev = src.device
    _need_cuda(src)
    _all_on(dev, dst)
    arr, n_pages = _page_caches(caches, page_size, dev)
    n = src.numel()
    if dst.numel() != n:
        raise ValueError("src and dst must have the same length")
    s, d = _i32("src", src, n), _i32("dst", dst, n)
    with _On(dev):
        _check(load().idx_page_copy(arr, len(caches), page_size, n_pages, s, d, n,
                                    _stream(dev)))


def _table(name: str, t: torch.Tensor):
    if t.dim() != 2 or t.dtype is not torch.int32:
        raise ValueError(f"{name} must be an int32 [sequences, pages] tensor with contiguous rows")
    rows, cols = t.shape
    s0, s1 = t.stride()
    if (cols > 1 and s1 != 1) or (rows > 1 and s0 < cols):
        raise ValueError(f"{name} must be an int32 [sequences, pages] tensor with contiguous rows")
    return t.data_ptr(), max(s0, cols), rows, cols


def _held(held, n_pages):
    if held is None:
        return None
    if held.dtype not in (torch.uint8, torch.bool) or not held.is_contiguous() or held.numel() != n_pages:
        raise ValueError("held must be a contiguous uint8 or bool tensor with one entry per page")
    return held.data_ptr()


def idx_page_update(page_table: torch.Tensor, parent: torch.Tensor, n_keep: torch.Tensor, n_new: torch.Tensor,
                    page_size: int, caches, *, held: Optional[torch.Tensor] = None,
                    new_table: Optional[torch.Tensor] = None, n_free: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None):
    """One step's frees, truncations, forks and growth of the sequences over a page table: row b of the
    new table is the first n_keep[b] positions of row parent[b] of the old one (-1: nothing), with pages
    for n_new[b] positions.  Whole pages are shared, a shared last page is copied in every cache, new pages
    are the lowest free ones (neither named by a new row nor held).  Returns (new_table, n_free): n_free
    (int32 [1], on the device) is the number of pages left, minus the number missing if there were too few
    (new_table is then not written), or -2**31 if a request was impossible."""
    dev = page_table.device
    _need_cuda(page_table)
    _all_on(dev, parent, n_keep, n_new, held, new_table, n_free, workspace)
    arr, n_pages = _page_caches(caches, page_size, dev)
    old, stride, n_old, cols = _table("page_table", page_table)
    n = parent.numel()
    if n_keep.numel() != n or n_new.numel() != n:
        raise ValueError("parent, n_keep and n_new must have the same length")
    par, keep, new = _i32("parent", parent, n), _i32("n_keep", n_keep, n), _i32("n_new", n_new, n)
    h = _held(held, n_pages)
    if new_table is None:
        new_table = torch.empty((n, cols), device=dev, dtype=torch.int32)
    out, new_stride, n_rows, new_cols = _table("new_table", new_table)
    if n_rows != n:
        raise ValueError("new_table must have one row per entry of parent")
    if n_free is None:
        n_free = torch.empty(1, device=dev, dtype=torch.int32)
    lib = load()
    with _On(dev):
        if workspace is None:
            workspace = torch.empty(max(lib.idx_page_workspace_size(n, n_pages), 16), device=dev, dtype=torch.uint8)
        _check(lib.idx_page_update(old, stride, cols, n_old, par, keep, new, n, page_size, n_pages, h, out, new_stride,
                                   new_cols, _i32("n_free", n_free, 1), arr, len(caches), *_space(workspace),
                                   _stream(dev)))
    return new_table, n_free


def idx_page_compact(page_table: torch.Tensor, n_len: torch.Tensor, page_size: int, caches, *,
                     held: Optional[torch.Tensor] = None, new_table: Optional[torch.Tensor] = None,
                     n_used: Optional[torch.Tensor] = None, remap: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None):
    """Moves the used pages (those of the first n_len[b] positions of each row; held ones stay where they
    are) to the lowest numbers, in every cache.  Returns (new_table, n_used, remap): n_used (int32 [1], on
    the device) counts the used and held pages, remap[p] is the new number of page p.  new_table may be
    page_table itself."""
    dev = page_table.device
    _need_cuda(page_table)
    _all_on(dev, n_len, held, new_table, n_used, remap, workspace)
    arr, n_pages = _page_caches(caches, page_size, dev)
    old, stride, n, cols = _table("page_table", page_table)
    if n_len.numel() != n:
        raise ValueError("n_len must have one entry per row of page_table")
    lens = _i32("n_len", n_len, n)
    h = _held(held, n_pages)
    if new_table is None:
        new_table = torch.empty((n, cols), device=dev, dtype=torch.int32)
    elif new_table.shape != page_table.shape:
        raise ValueError("new_table must have page_table's shape")
    out, new_stride, _, _ = _table("new_table", new_table)
    if n_used is None:
        n_used = torch.empty(1, device=dev, dtype=torch.int32)
    if remap is None:
        remap = torch.empty(n_pages, device=dev, dtype=torch.int32)
    lib = load()
    with _On(dev):
        if workspace is None:
            workspace = torch.empty(max(lib.idx_page_workspace_size(n, n_pages), 16), device=dev, dtype=torch.uint8)
        _check(lib.idx_page_compact(old, stride, cols, n, lens, page_size, n_pages, h, out, new_stride,
                                    _i32("n_used", n_used, 1), _i32("remap", remap, n_pages), arr, len(caches),
                                    *_space(workspace), _stream(dev)))
    return new_table, n_used, remap


def idx_device_status(reset: bool = True) -> int:
    """Synchronise and return the device fault word (0 = none)."""
    return int(load().idx_device_status(1 if reset else 0))
