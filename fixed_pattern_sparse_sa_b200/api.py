"""Thin torch binding over libsa.so.

Argument marshalling only: every function checks dtypes, devices and
contiguity, allocates outputs and workspace with torch, and calls the C entry
point of the same name on the current CUDA stream.  All computation happens in
the library's kernels; there is no CPU path.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import SAError, check, sa_dsa_layer, sa_pattern

__all__ = ["indexer_topk", "sparse_attn_fwd", "sparse_attn_bwd", "sparse_attn_fwd_split_static", "lse_combine",
           "nsa_fwd", "sink_attn_fwd", "sink_attn_bwd", "paged_attn_decode", "paged_extend", "paged_write",
           "paged_fork", "paged_free", "paged_compact", "indexer_scores_at", "topk_merge", "index_shard",
           "dsa_decode_layers", "check_device_status", "debug_set_spin_limit", "debug_inject_stall",
           "debug_exact_recompute_rows", "SAError"]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t: Optional[torch.Tensor], name: str, dtype, dev=None, ndim=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _workspace(nbytes: int, device) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def check_device_status(device=None):
    """Wait for the current stream and raise if a kernel found a bad index
    (SA_ERR_DEVICE_ASSERT) or stopped on a bounded wait (SA_ERR_TIMEOUT)."""
    lib = _lib.load()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        check(lib.sa_check_device_status(_stream(None)), "sa_check_device_status")


def debug_set_spin_limit(cycles: int, device=None):
    """sa_debug_set_spin_limit: SM clocks a kernel's progress wait may spin
    before it reports SA_ERR_TIMEOUT; cycles <= 0 restores the default."""
    lib = _lib.load()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        check(lib.sa_debug_set_spin_limit(int(cycles)), "sa_debug_set_spin_limit")


def debug_inject_stall(on: bool, device=None):
    """sa_debug_inject_stall: make the NSA tensor-core branch kernels wait on
    a barrier that nothing completes (a test of the timeout path)."""
    lib = _lib.load()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        check(lib.sa_debug_inject_stall(1 if on else 0), "sa_debug_inject_stall")


def debug_exact_recompute_rows(device=None) -> int:
    """sa_debug_exact_recompute_rows: rows whose top-k was taken by exact
    recompute since the last call (synchronizes the device)."""
    lib = _lib.load()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        n = int(lib.sa_debug_exact_recompute_rows())
    if n < 0:
        check(-n, "sa_debug_exact_recompute_rows")
    return n


# ------------------------------------------------------------------ indexer --
def indexer_topk(q_idx, k_idx, w, topk: int, window: int = 0,
                 q_pos0: Optional[int] = None, out_idx=None, out_count=None, workspace=None):
    """Exact causal top-k of the lightweight indexer (sa_indexer_topk).

    q_idx int8 [B,Tq,Hi,di], k_idx int8 [B,L,di], w int32 [B,Tq,Hi].
    q_pos0 defaults to L - Tq (the queries are the last Tq positions).
    Returns (idx int32 [B,Tq,topk+window], count int32 [B,Tq]).
    """
    lib = _lib.load()
    dev = q_idx.device
    _need(q_idx, "q_idx", torch.int8, dev, 4)
    _need(k_idx, "k_idx", torch.int8, dev, 3)
    _need(w, "w", torch.int32, dev, 3)
    B, Tq, Hi, di = q_idx.shape
    L = k_idx.shape[1]
    if k_idx.shape != (B, L, di) or w.shape != (B, Tq, Hi):
        raise ValueError("indexer_topk: shape mismatch")
    pos0 = L - Tq if q_pos0 is None else int(q_pos0)
    K = topk + window
    if out_idx is None:
        out_idx = torch.empty((B, Tq, K), dtype=torch.int32, device=dev)
    if out_count is None:
        out_count = torch.empty((B, Tq), dtype=torch.int32, device=dev)
    nbytes = lib.sa_indexer_topk_workspace_size(B, Tq, L, Hi, di, topk, window)
    ws = workspace if (workspace is not None and workspace.numel() >= nbytes) \
        else _workspace(nbytes, dev)
    with torch.cuda.device(dev):
        check(lib.sa_indexer_topk(_ptr(q_idx), _ptr(k_idx), _ptr(w), B, Tq, L, Hi, di, pos0,
                                  topk, window, _ptr(out_idx), _ptr(out_count), _ptr(ws),
                                  nbytes, _stream(dev)), "sa_indexer_topk")
    return out_idx, out_count


# ---------------------------------------------------------------- attention --
def sparse_attn_fwd(q, k, v, idx=None, pattern: Optional[Sequence[int]] = None,
                    cq=None, ck=None, beta=None, scale: Optional[float] = None,
                    n_split: int = 1, q_pos0: Optional[int] = None,
                    return_partials: bool = False, out=None, lse=None):
    """Gathered-KV sparse attention (sa_sparse_attn_fwd).

    q bf16 [B,Tq,Hq,d], k/v bf16 [B,L,Hkv,d]; idx int32 [B,Tq,K] or
    [B,Tq,idx_heads,K] (-1 padded), or pattern = (window, dilated).
    Optional coordinate bias cq fp32 [B,Tq,Hq,3], ck fp32 [B,L,Hkv,3],
    beta fp32 [Hq].  Returns (out bf16 [B,Tq,Hq,d], lse fp32 [B,Tq,Hq]) and,
    with return_partials (n_split > 1), also (part_o, part_lse).
    """
    lib = _lib.load()
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 4)
    _need(k, "k", torch.bfloat16, dev, 4)
    _need(v, "v", torch.bfloat16, dev, 4)
    B, Tq, Hq, d = q.shape
    L, Hkv = k.shape[1], k.shape[2]
    if k.shape != (B, L, Hkv, d) or v.shape != k.shape:
        raise ValueError("sparse_attn_fwd: k/v shape mismatch")
    pos0 = L - Tq if q_pos0 is None else int(q_pos0)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    pat = None
    idx_heads, K = 1, 0
    if idx is not None:
        _need(idx, "idx", torch.int32, dev)
        if idx.dim() == 3:
            idx_heads, K = 1, idx.shape[2]
        elif idx.dim() == 4:
            idx_heads, K = idx.shape[2], idx.shape[3]
        else:
            raise ValueError("idx must be [B,Tq,K] or [B,Tq,idx_heads,K]")
        if idx.shape[:2] != (B, Tq):
            raise ValueError("idx shape mismatch")
    elif pattern is not None:
        pat = sa_pattern(int(pattern[0]), int(bool(pattern[1])))
    else:
        raise ValueError("need idx or pattern")
    if cq is not None or ck is not None or beta is not None:
        _need(cq, "cq", torch.float32, dev, 4)
        _need(ck, "ck", torch.float32, dev, 4)
        _need(beta, "beta", torch.float32, dev, 1)
    if out is None:
        out = torch.empty((B, Tq, Hq, d), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, Tq, Hq), dtype=torch.float32, device=dev)
    po = pl = None
    if n_split > 1:
        po = torch.empty((n_split, B, Tq, Hq, d), dtype=torch.float32, device=dev)
        pl = torch.empty((n_split, B, Tq, Hq), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        check(lib.sa_sparse_attn_fwd(
            _ptr(q), _ptr(k), _ptr(v), B, Tq, L, Hq, Hkv, d, pos0,
            _ptr(idx), idx_heads, K, ctypes.byref(pat) if pat is not None else None,
            _ptr(cq), _ptr(ck), _ptr(beta), float(scale), int(n_split),
            _ptr(out), _ptr(lse), _ptr(po), _ptr(pl), None, 0, _stream(dev)),
            "sa_sparse_attn_fwd")
    if return_partials:
        return out, lse, po, pl
    return out, lse


def sparse_attn_fwd_split_static(q, k, v, idx, n_split: int, scale: Optional[float] = None,
                                 q_pos0: Optional[int] = None, out=None, lse=None):
    """Split-KV sparse attention over index lists that allocates no device
    memory (sa_sparse_attn_fwd_split_static).

    For callers that cannot allocate at call time; the partial results live in
    a fixed 8 MiB array inside the library, so n_split*B*Tq*Hq*(d+1)*4 bytes
    must fit in it, and calls that may overlap on the GPU must be ordered by
    the caller.  Pass out/lse to allocate nothing here either.
    """
    lib = _lib.load()
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 4)
    _need(k, "k", torch.bfloat16, dev, 4)
    _need(v, "v", torch.bfloat16, dev, 4)
    _need(idx, "idx", torch.int32, dev)
    B, Tq, Hq, d = q.shape
    L, Hkv = k.shape[1], k.shape[2]
    if k.shape != (B, L, Hkv, d) or v.shape != k.shape:
        raise ValueError("sparse_attn_fwd_split_static: k/v shape mismatch")
    if idx.dim() == 3:
        idx_heads, K = 1, idx.shape[2]
    elif idx.dim() == 4:
        idx_heads, K = idx.shape[2], idx.shape[3]
    else:
        raise ValueError("idx must be [B,Tq,K] or [B,Tq,idx_heads,K]")
    pos0 = L - Tq if q_pos0 is None else int(q_pos0)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, Tq, Hq, d), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, Tq, Hq), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        check(lib.sa_sparse_attn_fwd_split_static(
            _ptr(q), _ptr(k), _ptr(v), B, Tq, L, Hq, Hkv, d, pos0, _ptr(idx), idx_heads, K,
            float(scale), int(n_split), _ptr(out), _ptr(lse), _stream(dev)),
            "sa_sparse_attn_fwd_split_static")
    return out, lse


def sparse_attn_bwd(q, k, v, out, lse, dout, idx, scale: Optional[float] = None,
                    q_pos0: Optional[int] = None):
    """Backward of sparse_attn_fwd over explicit index lists (sa_sparse_attn_bwd).

    q, out, dout bf16 [B,Tq,Hq,d]; k, v bf16 [B,L,Hkv,d]; lse fp32 [B,Tq,Hq]
    (the forward's); idx int32 [B,Tq,K] or [B,Tq,idx_heads,K].
    Returns (dq fp32 [B,Tq,Hq,d], dk fp32 [B,L,Hkv,d], dv fp32 [B,L,Hkv,d]).
    """
    lib = _lib.load()
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _need(t, n, torch.bfloat16, dev, 4)
    _need(lse, "lse", torch.float32, dev, 3)
    _need(idx, "idx", torch.int32, dev)
    B, Tq, Hq, d = q.shape
    L, Hkv = k.shape[1], k.shape[2]
    if k.shape != (B, L, Hkv, d) or v.shape != k.shape or out.shape != q.shape or dout.shape != q.shape:
        raise ValueError("sparse_attn_bwd: shape mismatch")
    idx_heads = 1 if idx.dim() == 3 else idx.shape[2]
    K = idx.shape[-1]
    pos0 = L - Tq if q_pos0 is None else int(q_pos0)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty((B, Tq, Hq, d), dtype=torch.float32, device=dev)
    dk = torch.empty((B, L, Hkv, d), dtype=torch.float32, device=dev)
    dv = torch.empty((B, L, Hkv, d), dtype=torch.float32, device=dev)
    nbytes = lib.sa_sparse_attn_bwd_workspace_size(B, Tq, Hq)
    ws = _workspace(nbytes, dev)
    with torch.cuda.device(dev):
        check(lib.sa_sparse_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                     B, Tq, L, Hq, Hkv, d, pos0, _ptr(idx), idx_heads, K, float(scale),
                                     _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), nbytes, _stream(dev)),
              "sa_sparse_attn_bwd")
    return dq, dk, dv


def indexer_scores_at(q_idx, k_idx, w, idx):
    """Exact indexer scores of listed keys (sa_indexer_scores_at).

    q_idx int8 [B,Tq,Hi,di], k_idx int8 [B,L,di], w int32 [B,Tq,Hi],
    idx int32 [B,Tq,K] (-1 = none).  Returns int32 [B,Tq,K] (INT_MIN for -1).
    """
    lib = _lib.load()
    dev = q_idx.device
    _need(q_idx, "q_idx", torch.int8, dev, 4)
    _need(k_idx, "k_idx", torch.int8, dev, 3)
    _need(w, "w", torch.int32, dev, 3)
    _need(idx, "idx", torch.int32, dev, 3)
    B, Tq, Hi, di = q_idx.shape
    out = torch.empty(idx.shape, dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        check(lib.sa_indexer_scores_at(_ptr(q_idx), _ptr(k_idx), _ptr(w), B, Tq, k_idx.shape[1], Hi, di,
                                       _ptr(idx), idx.shape[-1], _ptr(out), _stream(dev)), "sa_indexer_scores_at")
    return out


def topk_merge(cand_score, cand_idx, part_off, topk: int, window: int, q_pos: int):
    """Exact top-k of gathered candidates (sa_topk_merge).

    cand_score / cand_idx int32 [n_parts, rows, kc] (part-local indices, -1 =
    none); part_off: n_parts ints (position of each part's index 0).  Returns
    (idx int32 [rows, topk+window] ascending, -1 padded, count int32 [rows]).
    """
    lib = _lib.load()
    dev = cand_score.device
    _need(cand_score, "cand_score", torch.int32, dev, 3)
    _need(cand_idx, "cand_idx", torch.int32, dev, 3)
    n_parts, rows, kc = cand_score.shape
    offs = (ctypes.c_int64 * n_parts)(*[int(x) for x in part_off])
    out = torch.empty((rows, topk + window), dtype=torch.int32, device=dev)
    cnt = torch.empty((rows,), dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        check(lib.sa_topk_merge(_ptr(cand_score), _ptr(cand_idx), offs, n_parts, rows, kc, topk, window,
                                int(q_pos), _ptr(out), _ptr(cnt), _stream(dev)), "sa_topk_merge")
    return out, cnt


def index_shard(idx, key_lo: int, key_hi: int):
    """Positions -> rows of the shard [key_lo, key_hi), -1 elsewhere (sa_index_shard)."""
    lib = _lib.load()
    dev = idx.device
    _need(idx, "idx", torch.int32, dev)
    out = torch.empty_like(idx)
    with torch.cuda.device(dev):
        check(lib.sa_index_shard(_ptr(idx), idx.numel(), int(key_lo), int(key_hi), _ptr(out), _stream(dev)),
              "sa_index_shard")
    return out


def lse_combine(part_o, part_lse, out=None, lse=None):
    """Log-sum-exp merge of split partials (sa_lse_combine).

    part_o fp32 [S, ..., d], part_lse fp32 [S, ...] -> (out bf16 [..., d], lse fp32 [...]).
    """
    lib = _lib.load()
    dev = part_o.device
    _need(part_o, "part_o", torch.float32, dev)
    _need(part_lse, "part_lse", torch.float32, dev)
    S, d = part_o.shape[0], part_o.shape[-1]
    lead = tuple(part_o.shape[1:-1])
    if tuple(part_lse.shape) != (S, *lead):
        raise ValueError("lse_combine: shape mismatch")
    rows = math.prod(lead)
    if out is None:
        out = torch.empty((*lead, d), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(lead, dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        check(lib.sa_lse_combine(_ptr(part_o), _ptr(part_lse), S, rows, d, _ptr(out), _ptr(lse),
                                 _stream(dev)), "sa_lse_combine")
    return out, lse


# ---------------------------------------------------------------------- NSA --
def nsa_fwd(q, k, v, gates, cmp_len: int, cmp_stride: int, sel_block: int, sel_topk: int,
            window: int, scale: Optional[float] = None, out=None):
    """NSA forward (sa_nsa_fwd): compressed, selected and window branches.

    Returns (out bf16 [B,T,Hq,d], lse_branches fp32 [B,T,Hq,3],
    sel_idx int32 [B,T,Hkv,sel_topk]).
    """
    lib = _lib.load()
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 4)
    _need(k, "k", torch.bfloat16, dev, 4)
    _need(v, "v", torch.bfloat16, dev, 4)
    _need(gates, "gates", torch.float32, dev, 4)
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, T, Hkv, d) or v.shape != k.shape or gates.shape != (B, T, Hq, 3):
        raise ValueError("nsa_fwd: shape mismatch")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, T, Hq, d), dtype=torch.bfloat16, device=dev)
    lse3 = torch.empty((B, T, Hq, 3), dtype=torch.float32, device=dev)
    sel = torch.empty((B, T, Hkv, sel_topk), dtype=torch.int32, device=dev)
    nbytes = lib.sa_nsa_workspace_size(B, T, Hq, Hkv, d, cmp_len, cmp_stride, sel_block, sel_topk)
    ws = _workspace(nbytes, dev)
    with torch.cuda.device(dev):
        check(lib.sa_nsa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(gates), B, T, Hq, Hkv, d, cmp_len,
                             cmp_stride, sel_block, sel_topk, window, float(scale), _ptr(out),
                             _ptr(lse3), _ptr(sel), _ptr(ws), nbytes, _stream(dev)), "sa_nsa_fwd")
    return out, lse3, sel


def nsa_fwd_train(q, k, v, gates, cmp_len: int, cmp_stride: int, sel_block: int, sel_topk: int,
                  window: int, scale: Optional[float] = None):
    """NSA forward that also returns what the backward needs (sa_nsa_fwd_train).

    Returns (out bf16 [B,T,Hq,d], lse_branches fp32 [B,T,Hq,3],
    sel_idx int32 [B,T,Hkv,sel_topk], o_branches fp32 [3,B,T,Hq,d]).
    """
    lib = _lib.load()
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 4)
    _need(k, "k", torch.bfloat16, dev, 4)
    _need(v, "v", torch.bfloat16, dev, 4)
    _need(gates, "gates", torch.float32, dev, 4)
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, T, Hkv, d) or v.shape != k.shape or gates.shape != (B, T, Hq, 3):
        raise ValueError("nsa_fwd_train: shape mismatch")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out = torch.empty((B, T, Hq, d), dtype=torch.bfloat16, device=dev)
    lse3 = torch.empty((B, T, Hq, 3), dtype=torch.float32, device=dev)
    sel = torch.empty((B, T, Hkv, sel_topk), dtype=torch.int32, device=dev)
    o3 = torch.empty((3, B, T, Hq, d), dtype=torch.float32, device=dev)
    nbytes = lib.sa_nsa_workspace_size(B, T, Hq, Hkv, d, cmp_len, cmp_stride, sel_block, sel_topk)
    ws = _workspace(nbytes, dev)
    with torch.cuda.device(dev):
        check(lib.sa_nsa_fwd_train(_ptr(q), _ptr(k), _ptr(v), _ptr(gates), B, T, Hq, Hkv, d, cmp_len,
                                   cmp_stride, sel_block, sel_topk, window, float(scale), _ptr(out),
                                   _ptr(lse3), _ptr(sel), _ptr(o3), _ptr(ws), nbytes, _stream(dev)),
              "sa_nsa_fwd_train")
    return out, lse3, sel, o3


def nsa_bwd(q, k, v, gates, dout, o_branches, lse_branches, sel_idx, cmp_len: int, cmp_stride: int,
            sel_block: int, sel_topk: int, window: int, scale: Optional[float] = None):
    """NSA backward (sa_nsa_bwd) with the forward's block choice held fixed.

    o_branches, lse_branches and sel_idx are nsa_fwd_train's.  Returns
    (dq fp32 [B,T,Hq,d], dk fp32 [B,T,Hkv,d], dv fp32 [B,T,Hkv,d],
    dgates fp32 [B,T,Hq,3]).
    """
    lib = _lib.load()
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout")):
        _need(t, n, torch.bfloat16, dev, 4)
    _need(gates, "gates", torch.float32, dev, 4)
    _need(o_branches, "o_branches", torch.float32, dev, 5)
    _need(lse_branches, "lse_branches", torch.float32, dev, 4)
    _need(sel_idx, "sel_idx", torch.int32, dev, 4)
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    if (k.shape != (B, T, Hkv, d) or v.shape != k.shape or dout.shape != q.shape
            or gates.shape != (B, T, Hq, 3) or o_branches.shape != (3, B, T, Hq, d)
            or lse_branches.shape != (B, T, Hq, 3) or sel_idx.shape != (B, T, Hkv, sel_topk)):
        raise ValueError("nsa_bwd: shape mismatch")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty((B, T, Hq, d), dtype=torch.float32, device=dev)
    dk = torch.empty((B, T, Hkv, d), dtype=torch.float32, device=dev)
    dv = torch.empty((B, T, Hkv, d), dtype=torch.float32, device=dev)
    dg = torch.empty((B, T, Hq, 3), dtype=torch.float32, device=dev)
    nbytes = lib.sa_nsa_bwd_workspace_size(B, T, Hq, Hkv, d, cmp_len, cmp_stride, sel_block, sel_topk)
    ws = _workspace(nbytes, dev)
    with torch.cuda.device(dev):
        check(lib.sa_nsa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(gates), _ptr(dout), _ptr(o_branches),
                             _ptr(lse_branches), _ptr(sel_idx), B, T, Hq, Hkv, d, cmp_len, cmp_stride,
                             sel_block, sel_topk, window, float(scale), _ptr(dq), _ptr(dk), _ptr(dv),
                             _ptr(dg), _ptr(ws), nbytes, _stream(dev)), "sa_nsa_bwd")
    return dq, dk, dv, dg


def full_attn_topk(q, k, v, topk: int, window: int, scale: Optional[float] = None,
                   out=None, lse=None, out_idx=None, workspace=None):
    """A full-attention layer as an exact indexer (sa_full_attn_topk).

    q bf16 [B,T,Hq,d], k/v bf16 [B,T,Hkv,d].  Returns (out bf16 [B,T,Hq,d],
    lse fp32 [B,T,Hq], idx int32 [B,T,topk+window]): the full layer's causal
    attention and, for the sparse layers, the forced window plus the top-k
    keys by the full layer's head-summed attention probabilities.
    """
    lib = _lib.load()
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 4)
    _need(k, "k", torch.bfloat16, dev, 4)
    _need(v, "v", torch.bfloat16, dev, 4)
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, T, Hkv, d) or v.shape != k.shape:
        raise ValueError("full_attn_topk: shape mismatch")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, T, Hq, d), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, T, Hq), dtype=torch.float32, device=dev)
    if out_idx is None:
        out_idx = torch.empty((B, T, topk + window), dtype=torch.int32, device=dev)
    nbytes = lib.sa_full_attn_topk_workspace_size(B, T, Hq, Hkv, d, topk, window)
    ws = workspace if workspace is not None else _workspace(nbytes, dev)
    with torch.cuda.device(dev):
        check(lib.sa_full_attn_topk(_ptr(q), _ptr(k), _ptr(v), B, T, Hq, Hkv, d, float(scale), topk,
                                    window, _ptr(out), _ptr(lse), _ptr(out_idx), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(dev)), "sa_full_attn_topk")
    return out, lse, out_idx


# --------------------------------------------------------------- IndexCache --
def dsa_decode_layers(pattern: str, layers, topk: int, window: int = 0, n_split: int = 1,
                      q_pos0: Optional[int] = None, scale: Optional[float] = None,
                      outs=None, lses=None, idx_cache=None, workspace=None):
    """IndexCache layer loop (sa_dsa_decode_layers).

    layers: list of dicts with q, k, v, q_idx, k_idx, w (same shapes for every
    layer).  F layers run the indexer, S layers reuse the cached indices.
    Returns (outs, lses, idx_cache).
    """
    lib = _lib.load()
    n = len(layers)
    if len(pattern) < n:
        raise ValueError("pattern shorter than the layer list")
    l0 = layers[0]
    dev = l0["q"].device
    B, Tq, Hq, d = l0["q"].shape
    L, Hkv = l0["k"].shape[1], l0["k"].shape[2]
    Hi, di = l0["q_idx"].shape[2], l0["q_idx"].shape[3]
    for ly in layers:
        _need(ly["q"], "q", torch.bfloat16, dev, 4)
        _need(ly["k"], "k", torch.bfloat16, dev, 4)
        _need(ly["v"], "v", torch.bfloat16, dev, 4)
        _need(ly["q_idx"], "q_idx", torch.int8, dev, 4)
        _need(ly["k_idx"], "k_idx", torch.int8, dev, 3)
        _need(ly["w"], "w", torch.int32, dev, 3)
    pos0 = L - Tq if q_pos0 is None else int(q_pos0)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if outs is None:
        outs = [torch.empty((B, Tq, Hq, d), dtype=torch.bfloat16, device=dev) for _ in range(n)]
    if lses is None:
        lses = [torch.empty((B, Tq, Hq), dtype=torch.float32, device=dev) for _ in range(n)]
    if idx_cache is None:
        idx_cache = torch.empty((B, Tq, topk + window), dtype=torch.int32, device=dev)
    arr = (sa_dsa_layer * n)()
    for i, ly in enumerate(layers):
        arr[i] = sa_dsa_layer(ly["q"].data_ptr(), ly["k"].data_ptr(), ly["v"].data_ptr(),
                              ly["q_idx"].data_ptr(), ly["k_idx"].data_ptr(), ly["w"].data_ptr(),
                              outs[i].data_ptr(), lses[i].data_ptr())
    nbytes = lib.sa_dsa_decode_layers_workspace_size(B, Tq, L, Hq, d, Hi, di, topk, window, n_split)
    if workspace is None or workspace.numel() < nbytes:
        workspace = _workspace(nbytes, dev)
    with torch.cuda.device(dev):
        check(lib.sa_dsa_decode_layers(pattern.encode(), n, arr, B, Tq, L, Hq, Hkv, d, Hi, di,
                                       pos0, topk, window, float(scale), int(n_split),
                                       _ptr(idx_cache), _ptr(workspace), nbytes, _stream(dev)),
              "sa_dsa_decode_layers")
    return outs, lses, idx_cache


def dsa_decode_workspace_bytes(B, Tq, L, Hq, d, Hi, di, topk, window=0, n_split=1) -> int:
    return int(_lib.load().sa_dsa_decode_layers_workspace_size(B, Tq, L, Hq, d, Hi, di, topk,
                                                               window, n_split))


# ------------------------------------------------- sink-window attention --
# These entry points serve single tokens, where a call costs less on the device
# than a careless binding on the host: the checks take a short way for tensors
# as they should be, and the slow helpers only word the refusal.
_ATTN_TYPES = {torch.bfloat16: _lib.SA_BF16, torch.float16: _lib.SA_FP16}
_SINK_SHAPE = struct.Struct("=7if20q2i")           # sa_sink_shape
_INT_MAX = 2 ** 31 - 1                              # a longer window sees no more
_PAGED_SHAPE = struct.Struct("=9if9q")             # sa_paged_shape
assert _SINK_SHAPE.size == ctypes.sizeof(_lib.sa_sink_shape)
assert _PAGED_SHAPE.size == ctypes.sizeof(_lib.sa_paged_shape)


class _on_device:
    """The device of a call made current, if it is not already."""
    __slots__ = ("index", "guard")

    def __init__(self, index):
        self.index = index

    def __enter__(self):
        self.guard = None
        if self.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(self.index)
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _need_rows(t, name: str, dtype, dev, shape):
    """Refuses a tensor of rows that has not strides of multiples of 16 bytes and a contiguous last dimension."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.numel():
        st, n = t.stride(), 16 // t.element_size()
        if st[-1] != 1 or t.data_ptr() % 16:
            raise ValueError(f"{name}: the last dimension must be contiguous and the data 16-byte aligned")
        for i in range(len(st) - 1):
            if t.shape[i] > 1 and st[i] % n:
                raise ValueError(f"{name}: strides must be multiples of 16 bytes, got {st}")
            if t.shape[i] > 1 and st[i] <= 0:
                raise ValueError(f"{name}: a broadcast input is not supported, got strides {st}")


def _rows(t, name: str, dtype, dev, shape, mask: int = 7):
    """Strides in front of the last dimension of a checked tensor of rows; mask: elements in 16 bytes, less 1.
    A dimension of size 1 is never stepped over (its stride is given as 0 where it would not pass)."""
    if t is not None and t.dtype == dtype and t.device == dev and t.shape == shape and not t.data_ptr() & 15:
        st = t.stride()
        if st[-1] == 1:
            st, bad = st[:-1], False
            for x in st:
                if x <= 0 or x & mask:
                    bad = True
            if not bad:
                return st
    _need_rows(t, name, dtype, dev, shape)
    return tuple(x if size > 1 else 0 for x, size in zip(t.stride()[:-1], t.shape))


def _need_out(t, name: str, like, dtype, shape):
    """The output given, checked, or a new one beside `like`."""
    if t is None:
        if dtype == like.dtype and shape == like.shape and like.is_contiguous():
            return torch.empty_like(like)
        return like.new_empty(tuple(shape), dtype=dtype)
    _need(t, name, dtype, like.device)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _scratch(workspace, like, need):
    """The caller's workspace, or a new one of need() bytes beside `like`; (tensor, bytes).  One that the device cannot
    reach is refused here: the library sees an address only."""
    if workspace is None:
        nbytes = need()
        return like.new_empty(nbytes, dtype=torch.uint8), nbytes
    if not isinstance(workspace, torch.Tensor) or workspace.device != like.device:
        raise ValueError(f"workspace must be a tensor on {like.device}, got "
                         f"{workspace.device if isinstance(workspace, torch.Tensor) else type(workspace).__name__}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


def _ints(t, name: str, dev, n=None):
    """The length of a list int32 [n] on the device."""
    if t is None or t.dtype != torch.int32 or t.device != dev or t.dim() != 1 or not t.is_contiguous():
        _need(t, name, torch.int32, dev, 1)
    m = t.shape[0]
    if n is not None and m != n:
        raise ValueError(f"{name} must have {n} entries, got {m}")
    return m


def _sink_shape(what, q, k, v, window, sinks, cu_q, cu_k, max_q, max_k, scale, q_pos0, dtypes):
    """Checks the inputs; the fields of sa_sink_shape up to v_stride, the device, whether the batch is packed."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise ValueError(f"{what}: q must be a CUDA tensor (there is no CPU path)")
    dev, dt, qs = q.device, q.dtype, q.shape
    if dt not in dtypes:
        raise TypeError(f"{what}: q must be one of {[str(x) for x in dtypes]}, got {dt}")
    packed = cu_q is not None
    if packed != (cu_k is not None):
        raise ValueError(f"{what}: cu_q and cu_k go together")
    if len(qs) != (3 if packed else 4) or k is None or k.dim() != len(qs):
        raise ValueError(f"{what}: q and k must have {3 if packed else 4} dims")
    ks = k.shape
    Hq, d = qs[-2:]
    Hkv = ks[-2]
    if packed:
        B, Tq, L = _ints(cu_q, "cu_q", dev) - 1, qs[0], ks[0]
        if B < 1 or _ints(cu_k, "cu_k", dev) != B + 1:
            raise ValueError(f"{what}: cu_q and cu_k must be int32 [B+1]")
        if q_pos0 is not None:
            raise ValueError(f"{what}: q_pos0 has no meaning for packed sequences")
        pos0, kshape = 0, (L, Hkv, d)
    else:
        B, Tq, L = qs[0], qs[1], ks[1]
        if max_q is not None and max_q != Tq or max_k is not None and max_k != L:
            raise ValueError(f"{what}: max_q and max_k of a dense batch are its lengths")
        pos0, kshape = L - Tq if q_pos0 is None else int(q_pos0), (B, L, Hkv, d)
        if pos0 < 0:
            raise ValueError(f"{what}: more queries than keys needs q_pos0")
        max_q = max_k = 0
    lead = (0,) if packed else ()
    st = (*lead, *_rows(q, "q", dt, dev, qs), *lead, *_rows(k, "k", dt, dev, kshape), *lead,
          *_rows(v, "v", dt, dev, kshape))
    return (_ATTN_TYPES[dt], B, Hq, Hkv, d, min(int(window), _INT_MAX), min(int(sinks), _INT_MAX), 1.0 / math.sqrt(d) if scale is None else scale,
            Tq, L, pos0, max_q or 0, max_k or 0, *st), dev, packed


def _parts(weight_parts) -> int:
    if weight_parts not in (None, 1, 2):
        raise ValueError(f"weight_parts must be 1, 2 or None (by the size of the call), got {weight_parts}")
    return weight_parts or 0


def sink_attn_fwd(q, k, v, window: int, sinks: int = 0, cu_q=None, cu_k=None, max_q: Optional[int] = None,
                  max_k: Optional[int] = None, scale: Optional[float] = None, q_pos0: Optional[int] = None,
                  out=None, lse=None, weight_parts: Optional[int] = None):
    """Causal attention over a sliding window plus the first `sinks` keys (sa_sink_attn_fwd).

    Dense: q bf16 or fp16 [B,Tq,Hq,d], k/v [B,L,Hkv,d]; q_pos0 defaults to
    L - Tq.  Packed: q [N,Hq,d], k/v [M,Hkv,d] with cu_q, cu_k int32 [B+1] (a
    sequence's last query stands at its last key) and max_q, max_k, upper
    bounds of the lengths.  q, k and v may be strided views (the parts of one
    projection).  weight_parts: 1 or 2, how exactly the weights enter the
    second product (None: 2 up to 8192 rows of q, 1 above; a fixed number
    makes a sequence's results independent of the batch).  Returns (out like
    q, contiguous, lse fp32 [..., Hq]); rows outside every packed sequence are
    left as they were in `out` and `lse`.
    """
    lib = _lib.load()
    f, dev, packed = _sink_shape("sink_attn_fwd", q, k, v, window, sinks, cu_q, cu_k, max_q, max_k, scale, q_pos0,
                                 _ATTN_TYPES)
    qs = q.shape
    out = _need_out(out, "out", q, q.dtype, qs)
    lse = _need_out(lse, "lse", q, torch.float32, qs[:-1])
    with _on_device(dev.index):
        rc = lib.sa_sink_attn_fwd(_SINK_SHAPE.pack(*f, 0, 0, 0, 0, 0, 0, _parts(weight_parts), 0), q.data_ptr(),
                                  k.data_ptr(), v.data_ptr(), _ptr(cu_q), _ptr(cu_k), out.data_ptr(), lse.data_ptr(),
                                  _raw_stream(dev.index))
    if rc:
        check(rc, "sa_sink_attn_fwd")
    return out, lse


def sink_attn_bwd(q, k, v, out, lse, dout, window: int, sinks: int = 0, cu_q=None, cu_k=None,
                  max_q: Optional[int] = None, max_k: Optional[int] = None, scale: Optional[float] = None,
                  q_pos0: Optional[int] = None, dq=None, dk=None, dv=None, weight_parts: Optional[int] = None):
    """Backward of sink_attn_fwd (sa_sink_attn_bwd), bf16.

    out and lse are the forward's (out may be None: only lse is read); the
    other arguments as there.  Returns (dq, dk, dv), bf16, shaped like q, k
    and v; rows outside every packed sequence are left as they were.
    """
    lib = _lib.load()
    bf = torch.bfloat16
    f, dev, packed = _sink_shape("sink_attn_bwd", q, k, v, window, sinks, cu_q, cu_k, max_q, max_k, scale, q_pos0,
                                 (bf,))
    qs, lead = q.shape, (0,) if packed else ()
    if out is not None:
        _rows(out, "out", bf, dev, qs)
    if not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32 or lse.device != dev or lse.shape != qs[:-1]:
        raise ValueError("sink_attn_bwd: lse must be the forward's, fp32 and shaped like q without d")
    shape = _SINK_SHAPE.pack(*f, *lead, *_rows(dout, "dout", bf, dev, qs), *lead, *lse.stride(),
                             _parts(weight_parts), 0)
    dq, dk, dv = _need_out(dq, "dq", q, bf, qs), _need_out(dk, "dk", k, bf, k.shape), _need_out(dv, "dv", v, bf, v.shape)
    with _on_device(dev.index):
        nbytes = lib.sa_sink_attn_bwd_workspace_size(shape, int(packed))
        ws = q.new_empty(nbytes, dtype=torch.uint8)
        rc = lib.sa_sink_attn_bwd(shape, q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(out), lse.data_ptr(),
                                  dout.data_ptr(), _ptr(cu_q), _ptr(cu_k), dq.data_ptr(), dk.data_ptr(),
                                  dv.data_ptr(), _ptr(ws), nbytes, _raw_stream(dev.index))
    if rc:
        check(rc, "sa_sink_attn_bwd")
    return dq, dk, dv


# ----------------------------------------------------------- paged caches --
def paged_attn_decode(q, k_cache, v_cache, block_table, seq_lens, window: Optional[int] = None, sinks: int = 0,
                      scale: Optional[float] = None, out=None, lse=None, workspace=None):
    """Attention of one new token per sequence over a paged cache (sa_paged_attn_decode).

    q bf16 or fp16 [B,Hq,d]; caches [n_pages,page,Hkv,d] (strided views
    allowed, e.g. K and V interleaved by page); block_table int32
    [B,max_pages], seq_lens int32 [B] (the new token counted).  window None:
    every key is visible.  Returns (out [B,Hq,d], lse fp32 [B,Hq]).
    """
    lib = _lib.load()
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise ValueError("paged_attn_decode: q must be a CUDA tensor (there is no CPU path)")
    dev, dt, qs = q.device, q.dtype, q.shape
    if dt not in _ATTN_TYPES:
        raise TypeError(f"paged_attn_decode: q must be bfloat16 or float16, got {dt}")
    if len(qs) != 3 or k_cache is None or k_cache.dim() != 4:
        raise ValueError("paged_attn_decode: q must be [B,Hq,d] and the caches [n_pages,page,Hkv,d]")
    B, Hq, d = qs
    n_pages, page, Hkv = k_cache.shape[:3]
    cs = (n_pages, page, Hkv, d)
    st = (*_rows(q, "q", dt, dev, qs), *_rows(k_cache, "k_cache", dt, dev, cs), *_rows(v_cache, "v_cache", dt, dev, cs))
    _need(block_table, "block_table", torch.int32, dev, 2)
    if block_table.shape[0] != B or _ints(seq_lens, "seq_lens", dev) != B:
        raise ValueError("paged_attn_decode: block_table and seq_lens must have a row per sequence")
    if window is not None and window < 1:
        raise ValueError("paged_attn_decode: window >= 1 (None: every key)")
    shape = _PAGED_SHAPE.pack(_ATTN_TYPES[dt], B, Hq, Hkv, d, page, block_table.shape[1],
                              min(int(window or 0), _INT_MAX), min(int(sinks), _INT_MAX), 1.0 / math.sqrt(d) if scale is None else scale, n_pages, *st)
    out = _need_out(out, "out", q, dt, qs)
    lse = _need_out(lse, "lse", q, torch.float32, qs[:-1])
    with _on_device(dev.index):
        ws, have = _scratch(workspace, q, lambda: lib.sa_paged_attn_decode_workspace_size(B, Hq, Hkv, d))
        rc = lib.sa_paged_attn_decode(shape, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                      block_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                      _ptr(ws), have, _raw_stream(dev.index))
    if rc:
        check(rc, "sa_paged_attn_decode")
    return out, lse


def paged_attn_decode_workspace_bytes(B, Hq, Hkv, d) -> int:
    return int(_lib.load().sa_paged_attn_decode_workspace_size(B, Hq, Hkv, d))


def _books(what, block_table, refcount, seq_lens=None):
    if not isinstance(block_table, torch.Tensor):
        raise ValueError(f"{what}: block_table is required")
    dev = block_table.device
    _need(block_table, "block_table", torch.int32, dev, 2)
    S, max_pages = block_table.shape
    if seq_lens is not None and _ints(seq_lens, "seq_lens", dev) != S:
        raise ValueError(f"{what}: block_table and seq_lens must have a row per sequence")
    return dev, S, max_pages, _ints(refcount, "refcount", dev)


def _page_caches(what, caches, dev, n_pages, page):
    """Caches [n_pages, page, ...] of one slot size as the C array; (array, bytes per slot, page)."""
    fields, slot_bytes = [], 0
    for i, c in enumerate(caches):
        if not isinstance(c, torch.Tensor) or c.dim() < 2 or c.device != dev:
            raise ValueError(f"{what}: caches must be tensors [n_pages, page, ...] on {dev}")
        shape, st, es = c.shape, c.stride(), c.element_size()
        page = shape[1] if page is None else page
        if shape[0] != n_pages or shape[1] != page:
            raise ValueError(f"{what}: cache {i} must be [{n_pages}, {page}, ...], got {tuple(shape)}")
        n = es
        for size, x in zip(shape[:1:-1], st[:1:-1]):
            if size != 1 and x * es != n:
                raise ValueError(f"{what}: the slots of cache {i} must be contiguous")
            n *= size
        if i and n != slot_bytes:
            raise ValueError(f"{what}: the caches must have the same bytes per slot")
        slot_bytes = n
        fields += c.data_ptr(), st[0] * es if n_pages > 1 else 0, st[1] * es if page > 1 else n
    if page is None:
        raise ValueError(f"{what}: page is required without caches")
    return struct.pack(f"={len(fields)}q", *fields), slot_bytes, page


def paged_books_workspace_bytes(S, n, n_pages) -> int:
    """Bytes that paged_extend and paged_fork of lists of n, and paged_compact (n = 0), need for tables of S rows."""
    return int(_lib.load().sa_paged_books_workspace_size(S, n, n_pages))


def paged_extend(block_table, seq_lens, refcount, seqs, n_new, page: int, start=None, workspace=None):
    """Pages for n_new more tokens of the listed sequences (sa_paged_extend).

    block_table int32 [S,max_pages], seq_lens int32 [S], refcount int32
    [n_pages] are updated in place.  Returns start int32 [n]: where each
    entry's new tokens begin, -1 where it was not served.
    """
    lib = _lib.load()
    dev, S, max_pages, n_pages = _books("paged_extend", block_table, refcount, seq_lens)
    n = _ints(seqs, "seqs", dev)
    _ints(n_new, "n_new", dev, n)
    start = _need_out(start, "start", seqs, torch.int32, (n,))
    with _on_device(dev.index):
        ws, have = _scratch(workspace, refcount, lambda: lib.sa_paged_books_workspace_size(S, n, n_pages))
        rc = lib.sa_paged_extend(block_table.data_ptr(), seq_lens.data_ptr(), refcount.data_ptr(), S, max_pages,
                                 n_pages, int(page), seqs.data_ptr(), n_new.data_ptr(), n, start.data_ptr(),
                                 _ptr(ws), have, _raw_stream(dev.index))
    if rc:
        check(rc, "sa_paged_extend")
    return start


def paged_write(k_new, v_new, k_cache, v_cache, block_table, seqs, start, cu_new=None):
    """Writes new tokens into their slots (sa_paged_write).

    k_new/v_new [N,Hkv,d] (strided views allowed) of any element type; entry i
    of the list has rows cu_new[i] .. cu_new[i+1]-1 (None: one row each) and
    goes to positions start[i], start[i]+1, ... of sequence seqs[i] in
    k_cache/v_cache [n_pages,page,Hkv,d].  Entries with start -1 are skipped.
    """
    lib = _lib.load()
    if not isinstance(k_new, torch.Tensor) or k_new.dim() != 3 or not isinstance(k_cache, torch.Tensor) or \
            k_cache.dim() != 4:
        raise ValueError("paged_write: k_new must be [N,Hkv,d] and k_cache [n_pages,page,Hkv,d]")
    dev, dt, es, ns = k_new.device, k_new.dtype, k_new.element_size(), k_new.shape
    if not k_new.is_cuda:
        raise ValueError("paged_write: k_new must be a CUDA tensor (there is no CPU path)")
    N, Hkv, d = ns
    n_pages, page = k_cache.shape[:2]
    cs, m = (n_pages, page, Hkv, d), 16 // es - 1
    strides = struct.pack("=10q", *_rows(k_new, "k_new", dt, dev, ns, m), *_rows(v_new, "v_new", dt, dev, ns, m),
                          *_rows(k_cache, "k_cache", dt, dev, cs, m), *_rows(v_cache, "v_cache", dt, dev, cs, m))
    _need(block_table, "block_table", torch.int32, dev, 2)
    n = _ints(seqs, "seqs", dev)
    _ints(start, "start", dev, n)
    if cu_new is not None:
        _ints(cu_new, "cu_new", dev, n + 1)
    elif N != n:
        raise ValueError("paged_write: without cu_new one row per entry")
    S, max_pages = block_table.shape
    with _on_device(dev.index):
        rc = lib.sa_paged_write(k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                block_table.data_ptr(), seqs.data_ptr(), start.data_ptr(), _ptr(cu_new), n, N, S,
                                max_pages, n_pages, page, Hkv, d, es, strides, _raw_stream(dev.index))
    if rc:
        check(rc, "sa_paged_write")


def paged_fork(block_table, seq_lens, refcount, src, dst, page: int, caches=(), done=None, workspace=None):
    """Sequences dst[i] become copies of src[i] that share its full pages (sa_paged_fork).

    caches: tensors [n_pages,page,...] (each layer's K and V) in which the
    partly filled last pages are copied.  Returns done int32 [n] (1 = forked).
    """
    lib = _lib.load()
    dev, S, max_pages, n_pages = _books("paged_fork", block_table, refcount, seq_lens)
    n = _ints(src, "src", dev)
    _ints(dst, "dst", dev, n)
    arr, slot_bytes, page = _page_caches("paged_fork", caches, dev, n_pages, int(page))
    done = _need_out(done, "done", src, torch.int32, (n,))
    with _on_device(dev.index):
        ws, have = _scratch(workspace, refcount, lambda: lib.sa_paged_books_workspace_size(S, n, n_pages))
        rc = lib.sa_paged_fork(block_table.data_ptr(), seq_lens.data_ptr(), refcount.data_ptr(), S, max_pages, n_pages,
                               page, src.data_ptr(), dst.data_ptr(), n, arr, len(caches), slot_bytes, done.data_ptr(),
                               _ptr(ws), have, _raw_stream(dev.index))
    if rc:
        check(rc, "sa_paged_fork")
    return done


def paged_free(block_table, seq_lens, refcount, seqs, page: Optional[int] = None, window: Optional[int] = None,
               sinks: int = 0):
    """Gives the pages of the listed sequences back, or with a window only
    those that no later query can see (sa_paged_free; page is needed then)."""
    lib = _lib.load()
    dev, S, max_pages, n_pages = _books("paged_free", block_table, refcount, seq_lens)
    n = _ints(seqs, "seqs", dev)
    if window is not None and (window < 1 or page is None):
        raise ValueError("paged_free: a window needs window >= 1 and page")
    with _on_device(dev.index):
        rc = lib.sa_paged_free(block_table.data_ptr(), seq_lens.data_ptr(), refcount.data_ptr(), S, max_pages, n_pages,
                               int(page or 1), seqs.data_ptr(), n, min(int(window or 0), _INT_MAX),
                               min(int(sinks), _INT_MAX), _raw_stream(dev.index))
    if rc:
        check(rc, "sa_paged_free")


def paged_compact(block_table, refcount, caches=(), page: Optional[int] = None, n_live=None, workspace=None):
    """Moves the live pages to the front of the pool (sa_paged_compact).

    caches: tensors [n_pages,page,...]; block_table and refcount follow.
    Returns n_live int32 [1] on the device.
    """
    lib = _lib.load()
    dev, S, max_pages, n_pages = _books("paged_compact", block_table, refcount)
    arr, slot_bytes, page = _page_caches("paged_compact", caches, dev, n_pages, page if caches else (page or 1))
    n_live = _need_out(n_live, "n_live", refcount, torch.int32, (1,))
    with _on_device(dev.index):
        ws, have = _scratch(workspace, refcount, lambda: lib.sa_paged_books_workspace_size(S, 0, n_pages))
        rc = lib.sa_paged_compact(block_table.data_ptr(), refcount.data_ptr(), S, max_pages, n_pages, page, arr,
                                  len(caches), slot_bytes, n_live.data_ptr(), _ptr(ws), have, _raw_stream(dev.index))
    if rc:
        check(rc, "sa_paged_compact")
    return n_live
