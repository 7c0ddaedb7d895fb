"""Thin ctypes binding over the C ABI in include/sparse_mla.h.

Argument marshalling only: shape/dtype/device checks, raw pointers and sizes,
output allocation through torch.  Every step of the attention runs in the
CUDA library; there is no fallback.  Loading fails loudly when the library
has not been built.

The C ABI receives pointers and sizes only, so the extents are checked
here: every tensor a call reads or writes (inputs, caller-supplied outputs
and workspaces) must sit on the call's device and hold at least the
elements the passed sizes address, and caller-supplied outputs must have
the output's dtype and be contiguous; otherwise ValueError is raised before
anything is launched.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

from . import build as _build

_LIB: Optional[ctypes.CDLL] = None

c_int, c_float, c_void_p, c_size_t = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
c_longlong = ctypes.c_longlong

STATUS = {0: "SPARSE_MLA_OK", 1: "SPARSE_MLA_ERR_INVALID_ARG", 2: "SPARSE_MLA_ERR_UNSUPPORTED_SHAPE",
          3: "SPARSE_MLA_ERR_UNSUPPORTED_ARCH", 4: "SPARSE_MLA_ERR_CUDA", 5: "SPARSE_MLA_ERR_DEVICE_TIMEOUT",
          6: "SPARSE_MLA_ERR_WORKSPACE_TOO_SMALL"}

# name -> (restype, argtypes); the exported surface of include/sparse_mla.h
SIGNATURES = {
    "sparse_mla_fwd": (c_int, [c_void_p, c_void_p, c_void_p, c_float, c_void_p, c_void_p,
                               c_int, c_int, c_int, c_int, c_int, c_int, c_void_p]),
    "sparse_mla_bwd": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_float,
                               c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int, c_int, c_void_p]),
    "sparse_mla_bwd_varlen": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p,
                                      c_void_p, c_void_p, c_float, c_void_p, c_void_p, c_int, c_int, c_int,
                                      c_int, c_int, c_int, c_void_p]),
    "sparse_mla_fwd_causal": (c_int, [c_void_p, c_void_p, c_float, c_void_p, c_void_p,
                                      c_int, c_int, c_int, c_int, c_int, c_void_p]),
    "sparse_mla_fwd_varlen": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_float,
                                      c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int, c_int, c_void_p]),
    "sparse_mla_decode_workspace_size": (c_size_t, [c_int, c_int, c_int, c_int, c_int]),
    "sparse_mla_decode": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_float, c_void_p,
                                  c_void_p, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                  c_void_p, c_size_t, c_void_p]),
    "sparse_mla_decode_fp8": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_float, c_void_p,
                                      c_void_p, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                      c_void_p, c_size_t, c_void_p]),
    "sparse_mla_decode_noalloc": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_float, c_void_p,
                                          c_void_p, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                          c_void_p]),
    "sparse_mla_decode_noalloc_max_scratch_bytes": (c_size_t, []),
    "sparse_mla_decode_fp4": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_float, c_float, c_void_p,
                                      c_void_p, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                      c_void_p, c_size_t, c_void_p]),
    "sparse_mla_decode_fp4_workspace_size": (c_size_t, [c_int, c_int, c_int, c_int, c_int]),
    "mla_norm_rope": (c_int, [c_void_p, c_longlong, c_longlong, c_void_p, c_longlong, c_void_p, c_void_p, c_int,
                              c_void_p, c_void_p, c_float, c_int, c_void_p, c_void_p, c_void_p, c_int, c_float,
                              c_void_p, c_int, c_int, c_int, c_int, c_void_p]),
    "mla_norm_rope_bwd": (c_int, [c_void_p, c_longlong, c_longlong, c_void_p, c_longlong, c_void_p, c_void_p, c_int,
                                  c_void_p, c_void_p, c_float, c_int, c_void_p, c_void_p, c_void_p, c_void_p,
                                  c_void_p, c_void_p, c_int, c_int, c_int, c_void_p, c_size_t, c_void_p]),
    "mla_norm_rope_bwd_workspace_size": (c_size_t, [c_int, c_int]),
    "mla_add_norm": (c_int, [c_void_p, c_longlong, c_void_p, c_longlong, c_void_p, c_float, c_void_p, c_void_p, c_int,
                             c_void_p, c_int, c_int, c_void_p]),
    "mla_add_norm_bwd": (c_int, [c_void_p, c_longlong, c_void_p, c_float, c_void_p, c_longlong, c_void_p, c_longlong,
                                 c_void_p, c_void_p, c_int, c_int, c_void_p, c_size_t, c_void_p]),
    "mla_add_norm_bwd_workspace_size": (c_size_t, [c_int, c_int]),
    "dense_mha_fwd": (c_int, [c_void_p, c_longlong, c_longlong, c_void_p, c_longlong, c_longlong, c_void_p, c_longlong,
                              c_longlong, c_void_p, c_void_p, c_int, c_float, c_void_p, c_void_p, c_int, c_int, c_int,
                              c_int, c_int, c_int, c_int, c_void_p]),
    "dense_mha_bwd": (c_int, [c_void_p, c_longlong, c_longlong, c_void_p, c_longlong, c_longlong, c_void_p, c_longlong,
                              c_longlong, c_void_p, c_void_p, c_int, c_float, c_void_p, c_void_p, c_void_p, c_longlong,
                              c_longlong, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int, c_int,
                              c_void_p, c_size_t, c_void_p]),
    "dense_mha_bwd_workspace_size": (c_size_t, [c_int, c_int, c_int, c_int, c_int, c_int, c_int]),
    "sparse_mla_debug_valid_count": (c_int, [c_void_p, c_int, c_int, c_int, c_void_p, c_void_p]),
    "sparse_mla_debug_valid_count_varlen": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int,
                                                    c_void_p, c_void_p]),
    "sparse_mla_debug_valid_count_paged": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int,
                                                   c_int, c_int, c_void_p, c_void_p]),
    "dsa_indexer_scores": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int,
                                   c_int, c_int, c_int, c_int, c_int, c_void_p, ctypes.c_longlong, c_void_p]),
    "dsa_topk": (c_int, [c_void_p, ctypes.c_longlong, c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int,
                         c_int, c_void_p, c_void_p]),
    "dsa_indexer_workspace_size": (c_size_t, [c_int, c_int, c_int]),
    "dsa_indexer_topk": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int,
                                 c_int, c_int, c_int, c_void_p, c_void_p, c_size_t, c_void_p]),
    "dsa_indexer_scores_paged": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int,
                                         c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_void_p,
                                         ctypes.c_longlong, c_void_p]),
    "dsa_indexer_topk_paged": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int,
                                       c_int, c_int, c_int, c_int, c_int, c_int, c_void_p, c_void_p, c_size_t,
                                       c_void_p]),
    "sparse_mla_status_string": (ctypes.c_char_p, [c_int]),
    "sparse_mla_get_device_error": (c_int, [ctypes.POINTER(c_int)]),
    "sparse_mla_clear_device_error": (c_int, []),
    "sparse_mla_set_wait_timeout_ns": (None, [ctypes.c_ulonglong]),
}


class SparseMLAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


def lib_path() -> str:
    return _build.LIB_PATH


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load the built library (raises if it is missing)."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or lib_path()
    if not os.path.exists(p):
        raise RuntimeError(f"CUDA library not built ({p}); run __graft_entry__.build()")
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _LIB = lib
    return lib


def _check(status: int, where: str):
    if status != 0:
        raise SparseMLAError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _on_cuda(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _need(t: torch.Tensor, dtype, name: str):
    _on_cuda(t, name)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _device_key(device):
    d = torch.device(device)
    if d.type == "cuda" and d.index is None:   # "cuda" means the current device
        return ("cuda", torch.cuda.current_device())
    return (d.type, d.index)


def _fits(t: Optional[torch.Tensor], need: int, name: str, device) -> None:
    """The kernels address t as a dense array of `need` elements on `device`.
    The C ABI sees only pointers and sizes, so extents are checked here: a
    tensor on another device, or with fewer elements than the sizes passed
    to the library imply, is refused before anything is launched."""
    if t is None:
        return
    if t.device != device and _device_key(t.device) != _device_key(device):
        raise ValueError(f"{name} is on {t.device}; the call's tensors are on {device}")
    if t.numel() < need:
        raise ValueError(f"{name} holds {t.numel()} elements; the call addresses {need}")


def _given(t: Optional[torch.Tensor], dtype, name: str, need: int, device) -> None:
    """A caller-supplied output or workspace: CUDA, dtype, contiguous, large
    enough and on the call's device."""
    if t is None or (t.is_cuda and t.dtype is dtype and t.device == device and t.is_contiguous()
                     and t.numel() >= need):
        return
    _need(t, dtype, name)
    _fits(t, need, name, device)


def sparse_mla_fwd(q: torch.Tensor, kv: torch.Tensor, indices: torch.Tensor, sm_scale: float,
                   out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """q [s_q,h_q,576] bf16, kv [s_kv,576] or [s_kv,1,576] bf16,
    indices [s_q,topk] or [s_q,1,topk] int32 -> (out [s_q,h_q,512] bf16,
    lse [s_q,h_q] fp32)."""
    lib = load()
    s_q, h_q, d_qk = q.shape
    s_kv = kv.shape[0]
    topk = indices.shape[-1]
    for t, dt, n in ((q, torch.bfloat16, "q"), (kv, torch.bfloat16, "kv"), (indices, torch.int32, "indices")):
        _need(t, dt, n)
    d_v = 512
    dev = q.device
    _fits(kv, s_kv * d_qk, "kv", dev)
    _fits(indices, s_q * topk, "indices", dev)
    _given(out, torch.bfloat16, "out", s_q * h_q * d_v, dev)
    _given(lse, torch.float32, "lse", s_q * h_q, dev)
    if out is None:
        out = torch.empty((s_q, h_q, d_v), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((s_q, h_q), dtype=torch.float32, device=q.device)
    st = lib.sparse_mla_fwd(_ptr(q), _ptr(kv), _ptr(indices), float(sm_scale), _ptr(out), _ptr(lse),
                            s_q, s_kv, h_q, d_qk, d_v, topk, _stream(stream))
    _check(st, "sparse_mla_fwd")
    return out, lse


def sparse_mla_bwd(q: torch.Tensor, kv: torch.Tensor, indices: torch.Tensor, sm_scale: float,
                   out: torch.Tensor, lse: torch.Tensor, dout: torch.Tensor,
                   dq: Optional[torch.Tensor] = None, dkv: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gradients of sparse_mla_fwd: q [s_q,h_q,576], kv [s_kv,576], indices
    [s_q,topk], the forward's out [s_q,h_q,512] bf16 and lse [s_q,h_q] fp32,
    dout [s_q,h_q,512] bf16 -> (dq [s_q,h_q,576] fp32, dkv [s_kv,576] fp32)."""
    lib = load()
    s_q, h_q, d_qk = q.shape
    s_kv = kv.shape[0]
    topk = indices.shape[-1]
    for t, dt, n in ((q, torch.bfloat16, "q"), (kv, torch.bfloat16, "kv"), (indices, torch.int32, "indices"),
                     (out, torch.bfloat16, "out"), (lse, torch.float32, "lse"), (dout, torch.bfloat16, "dout")):
        _need(t, dt, n)
    d_v = 512
    dev = q.device
    _fits(kv, s_kv * d_qk, "kv", dev)
    _fits(indices, s_q * topk, "indices", dev)
    _fits(out, s_q * h_q * d_v, "out", dev)
    _fits(lse, s_q * h_q, "lse", dev)
    _fits(dout, s_q * h_q * d_v, "dout", dev)
    _given(dq, torch.float32, "dq", s_q * h_q * d_qk, dev)
    _given(dkv, torch.float32, "dkv", s_kv * d_qk, dev)
    if dq is None:
        dq = torch.empty((s_q, h_q, d_qk), dtype=torch.float32, device=q.device)
    if dkv is None:
        dkv = torch.empty((s_kv, d_qk), dtype=torch.float32, device=q.device)
    st = lib.sparse_mla_bwd(_ptr(q), _ptr(kv), _ptr(indices), _ptr(out), _ptr(lse), _ptr(dout), float(sm_scale),
                            _ptr(dq), _ptr(dkv), s_q, s_kv, h_q, d_qk, d_v, topk, _stream(stream))
    _check(st, "sparse_mla_bwd")
    return dq, dkv


def sparse_mla_bwd_varlen(q, kv, indices, cu_seqlens_q, cu_seqlens_kv, sm_scale, out, lse, dout,
                          dq=None, dkv=None, stream=None):
    """Backward of sparse_mla_fwd_varlen -> (dq [total_q,h_q,576] fp32,
    dkv [total_kv,576] fp32)."""
    lib = load()
    total_q, h_q, d_qk = q.shape
    total_kv = kv.shape[0]
    topk = indices.shape[-1]
    batch = cu_seqlens_q.numel() - 1
    for t, dt, n in ((q, torch.bfloat16, "q"), (kv, torch.bfloat16, "kv"), (indices, torch.int32, "indices"),
                     (cu_seqlens_q, torch.int32, "cu_seqlens_q"), (cu_seqlens_kv, torch.int32, "cu_seqlens_kv"),
                     (out, torch.bfloat16, "out"), (lse, torch.float32, "lse"), (dout, torch.bfloat16, "dout")):
        _need(t, dt, n)
    dev = q.device
    _fits(kv, total_kv * d_qk, "kv", dev)
    _fits(indices, total_q * topk, "indices", dev)
    _fits(cu_seqlens_q, batch + 1, "cu_seqlens_q", dev)
    _fits(cu_seqlens_kv, batch + 1, "cu_seqlens_kv", dev)
    _fits(out, total_q * h_q * 512, "out", dev)
    _fits(lse, total_q * h_q, "lse", dev)
    _fits(dout, total_q * h_q * 512, "dout", dev)
    _given(dq, torch.float32, "dq", total_q * h_q * d_qk, dev)
    _given(dkv, torch.float32, "dkv", total_kv * d_qk, dev)
    if dq is None:
        dq = torch.empty((total_q, h_q, d_qk), dtype=torch.float32, device=q.device)
    if dkv is None:
        dkv = torch.empty((total_kv, d_qk), dtype=torch.float32, device=q.device)
    st = lib.sparse_mla_bwd_varlen(_ptr(q), _ptr(kv), _ptr(indices), _ptr(cu_seqlens_q), _ptr(cu_seqlens_kv),
                                   batch, _ptr(out), _ptr(lse), _ptr(dout), float(sm_scale), _ptr(dq), _ptr(dkv),
                                   total_q, total_kv, h_q, d_qk, 512, topk, _stream(stream))
    _check(st, "sparse_mla_bwd_varlen")
    return dq, dkv


def sparse_mla_fwd_causal(q: torch.Tensor, kv: torch.Tensor, sm_scale: float,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Indices-free causal forward: q [s_q,h_q,576] bf16 (the last s_q of the
    s_kv positions), kv [s_kv,576] or [s_kv,1,576] bf16 -> (out [s_q,h_q,512]
    bf16, lse [s_q,h_q] fp32)."""
    lib = load()
    s_q, h_q, d_qk = q.shape
    s_kv = kv.shape[0]
    for t, dt, n in ((q, torch.bfloat16, "q"), (kv, torch.bfloat16, "kv")):
        _need(t, dt, n)
    d_v = 512
    dev = q.device
    _fits(kv, s_kv * d_qk, "kv", dev)
    _given(out, torch.bfloat16, "out", s_q * h_q * d_v, dev)
    _given(lse, torch.float32, "lse", s_q * h_q, dev)
    if out is None:
        out = torch.empty((s_q, h_q, d_v), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((s_q, h_q), dtype=torch.float32, device=q.device)
    st = lib.sparse_mla_fwd_causal(_ptr(q), _ptr(kv), float(sm_scale), _ptr(out), _ptr(lse),
                                   s_q, s_kv, h_q, d_qk, d_v, _stream(stream))
    _check(st, "sparse_mla_fwd_causal")
    return out, lse


def sparse_mla_fwd_varlen(q, kv, indices, cu_seqlens_q, cu_seqlens_kv, sm_scale, out=None, lse=None,
                          stream=None):
    """Packed prefill; indices are local to each token's sequence."""
    lib = load()
    total_q, h_q, d_qk = q.shape
    total_kv = kv.shape[0]
    topk = indices.shape[-1]
    batch = cu_seqlens_q.numel() - 1
    for t, dt, n in ((q, torch.bfloat16, "q"), (kv, torch.bfloat16, "kv"), (indices, torch.int32, "indices"),
                     (cu_seqlens_q, torch.int32, "cu_seqlens_q"), (cu_seqlens_kv, torch.int32, "cu_seqlens_kv")):
        _need(t, dt, n)
    dev = q.device
    _fits(kv, total_kv * d_qk, "kv", dev)
    _fits(indices, total_q * topk, "indices", dev)
    _fits(cu_seqlens_q, batch + 1, "cu_seqlens_q", dev)
    _fits(cu_seqlens_kv, batch + 1, "cu_seqlens_kv", dev)
    _given(out, torch.bfloat16, "out", total_q * h_q * 512, dev)
    _given(lse, torch.float32, "lse", total_q * h_q, dev)
    if out is None:
        out = torch.empty((total_q, h_q, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((total_q, h_q), dtype=torch.float32, device=q.device)
    st = lib.sparse_mla_fwd_varlen(_ptr(q), _ptr(kv), _ptr(indices), _ptr(cu_seqlens_q), _ptr(cu_seqlens_kv),
                                   batch, float(sm_scale), _ptr(out), _ptr(lse), total_q, total_kv, h_q, d_qk,
                                   512, topk, _stream(stream))
    _check(st, "sparse_mla_fwd_varlen")
    return out, lse


def decode_workspace_size(batch: int, s_next: int, h_q: int, topk: int, d_v: int = 512) -> int:
    return int(load().sparse_mla_decode_workspace_size(batch, s_next, h_q, d_v, topk))


def sparse_mla_decode(q, kv_cache, block_table, cache_seqlens, indices, sm_scale, page_size=None,
                      workspace: Optional[torch.Tensor] = None, out=None, lse=None, stream=None):
    """Paged decode.  q [b,s_next,h_q,576]; kv_cache [num_blocks,page,576]
    (or [num_blocks,page,1,576]); block_table [b,max_blocks];
    cache_seqlens [b]; indices [b,s_next,topk] logical positions."""
    lib = load()
    batch, s_next, h_q, d_qk = q.shape
    num_blocks = kv_cache.shape[0]
    page = kv_cache.shape[1] if page_size is None else page_size
    max_blocks = block_table.shape[1]
    topk = indices.shape[-1]
    for t, dt, n in ((q, torch.bfloat16, "q"), (kv_cache, torch.bfloat16, "kv_cache"),
                     (block_table, torch.int32, "block_table"), (cache_seqlens, torch.int32, "cache_seqlens"),
                     (indices, torch.int32, "indices")):
        _need(t, dt, n)
    dev = q.device
    _fits(kv_cache, num_blocks * page * d_qk, "kv_cache", dev)
    _fits(block_table, batch * max_blocks, "block_table", dev)
    _fits(cache_seqlens, batch, "cache_seqlens", dev)
    _fits(indices, batch * s_next * topk, "indices", dev)
    _given(out, torch.bfloat16, "out", batch * s_next * h_q * 512, dev)
    _given(lse, torch.float32, "lse", batch * s_next * h_q, dev)
    _workspace(workspace, dev)
    if out is None:
        out = torch.empty((batch, s_next, h_q, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((batch, s_next, h_q), dtype=torch.float32, device=q.device)
    need = lib.sparse_mla_decode_workspace_size(batch, s_next, h_q, 512, topk)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.sparse_mla_decode(_ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(cache_seqlens), _ptr(indices),
                               float(sm_scale), _ptr(out), _ptr(lse), batch, s_next, h_q, d_qk, 512, topk, page,
                               max_blocks, num_blocks, _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "sparse_mla_decode")
    return out, lse


FP8_SLOT_BYTES = 656


def sparse_mla_decode_fp8(q, kv_cache, block_table, cache_seqlens, indices, sm_scale, page_size=None,
                          workspace: Optional[torch.Tensor] = None, out=None, lse=None, stream=None):
    """Paged decode over an FP8 cache: kv_cache uint8 [num_blocks, page, 656]
    (512 e4m3 codes, 4 fp32 tile scales, 64 bf16 rope values per slot);
    everything else as sparse_mla_decode."""
    lib = load()
    batch, s_next, h_q, d_qk = q.shape
    num_blocks = kv_cache.shape[0]
    page = kv_cache.shape[1] if page_size is None else page_size
    max_blocks = block_table.shape[1]
    topk = indices.shape[-1]
    for t, dt, n in ((q, torch.bfloat16, "q"), (kv_cache, torch.uint8, "kv_cache"),
                     (block_table, torch.int32, "block_table"), (cache_seqlens, torch.int32, "cache_seqlens"),
                     (indices, torch.int32, "indices")):
        _need(t, dt, n)
    if kv_cache.shape[-1] != FP8_SLOT_BYTES:
        raise ValueError(f"kv_cache slots must be {FP8_SLOT_BYTES} bytes, got {kv_cache.shape[-1]}")
    dev = q.device
    _fits(kv_cache, num_blocks * page * FP8_SLOT_BYTES, "kv_cache", dev)
    _fits(block_table, batch * max_blocks, "block_table", dev)
    _fits(cache_seqlens, batch, "cache_seqlens", dev)
    _fits(indices, batch * s_next * topk, "indices", dev)
    _given(out, torch.bfloat16, "out", batch * s_next * h_q * 512, dev)
    _given(lse, torch.float32, "lse", batch * s_next * h_q, dev)
    _workspace(workspace, dev)
    if out is None:
        out = torch.empty((batch, s_next, h_q, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((batch, s_next, h_q), dtype=torch.float32, device=q.device)
    need = lib.sparse_mla_decode_workspace_size(batch, s_next, h_q, 512, topk)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.sparse_mla_decode_fp8(_ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(cache_seqlens), _ptr(indices),
                                   float(sm_scale), _ptr(out), _ptr(lse), batch, s_next, h_q, d_qk, 512, topk, page,
                                   max_blocks, num_blocks, _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "sparse_mla_decode_fp8")
    return out, lse


# ---------------------------------------------------------------- 4-bit cache decode

FP4_SLOT_BYTES = 416
_BF16, _F32, _I32, _U8, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float8_e4m3fn


def _at(t: Optional[torch.Tensor]):
    """The address as the number that ctypes takes for a pointer argument."""
    return None if t is None else t.data_ptr()


# A decode step's calls take a few microseconds on the GPU, and a tensor's every
# attribute costs the host about a tenth of one: the entry points below first ask
# in one expression whether all is as it should be, and only where it is not go
# through the checks that say what is wrong.

def _dense(t: torch.Tensor, dtype, need: int, dev) -> bool:
    return t.dtype is dtype and t.device == dev and t.is_contiguous() and t.numel() >= need


class _launch_on:
    """The stream a call launches on, current meanwhile with its device (the
    library launches on the current device, and what the call allocates then
    belongs to the stream that uses it): `stream`, or the current stream of
    the tensors' device."""

    __slots__ = ("device", "stream", "guard")

    def __init__(self, device, stream):
        if stream is not None:
            on = getattr(stream, "device", None)
            if on is not None and on != device and _device_key(on) != _device_key(device):
                raise ValueError(f"stream is on {on}; the call's tensors are on {device}")
        self.device, self.stream, self.guard = device, stream, None

    def __enter__(self):
        dev = self.device
        if isinstance(self.stream, torch.cuda.Stream):
            self.guard = torch.cuda.stream(self.stream)
        elif dev.type == "cuda" and dev.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(dev)
        if self.guard is not None:
            self.guard.__enter__()
        if self.stream is not None:
            return self.stream.cuda_stream
        return torch.cuda.current_stream(dev).cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _launch(go, dev, stream, where: str):
    """go(stream handle) -> (status, results) with `dev` and the stream current;
    outputs and workspaces that the call allocates are made in go."""
    if stream is None and dev.index == torch._C._cuda_getDevice():
        st, results = go(torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        with _launch_on(dev, stream) as cs:
            st, results = go(cs)
    if st != 0:
        raise SparseMLAError(st, where)
    return results


def _run(call, dev, stream, where: str, *args):
    """call(stream handle, *args) -> (status, results), as _launch has it, without a closure."""
    if stream is None and dev.index == torch._C._cuda_getDevice():
        st, results = call(torch._C._cuda_getCurrentRawStream(dev.index), *args)
    else:
        with _launch_on(dev, stream) as cs:
            st, results = call(cs, *args)
    if st != 0:
        raise SparseMLAError(st, where)
    return results


def decode_fp4_workspace_size(batch: int, s_next: int, h_q: int, topk: int, d_v: int = 512) -> int:
    """Bytes sparse_mla_decode_fp4 needs on the current device."""
    return int(load().sparse_mla_decode_fp4_workspace_size(batch, s_next, h_q, d_v, topk))


def sparse_mla_decode_fp4(q, kv_cache, block_table, cache_seqlens, indices, sm_scale, page_size=None,
                          kv_scale: float = 1.0, workspace: Optional[torch.Tensor] = None, out=None, lse=None,
                          stream=None):
    """Paged decode over a 4-bit cache: kv_cache uint8 [num_blocks, page, 416]
    (512 e2m1 codes, 32 e4m3 scales, 64 bf16 rope values per slot, as
    mla_norm_rope writes them), a row's latent values code * scale *
    kv_scale; everything else as sparse_mla_decode."""
    lib = load()
    batch, s_next, h_q, d_qk = q.shape
    cache_shape = kv_cache.shape
    num_blocks = cache_shape[0]
    page = cache_shape[1] if page_size is None else page_size
    max_blocks = block_table.shape[1]
    topk = indices.shape[-1]
    dev = q.device
    if not (q.is_cuda and q.dtype is _BF16 and q.is_contiguous() and cache_shape[-1] == FP4_SLOT_BYTES
            and _dense(kv_cache, _U8, num_blocks * page * FP4_SLOT_BYTES, dev)
            and _dense(block_table, _I32, batch * max_blocks, dev) and _dense(cache_seqlens, _I32, batch, dev)
            and _dense(indices, _I32, batch * s_next * topk, dev)):
        for t, dt, n in ((q, _BF16, "q"), (kv_cache, _U8, "kv_cache"), (block_table, _I32, "block_table"),
                         (cache_seqlens, _I32, "cache_seqlens"), (indices, _I32, "indices")):
            _need(t, dt, n)
        if cache_shape[-1] != FP4_SLOT_BYTES:
            raise ValueError(f"kv_cache slots must be {FP4_SLOT_BYTES} bytes, got {cache_shape[-1]}")
        _fits(kv_cache, num_blocks * page * FP4_SLOT_BYTES, "kv_cache", dev)
        _fits(block_table, batch * max_blocks, "block_table", dev)
        _fits(cache_seqlens, batch, "cache_seqlens", dev)
        _fits(indices, batch * s_next * topk, "indices", dev)
    _given(out, _BF16, "out", batch * s_next * h_q * 512, dev)
    _given(lse, _F32, "lse", batch * s_next * h_q, dev)
    _workspace(workspace, dev)

    def go(cs):
        o = torch.empty((batch, s_next, h_q, 512), dtype=_BF16, device=dev) if out is None else out
        ls = torch.empty((batch, s_next, h_q), dtype=_F32, device=dev) if lse is None else lse
        ws = workspace
        if ws is None:
            need = lib.sparse_mla_decode_fp4_workspace_size(batch, s_next, h_q, 512, topk)
            if need > 0:
                ws = torch.empty(need, dtype=_U8, device=dev)
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
        return lib.sparse_mla_decode_fp4(q.data_ptr(), kv_cache.data_ptr(), block_table.data_ptr(),
                                         cache_seqlens.data_ptr(), indices.data_ptr(), sm_scale, kv_scale,
                                         o.data_ptr(), ls.data_ptr(), batch, s_next, h_q, d_qk, 512, topk, page,
                                         max_blocks, num_blocks, _at(ws), ws_bytes, cs), (o, ls)

    return _launch(go, dev, stream, "sparse_mla_decode_fp4")


# ---------------------------------------------------------------- norms, rotation, cache write

_CACHE_FORMATS = {(torch.bfloat16, 576): 0, (torch.uint8, FP8_SLOT_BYTES): 1, (torch.uint8, FP4_SLOT_BYTES): 2}
_ZERO_Q_PADDING, _ZERO_KV_PADDING = 0x100, 0x200


def _rows(t: torch.Tensor, name: str, heads: bool):
    """(token stride, head stride) in elements of bf16 rows of 576 values:
    [n, h, 576] with `heads`, else [n, 576] or [n, 1, 576].  The values of a
    row are contiguous; rows start on 16 bytes."""
    _on_cuda(t, name)
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    shape, steps = t.shape, t.stride()
    if not heads and len(shape) == 3 and shape[1] == 1:
        shape, steps = (shape[0], shape[2]), (steps[0], steps[2])
    if len(shape) != (3 if heads else 2) or shape[-1] != 576:
        raise ValueError(f"{name} must be {'[n, h, 576]' if heads else '[n, 576]'}, got {tuple(t.shape)}")
    if steps[-1] != 1:
        raise ValueError(f"the 576 values of a row of {name} must be contiguous")
    tok = steps[0] if shape[0] > 1 else 0
    head = steps[1] if heads and shape[1] > 1 else 0
    if tok % 8 or head % 8 or t.data_ptr() % 16:
        raise ValueError(f"rows of {name} must start on 16 bytes (strides {t.stride()})")
    return tok, head


def _is_weight(w, dev) -> bool:
    return w is None or (w.dtype is _BF16 and w.device == dev and w.is_contiguous() and w.numel() == 512)


def _norm_args(q, kv, positions, cos_sin, q_weight, kv_weight):
    """(tokens, heads, device, strides of q, token stride of kv) of checked arguments."""
    qs, qt, ks, kt, dev = q.shape, q.stride(), kv.shape, kv.stride(), q.device
    if (q.is_cuda and q.dtype is _BF16 and kv.dtype is _BF16 and len(qs) == 3 and len(ks) == 2 and qs[2] == 576
            and ks[1] == 576 and qs[0] == ks[0] and qt[2] == 1 and kt[1] == 1 and not (qt[0] | qt[1] | kt[0]) & 7
            and not (q.data_ptr() | kv.data_ptr()) & 15 and kv.device == dev
            and _dense(positions, _I32, qs[0], dev) and _dense(cos_sin, _F32, 0, dev) and cos_sin.dim() == 2
            and cos_sin.shape[1] == 64 and _is_weight(q_weight, dev) and _is_weight(kv_weight, dev)):
        return qs[0], qs[1], dev, qt[0], qt[1], kt[0]
    q_tok, q_head = _rows(q, "q", True)
    kv_tok, _ = _rows(kv, "kv", False)
    n = qs[0]
    if ks[0] != n:
        raise ValueError(f"kv has {ks[0]} rows; q has {n} tokens")
    _fits(kv, 0, "kv", dev)
    _need(positions, torch.int32, "positions")
    _fits(positions, n, "positions", dev)
    _need(cos_sin, torch.float32, "cos_sin")
    if cos_sin.dim() != 2 or cos_sin.shape[1] != 64:
        raise ValueError(f"cos_sin must be [n_pos, 64], got {tuple(cos_sin.shape)}")
    _fits(cos_sin, 0, "cos_sin", dev)
    for w, name in ((q_weight, "q_weight"), (kv_weight, "kv_weight")):
        if w is not None:
            _given(w, torch.bfloat16, name, 512, dev)
            if w.numel() != 512:
                raise ValueError(f"{name} must hold 512 values, got {w.numel()}")
    return n, qs[1], dev, q_tok, q_head, kv_tok


def mla_norm_rope(q, kv, positions, cos_sin, q_weight=None, kv_weight=None, eps: float = 1e-6,
                  interleaved: bool = True, kv_cache: Optional[torch.Tensor] = None,
                  slots: Optional[torch.Tensor] = None, kv_scale: float = 1.0, q_out=None, kv_out=None, stream=None):
    """RMS norm of every query head's row and of the latent row (their first
    512 values; a weight that is None leaves its rows unnormed), the position
    rotation of their last 64, and the latent row's write into its cache slot.

    q [n, h, 576] and kv [n, 576] (or [n, 1, 576]) bf16, rows strided as they
    are; positions [n] int32 (outside [0, n_pos): a padding token, left as it
    was in outputs that are given, zeros in those made here); cos_sin [n_pos, 64] fp32, 32 cosines then 32 sines; kv_cache
    [num_blocks, page, w]: bf16 with w = 576, or uint8 with w = 656 (FP8) or
    416 (4 bits, with its factor kv_scale); slots [n] int32, distinct (outside
    the cache: not stored).  -> (q_out [n, h, 576], kv_out [n, 576]), bf16;
    kv_out holds what the slots stand for, rounded to bf16 (4-bit slots with a
    factor that is not a power of two have more bits).  q_out / kv_out may be q / kv."""
    lib = load()
    n, h, dev, q_tok, q_head, kv_tok = _norm_args(q, kv, positions, cos_sin, q_weight, kv_weight)
    form, n_slots = 0, 0
    if kv_cache is not None:
        width = kv_cache.shape[-1]
        form = _CACHE_FORMATS.get((kv_cache.dtype, width), -1)
        if form < 0:
            raise ValueError("kv_cache must be bf16 [.., 576] or uint8 [.., 656] or [.., 416], got "
                             f"{kv_cache.dtype} {tuple(kv_cache.shape)}")
        if slots is None:
            raise ValueError("kv_cache is given without slots")
        _given(kv_cache, kv_cache.dtype, "kv_cache", 0, dev)
        _given(slots, _I32, "slots", n, dev)
        n_slots = kv_cache.numel() // width
        if n_slots > 2 ** 31 - 1:
            raise ValueError("a cache of more than 2^31 - 1 slots")
    elif slots is not None:
        raise ValueError("slots are given without kv_cache")
    # padding tokens' rows of outputs made here are zeros
    form |= (_ZERO_Q_PADDING if q_out is None else 0) | (_ZERO_KV_PADDING if kv_out is None else 0)
    _given(q_out, _BF16, "q_out", n * h * 576, dev)
    _given(kv_out, _BF16, "kv_out", n * 576, dev)

    def go(cs):
        qo = torch.empty((n, h, 576), dtype=_BF16, device=dev) if q_out is None else q_out
        ko = torch.empty((n, 576), dtype=_BF16, device=dev) if kv_out is None else kv_out
        return lib.mla_norm_rope(q.data_ptr(), q_tok, q_head, kv.data_ptr(), kv_tok, positions.data_ptr(),
                                 cos_sin.data_ptr(), cos_sin.shape[0], _at(q_weight), _at(kv_weight), eps,
                                 1 if interleaved else 0, qo.data_ptr(), ko.data_ptr(), _at(kv_cache), form,
                                 kv_scale, _at(slots), n_slots, n, h, 576, cs), (qo, ko)

    return _launch(go, dev, stream, "mla_norm_rope")


def norm_rope_bwd_workspace_size(n_tok: int, h_q: int) -> int:
    """Bytes mla_norm_rope_bwd needs on the current device."""
    return int(load().mla_norm_rope_bwd_workspace_size(n_tok, h_q))


def mla_norm_rope_bwd(q, kv, positions, cos_sin, dq, dkv, q_weight=None, kv_weight=None, eps: float = 1e-6,
                      interleaved: bool = True, workspace: Optional[torch.Tensor] = None, dq_in=None, dkv_in=None,
                      dq_weight=None, dkv_weight=None, stream=None):
    """Gradients of mla_norm_rope from dq [n, h, 576] and dkv [n, 576] fp32 (as
    sparse_mla_bwd returns them) -> (dq_in [n, h, 576] bf16, dkv_in [n, 576]
    bf16, dq_weight [512] fp32 or None, dkv_weight [512] fp32 or None).
    Padding tokens get zero rows."""
    lib = load()
    n, h, dev, q_tok, q_head, kv_tok = _norm_args(q, kv, positions, cos_sin, q_weight, kv_weight)
    _given(dq, _F32, "dq", n * h * 576, dev)
    _given(dkv, _F32, "dkv", n * 576, dev)
    _given(dq_in, _BF16, "dq_in", n * h * 576, dev)
    _given(dkv_in, _BF16, "dkv_in", n * 576, dev)
    if (q_weight is None and dq_weight is not None) or (kv_weight is None and dkv_weight is not None):
        raise ValueError(f"{'dq_weight' if q_weight is None and dq_weight is not None else 'dkv_weight'} is given "
                         "without its weight")
    _given(dq_weight, _F32, "dq_weight", 512, dev)
    _given(dkv_weight, _F32, "dkv_weight", 512, dev)
    _workspace(workspace, dev)

    def go(cs):
        dqi = torch.empty((n, h, 576), dtype=_BF16, device=dev) if dq_in is None else dq_in
        dki = torch.empty((n, 576), dtype=_BF16, device=dev) if dkv_in is None else dkv_in
        dqw, dkw = dq_weight, dkv_weight
        if q_weight is not None and dqw is None:
            dqw = torch.empty(512, dtype=_F32, device=dev)
        if kv_weight is not None and dkw is None:
            dkw = torch.empty(512, dtype=_F32, device=dev)
        ws = workspace
        if ws is None and (q_weight is not None or kv_weight is not None):
            ws = torch.empty(max(16, lib.mla_norm_rope_bwd_workspace_size(n, h)), dtype=_U8, device=dev)
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
        return lib.mla_norm_rope_bwd(q.data_ptr(), q_tok, q_head, kv.data_ptr(), kv_tok, positions.data_ptr(),
                                     cos_sin.data_ptr(), cos_sin.shape[0], _at(q_weight), _at(kv_weight), eps,
                                     1 if interleaved else 0, dq.data_ptr(), dkv.data_ptr(), dqi.data_ptr(),
                                     dki.data_ptr(), _at(dqw), _at(dkw), n, h, 576, _at(ws),
                                     ws_bytes, cs), (dqi, dki, dqw, dkw)

    return _launch(go, dev, stream, "mla_norm_rope_bwd")


# ---------------------------------------------------------------- residual norm

_INT_MAX = 2 ** 31 - 1


def _countable(**sizes) -> None:
    """Sizes go to the library as 32-bit counts, and ctypes cuts what has more bits: it
    would take 2^32 + 5 rows for 5."""
    for name, n in sizes.items():
        if n > _INT_MAX:
            raise ValueError(f"{name} is {n}; the library counts to 2^31 - 1")


def _wide_rows(t: torch.Tensor, n: int, d: int, name: str, dev) -> int:
    """Row stride in elements of bf16 rows [n, d], contiguous in themselves, each on 16 bytes."""
    _on_cuda(t, name)
    if t.dtype != _BF16:
        raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")
    _fits(t, 0, name, dev)
    if tuple(t.shape) != (n, d):
        raise ValueError(f"{name} must be [{n}, {d}], got {tuple(t.shape)}")
    step = t.stride(0) if n > 1 else 0
    if n > 0 and ((d > 1 and t.stride(1) != 1) or step % 8 or t.data_ptr() % 16):
        raise ValueError(f"rows of {name} must be contiguous and start on 16 bytes (strides {t.stride()})")
    return step


def _norm_rows(x, weight, others, names):
    """(n, d, device, row strides of x and of the others) of checked rows [n, d] and their weight [d]."""
    shape, dev = x.shape, x.device
    if len(shape) != 2:
        raise ValueError(f"{names[0]} must be [n, d], got {tuple(shape)}")
    n, d = shape
    if n > _INT_MAX or d > _INT_MAX:
        _countable(n=n, d=d)
    step, one = x.stride()
    bits = step & 7 | x.data_ptr() & 15
    good = (x.is_cuda and x.dtype is _BF16 and one == 1 and weight.dtype is _BF16 and weight.device == dev
            and weight.numel() == d and weight.is_contiguous())
    steps = [step]
    for t in others:
        if t is None:
            steps.append(0)
            continue
        if not (t.dtype is _BF16 and t.device == dev and t.shape == shape):
            good = False
            break
        step, one = t.stride()
        good = good and one == 1
        bits |= step & 7 | t.data_ptr() & 15
        steps.append(step)
    if good and not bits:
        return n, d, dev, steps
    steps = [_wide_rows(x, n, d, names[0], dev)]
    _given(weight, _BF16, "weight", d, dev)
    if weight.numel() != d:
        raise ValueError(f"weight must hold {d} values, got {weight.numel()}")
    steps += [0 if t is None else _wide_rows(t, n, d, name, dev) for t, name in zip(others, names[1:])]
    return n, d, dev, steps


def _apart(out: Optional[torch.Tensor], name: str, size: int, inputs, same=()) -> None:
    """A given output's first `size` bytes may not meet memory that the call still
    reads: `inputs` are (tensor, name).  An output of whole rows may be one of `same`,
    dense and at the same address (each row is read before it is written)."""
    if out is None:
        return
    at = out.data_ptr()
    for t, what in inputs:
        if t is None:
            continue
        lo, hi = _span(t)
        if at < hi and lo < at + size:
            if not (what in same and lo == at and t.is_contiguous()):
                raise ValueError(f"{name} shares memory with {what}"
                                 + (" other than as the same dense tensor" if what in same else ""))


def mla_add_norm(x, weight, residual=None, eps: float = 1e-6, group: Optional[int] = None, out=None, scales=None,
                 residual_out=None, stream=None):
    """z = x + residual (bf16), y = z * rsqrt(mean(z^2) + eps) * weight over rows [n, d].

    x and residual bf16, rows strided as they are; weight [d] bf16.  group None: out
    is y in bf16; 128 or 0: out is float8_e4m3fn, y's codes under a power-of-two
    scale for each 128 values of a row (the last group may be shorter), or for each
    row.  -> (out [n, d], scales [n, ceil(d / 128)] or [n, 1] fp32 or None,
    residual_out [n, d] bf16: z, or x itself where no residual is given).
    residual_out may be x or residual."""
    n, d, dev, (x_step, res_step) = _norm_rows(x, weight, (residual,), ("x", "residual"))
    if group is None:
        form, n_scales, kind, width = 0, 0, _BF16, 2
    elif group == 128 or group == 0:
        form, n_scales, kind, width = (1, (d + 127) // 128, _E4M3, 1) if group else (2, 1, _E4M3, 1)
    else:
        raise ValueError(f"group must be None, 128 or 0, got {group}")
    if out is not None or scales is not None or residual_out is not None:
        _given(out, kind, "out", n * d, dev)
        if scales is not None and not form:
            raise ValueError("scales are given without a group")
        _given(scales, _F32, "scales", n * n_scales, dev)
        if residual is None and residual_out is not None:
            raise ValueError("residual_out is given without residual")
        _given(residual_out, _BF16, "residual_out", n * d, dev)
        reads = (x, "x"), (residual, "residual"), (weight, "weight")
        _apart(residual_out, "residual_out", 2 * n * d, reads, ("x", "residual"))
        reads += ((residual_out, "residual_out"),)
        _apart(out, "out", width * n * d, reads)
        _apart(scales, "scales", 4 * n * n_scales, reads + ((out, "out"),))

    return _run(_add_norm, dev, stream, "mla_add_norm", x, x_step, residual, res_step, weight, eps, out, scales, form,
                n_scales, kind, residual_out, n, d)


def _add_norm(cs, x, x_step, residual, res_step, weight, eps, out, scales, form, n_scales, kind, z, n, d):
    dev = x.device
    if out is None:
        out = torch.empty((n, d), dtype=kind, device=dev)
    if form and scales is None:
        scales = torch.empty((n, n_scales), dtype=_F32, device=dev)
    res_at = z_at = None
    if residual is None:
        z = x
    else:
        if z is None:
            z = torch.empty((n, d), dtype=_BF16, device=dev)
        res_at, z_at = residual.data_ptr(), z.data_ptr()
    return load().mla_add_norm(x.data_ptr(), x_step, res_at, res_step, weight.data_ptr(), eps, out.data_ptr(),
                               scales.data_ptr() if form else None, form, z_at, n, d, cs), (out, scales, z)


def add_norm_bwd_workspace_size(n: int, d: int) -> int:
    """Bytes mla_add_norm_bwd needs on the current device."""
    _countable(n=n, d=d)
    return int(load().mla_add_norm_bwd_workspace_size(n, d))


def mla_add_norm_bwd(z, weight, dout, dresidual=None, eps: float = 1e-6, workspace: Optional[torch.Tensor] = None,
                     dx=None, dweight=None, stream=None):
    """Gradients of mla_add_norm: z [n, d] is its sum (what it returned last),
    dout the gradient of its rows, dresidual the one that reaches z from later
    layers (or None), all bf16, rows strided as they are -> (dx [n, d] bf16, the
    gradient of x and of the residual alike, dweight [d] fp32).  dx may be dout or
    dresidual."""
    n, d, dev, (z_step, g_step, r_step) = _norm_rows(z, weight, (dout, dresidual), ("z", "dout", "dresidual"))
    if dx is not None or dweight is not None or workspace is not None:
        _given(dx, _BF16, "dx", n * d, dev)
        _given(dweight, _F32, "dweight", d, dev)
        _workspace(workspace, dev)
        reads = (z, "z"), (weight, "weight"), (dout, "dout"), (dresidual, "dresidual")
        _apart(dx, "dx", 2 * n * d, reads, ("dout", "dresidual"))
        reads += ((dx, "dx"),)
        _apart(dweight, "dweight", 4 * d, reads)
        if workspace is not None:
            _apart(workspace, "workspace", workspace.numel() * workspace.element_size(), reads + ((dweight, "dweight"),))

    return _run(_add_norm_bwd, dev, stream, "mla_add_norm_bwd", z, z_step, weight, eps, dout, g_step, dresidual, r_step, dx,
                dweight, workspace, n, d)


def _add_norm_bwd(cs, z, z_step, weight, eps, dout, g_step, dresidual, r_step, dx, dweight, ws, n, d):
    lib, dev = load(), z.device
    if dx is None:
        dx = torch.empty((n, d), dtype=_BF16, device=dev)
    if dweight is None:
        dweight = torch.empty(d, dtype=_F32, device=dev)
    if ws is None:
        ws = torch.empty(max(16, lib.mla_add_norm_bwd_workspace_size(n, d)), dtype=_U8, device=dev)
    return lib.mla_add_norm_bwd(z.data_ptr(), z_step, weight.data_ptr(), eps, dout.data_ptr(), g_step, _at(dresidual),
                                r_step, dx.data_ptr(), dweight.data_ptr(), n, d, ws.data_ptr(),
                                ws.numel() * ws.element_size(), cs), (dx, dweight)


# ---------------------------------------------------------------- dense causal attention

def _heads(t: torch.Tensor, name: str, dev):
    """(token stride, head stride) in elements of bf16 rows [tokens, heads, width]."""
    shape, (tok, head, one) = t.shape, t.stride() if t.dim() == 3 else (0, 0, 0)
    if (t.is_cuda and t.dtype is _BF16 and one == 1 and not (tok | head) & 7 and tok > 0 and head > 0
            and not t.data_ptr() & 15 and t.device == dev):
        return tok, head
    _on_cuda(t, name)
    if t.dtype != _BF16:
        raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, width], got {tuple(shape)}")
    _fits(t, 0, name, dev)
    if t.numel() == 0:
        return 0, 0
    if one != 1:
        raise ValueError(f"the values of a row of {name} must be contiguous")
    tok, head = tok if shape[0] > 1 else 0, head if shape[1] > 1 else 0
    if tok % 8 or head % 8 or t.data_ptr() % 16:
        raise ValueError(f"rows of {name} must start on 16 bytes (strides {t.stride()})")
    if (shape[0] > 1 and tok <= 0) or (shape[1] > 1 and head <= 0):
        raise ValueError(f"{name} repeats rows (strides {t.stride()}); shared heads are given once")
    return tok, head


def _mha_args(q, k, v, cu_seqlens_q, cu_seqlens_kv):
    """(total_q, total_kv, heads, kv heads, d_qk, d_v, batch, device, strides) of checked arguments."""
    dev = q.device
    if q.dim() == 3 and k.dim() == 3 and v.dim() == 3:
        (nq, hq, dq), (nk, hk, dk), (nv, hv, dv) = q.shape, k.shape, v.shape
        (qt, qh, q1), (kt, kh, k1), (vt, vh, v1) = q.stride(), k.stride(), v.stride()
        if nq > _INT_MAX or nk > _INT_MAX or hq > _INT_MAX or dq > _INT_MAX or dv > _INT_MAX:
            _countable(total_q=nq, total_kv=nk, h_q=hq, d_qk=dq, d_v=dv)
        if (q.is_cuda and q.dtype is _BF16 and k.dtype is _BF16 and v.dtype is _BF16 and k.device == dev
                and v.device == dev and dq == dk and nk == nv and hk == hv and hk > 0 and hq % hk == 0
                and q1 == 1 and k1 == 1 and v1 == 1 and not (qt | qh | kt | kh | vt | vh) & 7
                and qt > 0 and qh > 0 and kt > 0 and kh > 0 and vt > 0 and vh > 0
                and not (q.data_ptr() | k.data_ptr() | v.data_ptr()) & 15):
            if cu_seqlens_q is None and cu_seqlens_kv is None:
                return nq, nk, hq, hk, dq, dv, 1, dev, (qt, qh, kt, kh, vt, vh)
            if cu_seqlens_q is not None and cu_seqlens_kv is not None:
                n = cu_seqlens_q.numel()
                if (0 < n <= _INT_MAX and cu_seqlens_kv.numel() == n and _dense(cu_seqlens_q, _I32, n, dev)
                        and _dense(cu_seqlens_kv, _I32, n, dev)):
                    return nq, nk, hq, hk, dq, dv, n - 1, dev, (qt, qh, kt, kh, vt, vh)
    steps = _heads(q, "q", dev) + _heads(k, "k", dev) + _heads(v, "v", dev)
    total_q, h_q, d_qk = q.shape
    total_kv, h_kv, d_k = k.shape
    if d_k != d_qk:
        raise ValueError(f"k has rows of {d_k} values; q of {d_qk}")
    if tuple(v.shape[:2]) != (total_kv, h_kv):
        raise ValueError(f"v must be [{total_kv}, {h_kv}, width], got {tuple(v.shape)}")
    if h_kv == 0 or h_q % h_kv:
        raise ValueError(f"{h_q} query heads do not share {h_kv} key heads evenly")
    batch = _seq_args(cu_seqlens_q, cu_seqlens_kv, dev)
    _countable(batch=batch)
    if cu_seqlens_q is not None and cu_seqlens_kv.numel() != batch + 1:
        raise ValueError(f"cu_seqlens_kv holds {cu_seqlens_kv.numel()} offsets; cu_seqlens_q {batch + 1}")
    return total_q, total_kv, h_q, h_kv, d_qk, v.shape[2], batch, dev, steps


_MHA_FILL_OUT, _MHA_FILL_LSE = 1, 2


def _span(t: torch.Tensor):
    """First and last byte (exclusive) that a tensor's values lie in; its strides are not negative."""
    at = t.data_ptr()
    if t.numel() == 0:
        return at, at
    return at, at + t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))


def _separate(outs, reads) -> None:
    """Given outputs (tensor or None, bytes written, name) may not meet each other or what the
    call reads (tensor or None, name): a tile's rows are written while others still read."""
    taken = [(*_span(t), name) for t, name in reads if t is not None]
    for t, size, name in outs:
        if t is None:
            continue
        at = t.data_ptr()
        for lo, hi, what in taken:
            if at < hi and lo < at + size:
                raise ValueError(f"{name} shares memory with {what}")
        taken.append((at, at + size, name))


def dense_mha_fwd(q, k, v, sm_scale, cu_seqlens_q=None, cu_seqlens_kv=None, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, stream=None):
    """Causal attention over whole prompts in the heads' own space: q [total_q, h_q,
    192 or 128], k [total_kv, h_kv, the same], v [total_kv, h_kv, 128] bf16, rows
    strided as they are; h_q / h_kv query heads share a key and value head.
    cu_seqlens_q / cu_seqlens_kv int32 [batch + 1] for packed sequences (neither: one
    sequence); a sequence's queries are its last positions.  -> (out [total_q, h_q,
    128] bf16, lse [total_q, h_q] fp32).  Rows behind the last sequence are left as
    they were in outputs that are given, zeros and -inf in those made here.  Outputs that
    are given share no memory with each other or the inputs."""
    total_q, total_kv, h_q, h_kv, d_qk, d_v, batch, dev, steps = _mha_args(q, k, v, cu_seqlens_q, cu_seqlens_kv)
    if out is not None or lse is not None:
        _given(out, _BF16, "out", total_q * h_q * d_v, dev)
        _given(lse, _F32, "lse", total_q * h_q, dev)
        _separate(((out, 2 * total_q * h_q * d_v, "out"), (lse, 4 * total_q * h_q, "lse")),
                  ((q, "q"), (k, "k"), (v, "v"), (cu_seqlens_q, "cu_seqlens_q"), (cu_seqlens_kv, "cu_seqlens_kv")))
    fill = (_MHA_FILL_OUT if out is None else 0) | (_MHA_FILL_LSE if lse is None else 0)

    return _run(_mha_fwd, dev, stream, "dense_mha_fwd", q, k, v, steps, cu_seqlens_q, cu_seqlens_kv, batch, sm_scale, out,
                lse, fill, total_q, total_kv, h_q, h_kv, d_qk, d_v)


def _mha_fwd(cs, q, k, v, steps, cu_q, cu_kv, batch, sm_scale, out, lse, fill, total_q, total_kv, h_q, h_kv, d_qk, d_v):
    dev = q.device
    if out is None:
        out = torch.empty((total_q, h_q, d_v), dtype=_BF16, device=dev)
    if lse is None:
        lse = torch.empty((total_q, h_q), dtype=_F32, device=dev)
    qt, qh, kt, kh, vt, vh = steps
    return load().dense_mha_fwd(q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, _at(cu_q), _at(cu_kv),
                                batch, sm_scale, out.data_ptr(), lse.data_ptr(), fill, total_q, total_kv, h_q, h_kv, d_qk,
                                d_v, cs), (out, lse)


def dense_mha_bwd_workspace_size(total_q: int, total_kv: int, batch: int, h_q: int, h_kv: int, d_qk: int,
                                 d_v: int = 128) -> int:
    """Bytes dense_mha_bwd needs."""
    _countable(total_q=total_q, total_kv=total_kv, batch=batch, h_q=h_q, h_kv=h_kv, d_qk=d_qk, d_v=d_v)
    return int(load().dense_mha_bwd_workspace_size(total_q, total_kv, batch, h_q, h_kv, d_qk, d_v))


def dense_mha_bwd(q, k, v, sm_scale, out, lse, dout, cu_seqlens_q=None, cu_seqlens_kv=None,
                  dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                  dv: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of dense_mha_fwd from its out and lse and the gradient dout [total_q,
    h_q, 128] bf16 of out -> (dq, dk, dv), bf16, dense, of the shapes of q, k and v.
    Rows behind the last sequence get zeros."""
    total_q, total_kv, h_q, h_kv, d_qk, d_v, batch, dev, steps = _mha_args(q, k, v, cu_seqlens_q, cu_seqlens_kv)
    _given(out, _BF16, "out", total_q * h_q * d_v, dev)
    _given(lse, _F32, "lse", total_q * h_q, dev)
    steps += _heads(dout, "dout", dev)
    if dout.shape != (total_q, h_q, d_v):
        raise ValueError(f"dout must be [{total_q}, {h_q}, {d_v}], got {tuple(dout.shape)}")
    if dq is not None or dk is not None or dv is not None or workspace is not None:
        _given(dq, _BF16, "dq", total_q * h_q * d_qk, dev)
        _given(dk, _BF16, "dk", total_kv * h_kv * d_qk, dev)
        _given(dv, _BF16, "dv", total_kv * h_kv * d_v, dev)
        _workspace(workspace, dev)
        _separate(((dq, 2 * total_q * h_q * d_qk, "dq"), (dk, 2 * total_kv * h_kv * d_qk, "dk"),
                   (dv, 2 * total_kv * h_kv * d_v, "dv"),
                   (workspace, 0 if workspace is None else workspace.numel() * workspace.element_size(), "workspace")),
                  ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (lse, "lse"), (dout, "dout"),
                   (cu_seqlens_q, "cu_seqlens_q"), (cu_seqlens_kv, "cu_seqlens_kv")))
    return _run(_mha_bwd, dev, stream, "dense_mha_bwd", q, k, v, steps, cu_seqlens_q, cu_seqlens_kv, batch, sm_scale, out,
                lse, dout, dq, dk, dv, workspace, total_q, total_kv, h_q, h_kv, d_qk, d_v)


def _mha_bwd(cs, q, k, v, steps, cu_q, cu_kv, batch, sm_scale, out, lse, dout, dq, dk, dv, ws, total_q, total_kv, h_q, h_kv,
             d_qk, d_v):
    lib, dev = load(), q.device
    if dq is None:
        dq = torch.empty((total_q, h_q, d_qk), dtype=_BF16, device=dev)
    if dk is None:
        dk = torch.empty((total_kv, h_kv, d_qk), dtype=_BF16, device=dev)
    if dv is None:
        dv = torch.empty((total_kv, h_kv, d_v), dtype=_BF16, device=dev)
    if ws is None:
        need = lib.dense_mha_bwd_workspace_size(total_q, total_kv, batch, h_q, h_kv, d_qk, d_v)
        ws = torch.empty(max(16, need), dtype=_U8, device=dev)
    qt, qh, kt, kh, vt, vh, gt, gh = steps
    return lib.dense_mha_bwd(q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, _at(cu_q), _at(cu_kv), batch,
                             sm_scale, out.data_ptr(), lse.data_ptr(), dout.data_ptr(), gt, gh, dq.data_ptr(),
                             dk.data_ptr(), dv.data_ptr(), total_q, total_kv, h_q, h_kv, d_qk, d_v, ws.data_ptr(),
                             ws.numel() * ws.element_size(), cs), (dq, dk, dv)


# ---------------------------------------------------------------- debug: valid entries per token

def debug_valid_count(indices, s_kv: int, stream=None) -> torch.Tensor:
    """Valid entries of each token's list as the dense forward gathers them:
    indices [s_q, topk] int32 -> counts [s_q] int32."""
    lib = load()
    _need(indices, torch.int32, "indices")
    s_q, topk = indices.shape[0], indices.shape[-1]
    counts = torch.empty(s_q, dtype=torch.int32, device=indices.device)
    _check(lib.sparse_mla_debug_valid_count(_ptr(indices), s_q, int(s_kv), topk, _ptr(counts), _stream(stream)),
           "sparse_mla_debug_valid_count")
    return counts


def debug_valid_count_varlen(indices, cu_seqlens_q, cu_seqlens_kv, total_kv: int, stream=None) -> torch.Tensor:
    """As debug_valid_count for the packed layout of sparse_mla_fwd_varlen."""
    lib = load()
    for t, n in ((indices, "indices"), (cu_seqlens_q, "cu_seqlens_q"), (cu_seqlens_kv, "cu_seqlens_kv")):
        _need(t, torch.int32, n)
    total_q, topk = indices.shape[0], indices.shape[-1]
    batch = cu_seqlens_q.numel() - 1
    dev = indices.device
    _fits(cu_seqlens_q, batch + 1, "cu_seqlens_q", dev)
    _fits(cu_seqlens_kv, batch + 1, "cu_seqlens_kv", dev)
    counts = torch.empty(total_q, dtype=torch.int32, device=dev)
    _check(lib.sparse_mla_debug_valid_count_varlen(_ptr(indices), _ptr(cu_seqlens_q), _ptr(cu_seqlens_kv), batch,
                                                   total_q, int(total_kv), topk, _ptr(counts), _stream(stream)),
           "sparse_mla_debug_valid_count_varlen")
    return counts


def debug_valid_count_paged(indices, block_table, cache_seqlens, page_size: int, num_blocks: int,
                            stream=None) -> torch.Tensor:
    """As debug_valid_count for the paged layout of sparse_mla_decode:
    indices [b, s_next, topk] -> counts [b * s_next] int32."""
    lib = load()
    for t, n in ((indices, "indices"), (block_table, "block_table"), (cache_seqlens, "cache_seqlens")):
        _need(t, torch.int32, n)
    batch, s_next, topk = indices.shape
    max_blocks = block_table.shape[1]
    dev = indices.device
    _fits(block_table, batch * max_blocks, "block_table", dev)
    _fits(cache_seqlens, batch, "cache_seqlens", dev)
    counts = torch.empty(batch * s_next, dtype=torch.int32, device=dev)
    _check(lib.sparse_mla_debug_valid_count_paged(_ptr(indices), _ptr(block_table), _ptr(cache_seqlens), batch,
                                                  s_next, topk, int(page_size), max_blocks, int(num_blocks),
                                                  _ptr(counts), _stream(stream)),
           "sparse_mla_debug_valid_count_paged")
    return counts


# ---------------------------------------------------------------- DSA indexer

def _seq_args(cu_seqlens_q, cu_seqlens_kv, device=None):
    if (cu_seqlens_q is None) != (cu_seqlens_kv is None):
        raise ValueError("give both cu_seqlens_q and cu_seqlens_kv, or neither")
    if cu_seqlens_q is None:
        return 1
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q")
    _need(cu_seqlens_kv, torch.int32, "cu_seqlens_kv")
    batch = cu_seqlens_q.numel() - 1
    if device is not None:
        _fits(cu_seqlens_q, batch + 1, "cu_seqlens_q", device)
        _fits(cu_seqlens_kv, batch + 1, "cu_seqlens_kv", device)
    return batch


def _workspace(workspace: Optional[torch.Tensor], device) -> None:
    if workspace is not None:
        _need(workspace, workspace.dtype, "workspace")
        _fits(workspace, 0, "workspace", device)


def _longest_kv(k_idx_rows: int, cu_seqlens_kv, max_seqlen_kv):
    if max_seqlen_kv is not None:
        return int(max_seqlen_kv)
    if cu_seqlens_kv is None:
        return int(k_idx_rows)
    if cu_seqlens_kv.numel() < 2:
        return 0
    return int((cu_seqlens_kv[1:] - cu_seqlens_kv[:-1]).max().item())   # a device read


def dsa_indexer_scores(q_idx, k_idx, weights, cu_seqlens_q=None, cu_seqlens_kv=None, row0: int = 0,
                       n_rows: Optional[int] = None, skip_len: int = 0, scores=None,
                       max_seqlen_kv: Optional[int] = None, stream=None):
    """Indexer scores of rows row0 .. row0+n_rows-1: q_idx [total_q,h_idx,128]
    bf16, k_idx [total_kv,128] bf16, weights [total_q,h_idx] fp32 ->
    scores [n_rows, row_stride] fp32 (row_stride = longest KV sequence
    rounded up to 4); positions a row does not see, and rows seeing at most
    skip_len positions, keep the given contents (-inf when allocated here)."""
    lib = load()
    total_q, h_idx, d_idx = q_idx.shape
    total_kv = k_idx.shape[0]
    _need(q_idx, torch.bfloat16, "q_idx")
    _need(k_idx, torch.bfloat16, "k_idx")
    _need(weights, torch.float32, "weights")
    dev = q_idx.device
    _fits(k_idx, total_kv * d_idx, "k_idx", dev)
    _fits(weights, total_q * h_idx, "weights", dev)
    batch = _seq_args(cu_seqlens_q, cu_seqlens_kv, dev)
    n_rows = total_q - row0 if n_rows is None else n_rows
    stride = (_longest_kv(total_kv, cu_seqlens_kv, max_seqlen_kv) + 3) // 4 * 4
    if scores is None:
        scores = torch.full((n_rows, max(stride, 4)), float("-inf"), dtype=torch.float32, device=q_idx.device)
    else:
        _given(scores, torch.float32, "scores", max(n_rows, 0) * scores.shape[-1], dev)
    st = lib.dsa_indexer_scores(_ptr(q_idx), _ptr(k_idx), _ptr(weights), _ptr(cu_seqlens_q), _ptr(cu_seqlens_kv),
                                batch, total_q, total_kv, h_idx, d_idx, row0, n_rows, skip_len, _ptr(scores),
                                scores.shape[-1], _stream(stream))
    _check(st, "dsa_indexer_scores")
    return scores


def dsa_topk(scores, topk: int, total_q: int, total_kv: int, cu_seqlens_q=None, cu_seqlens_kv=None,
             row0: int = 0, n_rows: Optional[int] = None, indices=None, stream=None):
    """Lists of rows row0 .. row0+n_rows-1 from scores [n_rows, row_stride]
    fp32 -> indices [total_q, topk] int32 (only those rows written)."""
    lib = load()
    if scores is not None:
        _need(scores, torch.float32, "scores")
    n_rows = total_q - row0 if n_rows is None else n_rows
    dev = scores.device if scores is not None else (indices.device if indices is not None else torch.device("cuda"))
    batch = _seq_args(cu_seqlens_q, cu_seqlens_kv, dev)
    if scores is not None:
        _fits(scores, max(n_rows, 0) * scores.shape[-1], "scores", dev)
    if indices is None:
        indices = torch.full((total_q, topk), -2, dtype=torch.int32, device=dev)
    else:
        _given(indices, torch.int32, "indices", total_q * topk, dev)
    stride = scores.shape[-1] if scores is not None else 1
    st = lib.dsa_topk(_ptr(scores), stride, _ptr(cu_seqlens_q), _ptr(cu_seqlens_kv), batch, total_q, total_kv,
                      row0, n_rows, topk, _ptr(indices), _stream(stream))
    _check(st, "dsa_topk")
    return indices


def dsa_indexer_workspace_size(total_q: int, max_seqlen_kv: int, topk: int) -> int:
    return int(load().dsa_indexer_workspace_size(total_q, max_seqlen_kv, topk))


def dsa_indexer_topk(q_idx, k_idx, weights, topk: int, cu_seqlens_q=None, cu_seqlens_kv=None,
                     max_seqlen_kv: Optional[int] = None, workspace: Optional[torch.Tensor] = None,
                     indices=None, stream=None):
    """Index lists [total_q, topk] int32 of every query row (scores and
    top-k in query-row chunks sized by the workspace; a full-size workspace
    is allocated when none is given)."""
    lib = load()
    total_q, h_idx, d_idx = q_idx.shape
    total_kv = k_idx.shape[0]
    _need(q_idx, torch.bfloat16, "q_idx")
    _need(k_idx, torch.bfloat16, "k_idx")
    _need(weights, torch.float32, "weights")
    dev = q_idx.device
    _fits(k_idx, total_kv * d_idx, "k_idx", dev)
    _fits(weights, total_q * h_idx, "weights", dev)
    batch = _seq_args(cu_seqlens_q, cu_seqlens_kv, dev)
    longest = _longest_kv(total_kv, cu_seqlens_kv, max_seqlen_kv)
    if indices is None:
        indices = torch.empty((total_q, topk), dtype=torch.int32, device=q_idx.device)
    else:
        _given(indices, torch.int32, "indices", total_q * topk, dev)
    _workspace(workspace, dev)
    if workspace is None:
        need = lib.dsa_indexer_workspace_size(total_q, longest, topk)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q_idx.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = lib.dsa_indexer_topk(_ptr(q_idx), _ptr(k_idx), _ptr(weights), _ptr(cu_seqlens_q), _ptr(cu_seqlens_kv),
                              batch, total_q, total_kv, longest, h_idx, d_idx, topk, _ptr(indices),
                              _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "dsa_indexer_topk")
    return indices


def _paged_args(q_idx, k_cache, weights, block_table, cache_seqlens):
    _need(q_idx, torch.bfloat16, "q_idx")
    _need(k_cache, torch.bfloat16, "k_cache")
    _need(weights, torch.float32, "weights")
    _need(block_table, torch.int32, "block_table")
    _need(cache_seqlens, torch.int32, "cache_seqlens")
    batch, s_next, h_idx, d_idx = q_idx.shape
    num_blocks, page = k_cache.shape[0], k_cache.shape[1]
    max_blocks = block_table.shape[1]
    dev = q_idx.device
    _fits(k_cache, num_blocks * page * d_idx, "k_cache", dev)
    _fits(weights, batch * s_next * h_idx, "weights", dev)
    _fits(block_table, batch * max_blocks, "block_table", dev)
    _fits(cache_seqlens, batch, "cache_seqlens", dev)
    return batch, s_next, h_idx, d_idx, page, max_blocks, num_blocks


def dsa_indexer_scores_paged(q_idx, k_cache, weights, block_table, cache_seqlens, max_seqlen_kv: int,
                             row0: int = 0, n_rows: Optional[int] = None, skip_len: int = 0, scores=None,
                             stream=None):
    """Decode indexer scores over a paged key cache: q_idx [b,s_next,h_idx,128],
    k_cache [num_blocks,64,128], weights [b,s_next,h_idx], block_table
    [b,max_blocks], cache_seqlens [b] -> scores [n_rows, row_stride] fp32 over
    the flattened rows b*s_next + j (-inf where not written)."""
    lib = load()
    batch, s_next, h_idx, d_idx, page, max_blocks, num_blocks = _paged_args(q_idx, k_cache, weights, block_table,
                                                                            cache_seqlens)
    n_rows = batch * s_next - row0 if n_rows is None else n_rows
    stride = (int(max_seqlen_kv) + 3) // 4 * 4
    if scores is None:
        scores = torch.full((n_rows, max(stride, 4)), float("-inf"), dtype=torch.float32, device=q_idx.device)
    else:
        _given(scores, torch.float32, "scores", max(n_rows, 0) * scores.shape[-1], q_idx.device)
    st = lib.dsa_indexer_scores_paged(_ptr(q_idx), _ptr(k_cache), _ptr(weights), _ptr(block_table),
                                      _ptr(cache_seqlens), batch, s_next, h_idx, d_idx, page, max_blocks, num_blocks,
                                      row0, n_rows, skip_len, _ptr(scores), scores.shape[-1], _stream(stream))
    _check(st, "dsa_indexer_scores_paged")
    return scores


def dsa_indexer_topk_paged(q_idx, k_cache, weights, block_table, cache_seqlens, topk: int,
                           max_seqlen_kv: Optional[int] = None, workspace: Optional[torch.Tensor] = None,
                           indices=None, stream=None):
    """Decode index lists [b, s_next, topk] int32 over a paged key cache
    (positions local to each request)."""
    lib = load()
    batch, s_next, h_idx, d_idx, page, max_blocks, num_blocks = _paged_args(q_idx, k_cache, weights, block_table,
                                                                            cache_seqlens)
    if max_seqlen_kv is None:
        max_seqlen_kv = int(cache_seqlens.max().item()) if cache_seqlens.numel() else 0   # a device read
    if indices is None:
        indices = torch.empty((batch, s_next, topk), dtype=torch.int32, device=q_idx.device)
    else:
        _given(indices, torch.int32, "indices", batch * s_next * topk, q_idx.device)
    _workspace(workspace, q_idx.device)
    if workspace is None:
        need = lib.dsa_indexer_workspace_size(batch * s_next, int(max_seqlen_kv), topk)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q_idx.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = lib.dsa_indexer_topk_paged(_ptr(q_idx), _ptr(k_cache), _ptr(weights), _ptr(block_table),
                                    _ptr(cache_seqlens), batch, s_next, h_idx, d_idx, page, max_blocks, num_blocks,
                                    int(max_seqlen_kv), topk, _ptr(indices), _ptr(workspace), ws_bytes,
                                    _stream(stream))
    _check(st, "dsa_indexer_topk_paged")
    return indices


def get_device_error() -> int:
    code = c_int(0)
    _check(load().sparse_mla_get_device_error(ctypes.byref(code)), "sparse_mla_get_device_error")
    return code.value


def clear_device_error():
    _check(load().sparse_mla_clear_device_error(), "sparse_mla_clear_device_error")


def set_wait_timeout_ns(ns: int):
    load().sparse_mla_set_wait_timeout_ns(int(ns))
