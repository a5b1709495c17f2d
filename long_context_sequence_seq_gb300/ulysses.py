"""Thin ctypes binding over libulysses.so (argument marshalling only).

Every step of the path runs in the library's CUDA kernels; this module only
checks tensor properties, allocates outputs through PyTorch and passes raw
device pointers and the current CUDA stream.  Importing it does not load the
library; the first call does, and fails loudly if the library is missing.

Layouts: sequence layout [B, S, H, D] (P stacked rank chunks of S/P tokens),
head layout [B, n, S, D] (the n heads of one UPipe stage, or all heads).
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
import struct

import torch

from .build import fastcall_path

_PKG = os.path.dirname(os.path.abspath(__file__))
# ULYSSES_CHECKED=1 loads the bounds-checked build of the same library
LIB_PATH = os.path.join(_PKG, "libulysses_checked.so" if os.environ.get("ULYSSES_CHECKED") == "1"
                        else "libulysses.so")

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_BAD_SEQLENS, ERR_BOUNDS, ERR_BAD_PAGES = range(8)
BF16, FP32, E4M3, E2M1 = 0, 1, 2, 3
PAIRS_HALF, PAIRS_ADJACENT = 0, 1
KERNEL_AUTO, KERNEL_SIMT, KERNEL_NO_MULTICAST = 0, 1, 2

_lib = None
# C++ marshalling of the strided calls (_fastcall-*.so), bound to the loaded
# library; None where it has not been built: the Python marshalling serves then.
_fast = None


class RelayoutItem(ctypes.Structure):
    """ulysses_relayout_item: one tensor of a batched re-layout launch."""
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("H", ctypes.c_int),
                ("head_chunk", ctypes.c_int), ("stage", ctypes.c_int), ("add", ctypes.c_int)]


class RopeItem(ctypes.Structure):
    """ulysses_rope_item: one tensor of a rotary launch (element strides)."""
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("H", ctypes.c_int),
                ("src_b", ctypes.c_int64), ("src_s", ctypes.c_int64), ("src_h", ctypes.c_int64),
                ("dst_b", ctypes.c_int64), ("dst_s", ctypes.c_int64), ("dst_h", ctypes.c_int64)]


class UlyssesError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"ulysses error {code}: {msg}")
        self.code = code


def lib():
    """Load libulysses.so (built by ``build.build()``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "long_context_sequence_seq_gb300.build.build() (checked=True for the "
                           "bounds-checked variant)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.ulysses_seq2head.argtypes = [vp, vp, i64, i32, i32, i32, i32, i32, i32, i32, vp]
    L.ulysses_head2seq.argtypes = [vp, vp, i64, i32, i32, i32, i32, i32, i32, i32, vp]
    L.ulysses_head2seq_add.argtypes = [vp, vp, i64, i32, i32, i32, i32, i32, i32, i32, vp]
    L.ulysses_seq2head_n.argtypes = [ctypes.POINTER(RelayoutItem), i32, i64, i32, i32, i32, i32, vp]
    L.ulysses_head2seq_n.argtypes = [ctypes.POINTER(RelayoutItem), i32, i64, i32, i32, i32, i32, vp]
    L.ulysses_selftest_wait_timeout.argtypes = [i64, vp]
    L.ulysses_ring_workspace.argtypes = [i64, i32, i32, i32, i32, i32]
    L.ulysses_ring_workspace.restype = sz
    L.ulysses_ring_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, i32, f32, i32, vp, sz, vp]
    L.ulysses_ring_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, i32, f32, i32,
                                   vp, sz, vp]
    L.ulysses_pad_seq.argtypes = [vp, vp, i64, i64, i32, i32, i32, i32, vp]
    L.ulysses_pad_cu_seqlens.argtypes = [vp, i32, vp, i64, i64, vp]
    L.ulysses_lse_merge.argtypes = [vp, vp, vp, vp, i64, i32, i32, i32, vp]
    L.ulysses_cast_f32.argtypes = [vp, vp, i64, i32, vp]
    L.ulysses_add_f32.argtypes = [vp, vp, i64, vp]
    L.ulysses_qkv_proj.argtypes = [vp, vp, vp, i64, i32, i32, i32, i32, vp]
    L.ulysses_out_proj.argtypes = [vp, vp, vp, i64, i32, i32, i32, vp]
    L.ulysses_layer_fused_workspace.argtypes = [i64, i32, i32, i32, i32, i32, i32, i32]
    L.ulysses_layer_fused_workspace.restype = ctypes.c_size_t
    L.ulysses_layer_fwd_fused.argtypes = [vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, i32, i32, vp, i32,
                                          i32, ctypes.c_float, i32, vp]
    L.ulysses_layer_bwd_fused.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, i32,
                                          i32, vp, i32, i32, ctypes.c_float, i32, vp, ctypes.c_size_t, vp]
    L.ulysses_attn_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, i32, i32, i32,
                                   vp, i32, i32, f32, i32, vp]
    L.ulysses_attn_bwd_workspace.argtypes = [i64, i32, i32, i32, i32, i32, i32, i32, i32]
    L.ulysses_attn_bwd_workspace.restype = sz
    L.ulysses_attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i64, i32, i32,
                                   i32, i32, i32, i32, i32, vp, i32, i32, f32, i32, vp]
    L.ulysses_attn_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32,
                                           i32, i32, i32, i32, vp, i32, i32, f32, i32, vp]
    L.ulysses_layer_workspace.argtypes = [i64, i32, i32, i32, i32, i32, i32, i32]
    L.ulysses_layer_workspace.restype = sz
    L.ulysses_layer_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, i32, i32, vp,
                                    i32, i32, f32, i32, vp, sz, vp]
    L.ulysses_layer_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32,
                                    i32, i32, vp, i32, i32, f32, i32, vp, sz, vp]
    for fn in (L.ulysses_rope_fwd, L.ulysses_rope_bwd):
        fn.argtypes = [vp, i32, vp, i32, vp, vp, i32, i32, i64, i32, i32, i32, i32, vp]
    L.ulysses_cache_write.argtypes = [vp, vp, i64, i64, i64, i64, i64, i32, vp, vp, i32, vp, vp, vp, vp, vp, i64, i32,
                                      i32, i32, i32, i32, vp]
    L.ulysses_cache_read.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, i64, i32,
                                     i32, i32, i32, i32, vp]
    L.ulysses_attn_decode_workspace.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32]
    L.ulysses_attn_decode_workspace.restype = sz
    L.ulysses_attn_decode.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp, i32, vp, vp, i64, i64, vp, i32, i32, i32, i32,
                                      i64, i32, f32, i32, i32, vp, sz, vp]
    L.ulysses_cache_write_weights.argtypes = [vp, vp, i64, i64, i64, i64, i64, i32, vp, vp, i32, vp, vp, vp, vp, vp, vp, i64,
                                              i32, i32, i32, i32, i32, vp]
    L.ulysses_attn_decode_weights_workspace.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32]
    L.ulysses_attn_decode_weights_workspace.restype = sz
    L.ulysses_attn_decode_weights.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp, i32, vp, vp, i64, i64, vp, vp, i32, i32, i32,
                                              i32, i64, i32, f32, i32, i32, vp, sz, vp]
    L.ulysses_cache_evict_workspace.argtypes = [i32, i32, i32, i32]
    L.ulysses_cache_evict_workspace.restype = sz
    L.ulysses_cache_evict.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, vp, i32, vp, i32, i64, i32, i32, i32, i32, vp, sz, vp]
    L.ulysses_check.argtypes = [vp]
    L.ulysses_last_error.restype = ctypes.c_char_p
    L.ulysses_set_kernel.argtypes = [i32]
    L.ulysses_launch_count.restype = ctypes.c_longlong
    L.ulysses_checked_build.restype = ctypes.c_int
    _lib = L
    _bind_fast(L)
    return L


def _bind_fast(L):
    """Load the C++ marshalling built for this interpreter and torch, if it is
    there, and give it the library's functions."""
    global _fast
    path = fastcall_path()
    if not os.path.exists(path):
        return
    spec = importlib.util.spec_from_file_location(f"{__package__}._fastcall", path)
    try:
        _fastcall = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(_fastcall)
    except ImportError:
        return
    _fastcall.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        L.ulysses_rope_fwd, L.ulysses_rope_bwd, L.ulysses_cache_write, L.ulysses_cache_read, L.ulysses_attn_decode,
        L.ulysses_attn_decode_workspace, L.ulysses_cache_write_weights, L.ulysses_attn_decode_weights,
        L.ulysses_attn_decode_weights_workspace, L.ulysses_cache_evict, L.ulysses_cache_evict_workspace)))
    _fast = _fastcall


def _ck(rc):
    if rc != OK:
        raise UlyssesError(rc, lib().ulysses_last_error().decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _p(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _cu(cu_seqlens):
    if cu_seqlens is None:
        return None, 0
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    return _p(cu_seqlens), cu_seqlens.numel() - 1


def _stage(stage):
    return -1 if stage is None else int(stage)


# --------------------------------------------------------------- re-layout

def seq2head(x_seq, P, head_chunk=None, stage=None, out=None, stream=None):
    """All-to-all #1: [B,S,H,D] -> [B,n,S,D] for the stage (all heads if None).
    With H < P (kv-head replication) `stage` names a rank and n = 1."""
    B, S, H, D = x_seq.shape
    n = H if stage is None else (1 if H < P else head_chunk)
    if out is None:
        out = torch.empty((B, n, S, D), dtype=x_seq.dtype, device=x_seq.device)
    _ck(lib().ulysses_seq2head(_p(x_seq), _p(out), S, B, H, D, P, head_chunk or 0,
                               _stage(stage), _dtype_code(x_seq), _stream(stream)))
    return out


def head2seq(x_head, x_seq, P, head_chunk=None, stage=None, stream=None):
    """All-to-all #2: write [B,n,S,D] into the stage's heads of [B,S,H,D]."""
    B, S, H, D = x_seq.shape
    if x_head.dtype != x_seq.dtype:
        raise TypeError("dtype mismatch")
    _ck(lib().ulysses_head2seq(_p(x_head), _p(x_seq), S, B, H, D, P, head_chunk or 0,
                               _stage(stage), _dtype_code(x_seq), _stream(stream)))
    return x_seq


def head2seq_add(x_head, x_seq, P, head_chunk=None, stage=None, stream=None):
    """As head2seq, adding into the fp32 sequence tensor (partial gradients of a
    replicated kv head)."""
    B, S, H, D = x_seq.shape
    if x_head.dtype != x_seq.dtype:
        raise TypeError("dtype mismatch")
    _ck(lib().ulysses_head2seq_add(_p(x_head), _p(x_seq), S, B, H, D, P, head_chunk or 0,
                                   _stage(stage), _dtype_code(x_seq), _stream(stream)))
    return x_seq


def _relayout_n(fn, pairs, P, stream, head_seq_index):
    """pairs: (src, dst, head_chunk, stage[, add]) per tensor; the sequence-
    layout tensor of each pair gives S, B, H, D (head_seq_index picks it)."""
    if not pairs:
        return
    items = (RelayoutItem * len(pairs))()
    seq0 = pairs[0][head_seq_index]
    B, S, _, D = seq0.shape
    dt = _dtype_code(seq0)
    for i, pr in enumerate(pairs):
        src, dst, C, stage = pr[:4]
        add = pr[4] if len(pr) > 4 else 0
        seq = pr[head_seq_index]
        if _dtype_code(src) != dt or _dtype_code(dst) != dt:
            raise TypeError("every tensor of a batched re-layout has the same dtype")
        items[i] = RelayoutItem(_p(src).value, _p(dst).value, seq.shape[2], C or 0, _stage(stage), int(add))
    _ck(fn(items, len(pairs), S, B, D, P, dt, _stream(stream)))


def seq2head_n(pairs, P, stream=None):
    """Batched all-to-all #1, one launch: pairs of (x_seq [B,S,H,D], x_head
    [B,n,S,D] out, head_chunk, stage) sharing S, B, D and dtype."""
    _relayout_n(lib().ulysses_seq2head_n, pairs, P, stream, 0)


def head2seq_n(pairs, P, stream=None):
    """Batched all-to-all #2, one launch: (x_head, x_seq, head_chunk, stage[,
    add]) per tensor; add (fp32 only) accumulates into x_seq."""
    _relayout_n(lib().ulysses_head2seq_n, pairs, P, stream, 1)


def padded_length(S, P):
    """S rounded up to a multiple of P."""
    return (S + P - 1) // P * P


def pad_to_multiple(tensors, P, cu_seqlens=None, stream=None):
    """Pad [B,S,H,D] device tensors along S to a multiple of P (as
    pad_to_multiple_of does for sequence parallelism) with the library's pad
    kernels.  Returns (padded tensors, cu_seqlens, S): the padding positions
    form a document of their own, so no real position attends to them or is
    attended by them (S stays the caller's length for slicing the results
    back).  cu_seqlens (int32, device) describes the real documents, or None
    for one document; it is needed with B == 1 only."""
    S = tensors[0].shape[1]
    S_pad = padded_length(S, P)
    if S_pad == S:
        return list(tensors), cu_seqlens, S
    out = []
    for t in tensors:
        B, _, H, D = t.shape
        p = torch.empty((B, S_pad, H, D), dtype=t.dtype, device=t.device)
        _ck(lib().ulysses_pad_seq(_p(t), _p(p), S, S_pad, B, H, D, _dtype_code(t), _stream(stream)))
        out.append(p)
    nd = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    cu = torch.empty(nd + 2, dtype=torch.int32, device=tensors[0].device)
    cp, _ = _cu(cu_seqlens)
    _ck(lib().ulysses_pad_cu_seqlens(cp, nd, _p(cu), S, S_pad, _stream(stream)))
    return out, cu, S


# --------------------------------------------------------------- attention

def attn_fwd(q_h, k_h, v_h, H_q, H_kv, P, head_chunk=None, stage=None, cu_seqlens=None,
             causal=True, scale=None, out=None, lse=None, stream=None):
    """Local attention on head-layout buffers: returns (O [B,n,S,D], LSE [B,n,S])."""
    B, n, S, D = q_h.shape
    if out is None:
        out = torch.empty_like(q_h)
    if lse is None:
        lse = torch.empty((B, n, S), dtype=torch.float32, device=q_h.device)
    cp, nd = _cu(cu_seqlens)
    _ck(lib().ulysses_attn_fwd(_p(q_h), _p(k_h), _p(v_h), _p(out), _p(lse), S, B, H_q, H_kv, D, P,
                               head_chunk or 0, _stage(stage), cp, nd, int(bool(causal)),
                               float(scale or 0.0), _dtype_code(q_h), _stream(stream)))
    return out, lse


def attn_bwd_workspace_bytes(S, B, H_q, H_kv, D, P, head_chunk=None, stage=None, dtype=BF16):
    return lib().ulysses_attn_bwd_workspace(S, B, H_q, H_kv, D, P, head_chunk or 0,
                                            _stage(stage), dtype)


def attn_bwd(q_h, k_h, v_h, o_h, do_h, lse, H_q, H_kv, P, head_chunk=None, stage=None,
             cu_seqlens=None, causal=True, scale=None, workspace=None, dq=None, dk=None, dv=None,
             stream=None):
    """Backward on head-layout buffers: returns fp32 (dQ, dK, dV)."""
    B, n, S, D = q_h.shape
    dev = q_h.device
    dq = torch.empty(q_h.shape, dtype=torch.float32, device=dev) if dq is None else dq
    dk = torch.empty(k_h.shape, dtype=torch.float32, device=dev) if dk is None else dk
    dv = torch.empty(v_h.shape, dtype=torch.float32, device=dev) if dv is None else dv
    ws_b = attn_bwd_workspace_bytes(S, B, H_q, H_kv, D, P, head_chunk, stage, _dtype_code(q_h))
    if workspace is None:
        workspace = torch.empty(max(ws_b, 256), dtype=torch.uint8, device=dev)
    cp, nd = _cu(cu_seqlens)
    _ck(lib().ulysses_attn_bwd(_p(q_h), _p(k_h), _p(v_h), _p(o_h), _p(do_h), _p(lse), _p(dq),
                               _p(dk), _p(dv), _p(workspace), workspace.numel(), S, B, H_q, H_kv,
                               D, P, head_chunk or 0, _stage(stage), cp, nd, int(bool(causal)),
                               float(scale or 0.0), _dtype_code(q_h), _stream(stream)))
    return dq, dk, dv


def attn_bwd_noalloc(q_h, k_h, v_h, o_h, do_h, lse, H_q, H_kv, P, head_chunk=None, stage=None,
                     cu_seqlens=None, causal=True, scale=None, dq=None, dk=None, dv=None,
                     stream=None):
    """attn_bwd through the entry point that needs no workspace (the library's
    built-in scratch holds D_i; see include/ulysses.h for its limit and the
    rule that calls sharing it must not overlap on the GPU)."""
    B, n, S, D = q_h.shape
    dev = q_h.device
    dq = torch.empty(q_h.shape, dtype=torch.float32, device=dev) if dq is None else dq
    dk = torch.empty(k_h.shape, dtype=torch.float32, device=dev) if dk is None else dk
    dv = torch.empty(v_h.shape, dtype=torch.float32, device=dev) if dv is None else dv
    cp, nd = _cu(cu_seqlens)
    _ck(lib().ulysses_attn_bwd_noalloc(_p(q_h), _p(k_h), _p(v_h), _p(o_h), _p(do_h), _p(lse),
                                       _p(dq), _p(dk), _p(dv), S, B, H_q, H_kv, D, P,
                                       head_chunk or 0, _stage(stage), cp, nd, int(bool(causal)),
                                       float(scale or 0.0), _dtype_code(q_h), _stream(stream)))
    return dq, dk, dv


# --------------------------------------------------------------- whole layer

def layer_workspace_bytes(S, B, H_q, H_kv, D, P, head_chunk, dtype=BF16):
    return lib().ulysses_layer_workspace(S, B, H_q, H_kv, D, P, head_chunk, dtype)


def layer_workspace(S, B, H_q, H_kv, D, P, head_chunk, dtype=BF16, device="cuda"):
    n = layer_workspace_bytes(S, B, H_q, H_kv, D, P, head_chunk, dtype)
    if n == 0:
        raise UlyssesError(ERR_INVALID, "invalid layer shape")
    return torch.empty(n, dtype=torch.uint8, device=device)


def layer_fwd(q_seq, k_seq, v_seq, P, head_chunk, cu_seqlens=None, causal=True, scale=None,
              workspace=None, out=None, lse=None, stream=None):
    """Steps 3-5 with the UPipe stage loop: returns (O [B,S,H_q,D], LSE [B,H_q,S])."""
    B, S, H_q, D = q_seq.shape
    H_kv = k_seq.shape[2]
    dt = _dtype_code(q_seq)
    if workspace is None:
        workspace = layer_workspace(S, B, H_q, H_kv, D, P, head_chunk, dt, q_seq.device)
    out = torch.empty_like(q_seq) if out is None else out
    lse = torch.empty((B, H_q, S), dtype=torch.float32, device=q_seq.device) if lse is None else lse
    cp, nd = _cu(cu_seqlens)
    _ck(lib().ulysses_layer_fwd(_p(q_seq), _p(k_seq), _p(v_seq), _p(out), _p(lse), S, B, H_q, H_kv,
                                D, P, head_chunk, cp, nd, int(bool(causal)), float(scale or 0.0),
                                dt, _p(workspace), workspace.numel(), _stream(stream)))
    return out, lse


def layer_bwd(q_seq, k_seq, v_seq, o_seq, do_seq, lse, P, head_chunk, cu_seqlens=None,
              causal=True, scale=None, workspace=None, dq=None, dk=None, dv=None, stream=None):
    """Backward of the layer: returns fp32 (dQ, dK, dV) in sequence layout."""
    B, S, H_q, D = q_seq.shape
    H_kv = k_seq.shape[2]
    dt = _dtype_code(q_seq)
    dev = q_seq.device
    if workspace is None:
        workspace = layer_workspace(S, B, H_q, H_kv, D, P, head_chunk, dt, dev)
    dq = torch.empty(q_seq.shape, dtype=torch.float32, device=dev) if dq is None else dq
    dk = torch.empty(k_seq.shape, dtype=torch.float32, device=dev) if dk is None else dk
    dv = torch.empty(v_seq.shape, dtype=torch.float32, device=dev) if dv is None else dv
    cp, nd = _cu(cu_seqlens)
    _ck(lib().ulysses_layer_bwd(_p(q_seq), _p(k_seq), _p(v_seq), _p(o_seq), _p(do_seq), _p(lse),
                                _p(dq), _p(dk), _p(dv), S, B, H_q, H_kv, D, P, head_chunk, cp, nd,
                                int(bool(causal)), float(scale or 0.0), dt, _p(workspace),
                                workspace.numel(), _stream(stream)))
    return dq, dk, dv


# --------------------------------------------------------------- diagnostics

def check(stream=None):
    """Synchronise and raise if a kernel flagged a timeout or bad cu_seqlens."""
    _ck(lib().ulysses_check(_stream(stream)))


def set_kernel(which: int):
    _ck(lib().ulysses_set_kernel(which))


def launch_count() -> int:
    return int(lib().ulysses_launch_count())


def selftest_wait_timeout(limit_ns=50_000_000, stream=None):
    """Launch the bounded-wait self-test (a wait nothing completes); the next
    check() raises UlyssesError with code ERR_TIMEOUT."""
    _ck(lib().ulysses_selftest_wait_timeout(int(limit_ns), _stream(stream)))


# --------------------------------------------------------------- ring variant

def ring_workspace(S, H_q, H_kv, D, P, dtype=BF16, device="cuda"):
    n = lib().ulysses_ring_workspace(S, H_q, H_kv, D, P, dtype)
    if n == 0:
        raise UlyssesError(ERR_INVALID, "invalid ring shape")
    return torch.empty(n, dtype=torch.uint8, device=device)


def ring_attention_fwd(q_seq, k_seq, v_seq, P, causal=True, scale=None, workspace=None, stream=None):
    """Ring-attention variant of the same layer (the scheme the pages compare
    Ulysses with), on P virtual ranks, run by the library's ring driver: rank
    r keeps query chunk r and meets KV chunk (r - t) mod P at ring step t;
    steps wholly in the future are skipped under the causal mask, the
    diagonal step is causal and the others are full; the steps' (O, LSE) are
    merged with their log-sum-exp weights.  Returns (O [1,S,H_q,D], LSE
    chunks [P,H_q,L])."""
    B, S, Hq, D = q_seq.shape
    Hkv = k_seq.shape[2]
    if B != 1 or S % P:
        raise ValueError("ring variant: B == 1 and S divisible by P")
    dt = _dtype_code(q_seq)
    if workspace is None:
        workspace = ring_workspace(S, Hq, Hkv, D, P, dt, q_seq.device)
    out = torch.empty_like(q_seq)
    lse = torch.empty((P, Hq, S // P), dtype=torch.float32, device=q_seq.device)
    _ck(lib().ulysses_ring_fwd(_p(q_seq), _p(k_seq), _p(v_seq), _p(out), _p(lse), S, Hq, Hkv, D, P,
                               int(bool(causal)), float(scale or 0.0), dt, _p(workspace), workspace.numel(),
                               _stream(stream)))
    return out, lse


def ring_attention_bwd(q_seq, k_seq, v_seq, o_seq, do_seq, lse, P, causal=True, scale=None, workspace=None,
                       stream=None):
    """Backward of ring_attention_fwd (library ring driver): every (query
    chunk, KV chunk) step runs the attention backward with the merged LSE and
    O, and the steps' partial dQ, dK, dV are summed.  Returns fp32 (dQ, dK,
    dV) in sequence layout."""
    B, S, Hq, D = q_seq.shape
    Hkv = k_seq.shape[2]
    if B != 1 or S % P:
        raise ValueError("ring variant: B == 1 and S divisible by P")
    dt = _dtype_code(q_seq)
    dev = q_seq.device
    if workspace is None:
        workspace = ring_workspace(S, Hq, Hkv, D, P, dt, dev)
    dq = torch.empty(q_seq.shape, dtype=torch.float32, device=dev)
    dk = torch.empty(k_seq.shape, dtype=torch.float32, device=dev)
    dv = torch.empty(v_seq.shape, dtype=torch.float32, device=dev)
    _ck(lib().ulysses_ring_bwd(_p(q_seq), _p(k_seq), _p(v_seq), _p(o_seq), _p(do_seq), _p(lse), _p(dq), _p(dk),
                               _p(dv), S, Hq, Hkv, D, P, int(bool(causal)), float(scale or 0.0), dt,
                               _p(workspace), workspace.numel(), _stream(stream)))
    return dq, dk, dv


# --------------------------------------------------------------- projections

def qkv_proj(x, w_qkv, H_q, H_kv, out=None, stream=None):
    """[Q|K|V] = X W_qkv^T written straight into head layout: x [S,hidden]
    bf16, w_qkv [(H_q+2H_kv) D, hidden] bf16 -> [H_q+2H_kv, S, D] bf16."""
    S, hidden = x.shape
    nf = w_qkv.shape[0]
    D = nf // (H_q + 2 * H_kv)
    if out is None:
        out = torch.empty((H_q + 2 * H_kv, S, D), dtype=torch.bfloat16, device=x.device)
    _ck(lib().ulysses_qkv_proj(_p(x), _p(w_qkv), _p(out), S, hidden, H_q, H_kv, D, _stream(stream)))
    return out


def out_proj(o_head, w_o, out=None, stream=None):
    """Y = O W_o^T with O read from head layout: o_head [H_q, S, D] bf16,
    w_o [hidden, H_q D] bf16 -> [S, hidden] bf16."""
    H_q, S, D = o_head.shape
    hidden = w_o.shape[0]
    if out is None:
        out = torch.empty((S, hidden), dtype=torch.bfloat16, device=o_head.device)
    _ck(lib().ulysses_out_proj(_p(o_head), _p(w_o), _p(out), S, H_q, D, hidden, _stream(stream)))
    return out


# --------------------------------------------------------------- fused layer

def layer_fwd_fused(q_seq, k_seq, v_seq, P, head_chunk, cu_seqlens=None, causal=True, scale=None,
                    out=None, lse=None, stream=None):
    """layer_fwd with the all-to-alls folded into the kernels' addressing (no
    head-layout copies): returns (O [1,S,H_q,D], LSE [1,H_q,S])."""
    B, S, H_q, D = q_seq.shape
    H_kv = k_seq.shape[2]
    out = torch.empty_like(q_seq) if out is None else out
    lse = torch.empty((B, H_q, S), dtype=torch.float32, device=q_seq.device) if lse is None else lse
    cp, nd = _cu(cu_seqlens)
    _ck(lib().ulysses_layer_fwd_fused(_p(q_seq), _p(k_seq), _p(v_seq), _p(out), _p(lse), S, B, H_q, H_kv, D, P,
                                      head_chunk, cp, nd, int(bool(causal)), float(scale or 0.0),
                                      _dtype_code(q_seq), _stream(stream)))
    return out, lse


def layer_bwd_fused(q_seq, k_seq, v_seq, o_seq, do_seq, lse, P, head_chunk, cu_seqlens=None, causal=True,
                    scale=None, workspace=None, dq=None, dk=None, dv=None, stream=None):
    """layer_bwd with the all-to-alls folded into the kernels' addressing:
    returns fp32 (dQ, dK, dV) in sequence layout."""
    B, S, H_q, D = q_seq.shape
    H_kv = k_seq.shape[2]
    dt = _dtype_code(q_seq)
    dev = q_seq.device
    if workspace is None:
        nb = lib().ulysses_layer_fused_workspace(S, B, H_q, H_kv, D, P, head_chunk, dt)
        workspace = torch.empty(max(nb, 256), dtype=torch.uint8, device=dev)
    dq = torch.empty(q_seq.shape, dtype=torch.float32, device=dev) if dq is None else dq
    dk = torch.empty(k_seq.shape, dtype=torch.float32, device=dev) if dk is None else dk
    dv = torch.empty(v_seq.shape, dtype=torch.float32, device=dev) if dv is None else dv
    cp, nd = _cu(cu_seqlens)
    _ck(lib().ulysses_layer_bwd_fused(_p(q_seq), _p(k_seq), _p(v_seq), _p(o_seq), _p(do_seq), _p(lse), _p(dq),
                                      _p(dk), _p(dv), S, B, H_q, H_kv, D, P, head_chunk, cp, nd,
                                      int(bool(causal)), float(scale or 0.0), dt, _p(workspace),
                                      workspace.numel(), _stream(stream)))
    return dq, dk, dv


# --------------------------------------------------------------- strided calls
# The calls below take tensors by their strides: sequence layout, head layout
# and slices of a fused projection's result alike ("seq": tokens, heads, D;
# "head": heads, tokens, D; D contiguous).  They run on the device of their
# tensors, whichever is current, on `stream` or that device's current stream;
# outputs and workspaces made here belong to that stream.
# A call's kernels take a few microseconds at decode sizes.  Plain calls (no
# stream given, everything as it should be) are marshalled by _fastcall-*.so; the
# Python below serves the others and says what is wrong with a call.  It reads
# each tensor property once and makes no objects besides the results.

_CODES = {torch.bfloat16: BF16, torch.float32: FP32, torch.float8_e4m3fn: E4M3}
_BF16, _F32, _F64, _I32, _U8, _F8 = (torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8,
                                     torch.float8_e4m3fn)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda idx: torch.cuda.current_stream(idx).cuda_stream)


def _code(dtype, what):
    c = _CODES.get(dtype)
    if c is None:
        raise TypeError(f"{what}: unsupported dtype {dtype}")
    return c


def _device_of(tensors):
    """Index of the one CUDA device of the tensors (None entries left out)."""
    idx = -2
    for t in tensors:
        if t is not None:
            i = t.get_device()
            if i != idx:
                if i < 0:
                    raise ValueError("expected a CUDA tensor")
                if idx >= 0:
                    raise ValueError(f"tensors on different devices: cuda:{idx} and cuda:{i}")
                idx = i
    return idx


def _flat(t, dtype, what):
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _rows(t, layout, what):
    """(token stride, head stride, tokens, heads, D) of a tensor of rows, its
    last three dimensions."""
    sh, st = t.shape, t.stride()
    if len(sh) < 3:
        raise ValueError(f"{what} must have three dimensions")
    if st[-1] != 1 and t.numel():
        raise ValueError(f"{what}: the last dimension must be contiguous")
    if layout == "seq":
        return st[-3], st[-2], sh[-3], sh[-2], sh[-1]
    if layout == "head":
        return st[-2], st[-3], sh[-2], sh[-3], sh[-1]
    raise ValueError(f"unknown layout {layout!r}")


def _rows3(t, layout, what):
    sh, st = t.shape, t.stride()
    if len(sh) != 3:
        raise ValueError(f"{what} must have three dimensions")
    if st[2] != 1 and t.numel():
        raise ValueError(f"{what}: the last dimension must be contiguous")
    if layout == "head":
        return st[1], st[0], sh[1], sh[0], sh[2]
    if layout == "seq":
        return st[0], st[1], sh[0], sh[1], sh[2]
    raise ValueError(f"unknown layout {layout!r}")


def _launch(fn, idx, stream, tensors, args):
    """fn(*args, stream) on device idx.  A stream given by the caller is
    recorded on the tensors, so that freeing one of them does not hand its
    memory on while the call still runs."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    if idx == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(idx) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(idx):
            rc = fn(*args, _raw_stream(idx) if stream is None else stream.cuda_stream)
    if rc != OK:
        _ck(rc)


def _empty(like, shape, dtype, stream):
    # empty_strided: the shortest way through torch's dispatcher (a microsecond less than empty)
    n = len(shape)
    strides = (shape[1] * shape[2], shape[2], 1) if n == 3 else (1,) if n == 1 else (shape[1], 1) if n == 2 else \
        (shape[1] * shape[2] * shape[3], shape[2] * shape[3], shape[3], 1)
    if stream is None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty_strided(shape, strides, dtype=dtype, device=like.device)


# --------------------------------------------------------------- rotary positions

def rope_frequencies(rot_dim, base=10000.0, sections=None):
    """Host tensors (inv_freq [rot_dim/2] float64, axes [rot_dim/2] int32) for
    rope_fwd / rope_bwd: inv_freq[i] = base^(-2i/rot_dim).  sections gives, for
    positions of several axes (time, height, width), how many of the pairs turn
    by each axis, in order; None is one axis."""
    half = rot_dim // 2
    inv = torch.tensor([float(base) ** (-i / half) for i in range(half)], dtype=torch.float64)
    sections = [half] if sections is None else list(sections)
    if sum(sections) != half:
        raise ValueError(f"sections {sections} must add up to rot_dim/2 = {half}")
    return inv, torch.tensor([a for a, n in enumerate(sections) for _ in range(n)], dtype=torch.int32)


_PACK_ITEM = struct.Struct("@PPi6q").pack     # ulysses_rope_item
_PAIRS = {"half": PAIRS_HALF, "adjacent": PAIRS_ADJACENT}


def _rope(fn, q, k, positions, inv_freq, axes, layout, pairs, dtype, out, stream):
    given = (q,) if k is None else (k,) if q is None else (q, k)
    first = given[0]
    if first is None:
        raise ValueError("rope: no tensor given")
    if out is not None:
        out = tuple(out) if isinstance(out, (tuple, list)) else (out,)
        if len(out) != len(given):
            raise ValueError("rope: one output for each tensor")
    idx = _device_of((*given, positions) if out is None else (*given, positions, *out))
    din = first.dtype
    dout = din if dtype is None else dtype
    code_in, code_out = _code(din, "rope"), _code(dout, "rope")
    head = layout == "head"
    if not head and layout != "seq":
        raise ValueError(f"unknown layout {layout!r}")
    items, results, tokens = b"", [], None
    for i, t in enumerate(given):
        sh, st = t.shape, t.stride()
        if len(sh) == 3:
            B, sb = 1, 0
            n, H, D = sh if not head else (sh[1], sh[0], sh[2])
            ss, sn, sd = st if not head else (st[1], st[0], st[2])
        elif len(sh) == 4:
            B, n, H, D = sh if not head else (sh[0], sh[2], sh[1], sh[3])
            sb, ss, sn, sd = st if not head else (st[0], st[2], st[1], st[3])
        else:
            raise ValueError("rope: tensors have three or four dimensions")
        if sd != 1 and t.numel():
            raise ValueError("rope input: the last dimension must be contiguous")
        if tokens is None:
            tokens = (len(sh), B, n, D)
        elif tokens != (len(sh), B, n, D) or t.dtype is not din:
            raise ValueError("rope: tensors of one call share their tokens, D and dtype")
        if out is None:
            o = _empty(t, sh, dout, stream)
            os_, on = (D, n * D) if head else (H * D, D)
            ob = n * H * D
        else:
            o = out[i]
            if o.shape != sh or o.dtype is not dout:
                raise ValueError("rope: an output must have its input's shape and the call's dtype")
            os_, on, _, _, _ = _rows(o, layout, "rope output")
            ob = o.stride(0) if len(sh) == 4 else 0
        items += _PACK_ITEM(t.data_ptr(), o.data_ptr(), H, sb, ss, sn, ob, os_, on)
        results.append(o)
    dims, B, S, D = tokens
    psh = positions.shape
    n_axes, psh = (1, psh) if len(psh) == dims - 2 else (psh[0], psh[1:])
    if psh != ((S,) if dims == 3 else (B, S)):
        raise ValueError(f"rope: positions {tuple(positions.shape)} do not match {B} x {S} tokens")
    half = inv_freq.numel()
    if inv_freq.dtype is not _F64 or inv_freq.is_cuda or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 tensor in host memory")
    ax = None
    if axes is not None:
        if axes.dtype is not _I32 or axes.is_cuda or not axes.is_contiguous() or axes.numel() != half:
            raise ValueError("axes must be a contiguous int32 tensor in host memory, one entry for each frequency")
        ax = axes.data_ptr()
    if pairs not in _PAIRS:
        raise ValueError(f"unknown pair order {pairs!r}")
    _launch(fn, idx, stream, (*given, positions, *results),
            (items, len(given), _flat(positions, _I32, "positions"), n_axes, inv_freq.data_ptr(), ax, 2 * half,
             _PAIRS[pairs], S, B, D, code_in, code_out))
    return results[0] if k is None or q is None else (results[0], results[1])


def rope_fwd(q, k, positions, inv_freq, axes=None, layout="seq", pairs="half", out=None, stream=None):
    """Rotary positions on Q and K (either may be None), one launch.

    q, k: [T, H, D] or [B, S, H, D] in sequence layout ("seq"), [H, T, D] or
    [B, n, S, D] in head layout ("head"); bf16 or fp32, any strides with D
    contiguous.  positions: int32 [T] ([B, S]), or [n_axes, ...] with axes
    naming the axis of every pair; inv_freq, axes: host tensors
    (rope_frequencies).  The first 2 * len(inv_freq) features of a head turn:
    pairs (i, i + half) with "half", (2i, 2i+1) with "adjacent"; the others are
    copied.  out: the outputs, q and k themselves for in place.  Returns the
    rotated tensors, in the order given."""
    if _fast is not None and stream is None:
        r = _fast.rope(False, q, k, positions, inv_freq, axes, layout, pairs, None, out)
        if r is not None:
            return r if type(r) is not int else _ck(r)
    return _rope(lib().ulysses_rope_fwd, q, k, positions, inv_freq, axes, layout, pairs, None, out, stream)


def rope_bwd(dq, dk, positions, inv_freq, axes=None, layout="seq", pairs="half", dtype=None, out=None, stream=None):
    """Adjoint of rope_fwd: gradients of the rotated Q and K (as layer_bwd
    gives them, fp32 or bf16) to those of the projection's Q and K.  dtype: the
    outputs' type (default: the gradients'; bf16 from fp32 rounds once)."""
    if _fast is not None and stream is None:
        r = _fast.rope(True, dq, dk, positions, inv_freq, axes, layout, pairs, dtype, out)
        if r is not None:
            return r if type(r) is not int else _ck(r)
    return _rope(lib().ulysses_rope_bwd, dq, dk, positions, inv_freq, axes, layout, pairs, dtype, out, stream)


# --------------------------------------------------------------- paged key-value cache

def kv_cache(num_pages, page_size, H_kv, D, dtype=torch.bfloat16, device="cuda"):
    """Buffers of a paged cache: (k_cache, v_cache [num_pages, H_kv, page_size,
    D], k_scale, v_scale [num_pages, H_kv, page_size] fp32, or None unless
    dtype is torch.float8_e4m3fn or torch.uint8).  Zero-filled.  torch.uint8 is
    the 4-bit cache, [num_pages, H_kv, page_size, 9 D / 16] bytes: a page of a
    head holds its rows' e2m1 codes ([page_size, D / 2], two a byte, the first in
    the low half) and behind them their e4m3 scales of 16 codes each
    ([page_size, D / 16])."""
    four = dtype == torch.uint8
    shape = (num_pages, H_kv, page_size, D * 9 // 16 if four else D)
    k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
    if not four and dtype != torch.float8_e4m3fn:
        return k, v, None, None
    ks, vs = (torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2))
    return k, v, ks, vs


def cache_weights(k_cache):
    """Attention weights that the tokens of a cache have gathered: zeros
    [num_pages, H_kv, page_size] fp32, for cache_write, attn_decode and
    cache_evict."""
    return torch.zeros(k_cache.shape[:3], dtype=torch.float32, device=k_cache.device)


def _cache(k_cache, v_cache, k_scale, v_scale):
    """Pointers of the cache's buffers, its sizes and its type's code, after the
    checks that need the tensors."""
    sh, dt = k_cache.shape, k_cache.dtype
    if len(sh) != 4 or sh != v_cache.shape or dt is not v_cache.dtype:
        raise ValueError("k_cache and v_cache must be [num_pages, H_kv, page_size, D] of one shape and dtype")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("k_cache and v_cache must be contiguous")
    if dt is _U8:
        code = E2M1
        if sh[3] % 9:
            raise ValueError("a 4-bit cache (uint8) must have 9 D / 16 bytes a row")
        sh = (*sh[:3], sh[3] // 9 * 16)
    else:
        code = _code(dt, "k_cache")
    ks = vs = None
    if k_scale is not None:
        if k_scale.shape != sh[:3]:
            raise ValueError("scales must be [num_pages, H_kv, page_size]")
        ks = _flat(k_scale, _F32, "k_scale")
    if v_scale is not None:
        if v_scale.shape != sh[:3]:
            raise ValueError("scales must be [num_pages, H_kv, page_size]")
        vs = _flat(v_scale, _F32, "v_scale")
    return k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, sh, code


def _weights(weights, sh):
    if weights.shape != sh[:3]:
        raise ValueError("weights must be [num_pages, H_kv, page_size]")
    return _flat(weights, _F32, "weights")


def _batch_table(page_table, n, what):
    sh = page_table.shape
    if len(sh) != 2 or sh[0] != n:
        raise ValueError(f"page_table must be [B, columns], B = {n} as {what}")
    return _flat(page_table, _I32, "page_table"), sh[1]


def cache_write(k, v, k_cache, v_cache, page_table, seq_lens, cu_new=None, k_scale=None, v_scale=None, layout="seq",
                stream=None, weights=None):
    """Store the K and V rows of new tokens in the paged cache.

    k, v: [T, H_kv, D] ("seq") or [H_kv, T, D] ("head"), any strides with D
    contiguous.  page_table int32 [B, columns], seq_lens int32 [B]: the lengths
    with the new tokens.  cu_new int32 [B + 1]: sequence b's new tokens are
    rows [cu_new[b], cu_new[b+1]); None: one token per sequence, and a length
    of 0 marks an empty place of the batch.  An e4m3 or 4-bit (uint8) cache, with
    its scales, is quantised row by row on the way.  weights (cache_weights()):
    those of the new tokens are set to 0.  Bad positions or pages raise in
    check()."""
    if _fast is not None and stream is None:
        r = _fast.cache_write(k, v, k_cache, v_cache, page_table, seq_lens, cu_new, k_scale, v_scale, layout, weights)
        if r is not None:
            return _ck(r)
    ks, kh, T, H, D = _rows3(k, layout, "k")
    vs, vh, Tv, Hv, Dv = _rows3(v, layout, "v")
    dt = k.dtype
    if T != Tv or H != Hv or D != Dv or dt is not v.dtype:
        raise ValueError("k and v must have one shape and dtype")
    tensors = (k, v, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, cu_new, weights)
    pk, pv, pks, pvs, sh, held = _cache(k_cache, v_cache, k_scale, v_scale)
    if H != sh[1] or D != sh[3]:
        raise ValueError("rows and cache differ in heads or D")
    idx = _device_of(tensors)
    B = seq_lens.numel()
    tab, cols = _batch_table(page_table, B, "seq_lens")
    cu = None
    if cu_new is not None:
        if cu_new.numel() != B + 1:
            raise ValueError("cu_new must have B + 1 entries")
        cu = _flat(cu_new, _I32, "cu_new")
    args = (k.data_ptr(), v.data_ptr(), ks, kh, vs, vh, T, B, cu, tab, cols, _flat(seq_lens, _I32, "seq_lens"), pk, pv, pks,
            pvs)
    sizes = (sh[0], sh[2], H, D, _code(dt, "k"), held)
    if weights is None:
        _launch(lib().ulysses_cache_write, idx, stream, tensors, (*args, *sizes))
    else:
        _launch(lib().ulysses_cache_write_weights, idx, stream, tensors, (*args, _weights(weights, sh), *sizes))


def cache_read(k_cache, v_cache, page_table, cu_seqlens, T, first=None, k_scale=None, v_scale=None, dtype=None,
               layout="seq", out=None, stream=None):
    """Gather cached rows back: token t of the packed outputs, in sequence b
    (cu_seqlens[b] <= t < cu_seqlens[b+1]), is position first[b] + t -
    cu_seqlens[b] (first None: 0).  Returns (k, v) with T tokens, [T, H_kv, D]
    or [H_kv, T, D]; rows from cu_seqlens[B] on are left as they were.  dtype:
    the cache's, or bf16 (default) / fp32 from an e4m3 or 4-bit cache."""
    if _fast is not None and stream is None:
        r = _fast.cache_read(k_cache, v_cache, page_table, cu_seqlens, T, first, k_scale, v_scale, dtype, layout, out)
        if r is not None:
            return r if type(r) is not int else _ck(r)
    pk, pv, pks, pvs, (n_pages, H, page, D), held = _cache(k_cache, v_cache, k_scale, v_scale)
    if dtype is None:
        dtype = out[0].dtype if out is not None else _BF16 if held in (E4M3, E2M1) else k_cache.dtype
    B = cu_seqlens.numel() - 1
    tab, cols = _batch_table(page_table, B, "cu_seqlens")
    at = None
    if first is not None:
        if first.numel() != B:
            raise ValueError("first must have B entries")
        at = _flat(first, _I32, "first")
    if layout != "seq" and layout != "head":
        raise ValueError(f"unknown layout {layout!r}")
    shape = (T, H, D) if layout == "seq" else (H, T, D)
    idx = _device_of((k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, first, *(out or ())))
    if out is None:
        k, v = _empty(k_cache, shape, dtype, stream), _empty(k_cache, shape, dtype, stream)
        ks, kh = vs, vh = (H * D, D) if layout == "seq" else (D, T * D)
    else:
        k, v = out
        if k.shape != shape or v.shape != shape or k.dtype is not dtype or v.dtype is not dtype:
            raise ValueError(f"cache_read: outputs must be {shape} of {dtype}")
        ks, kh, _, _, _ = _rows3(k, layout, "k")
        vs, vh, _, _, _ = _rows3(v, layout, "v")
    tensors = (k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, first)
    _launch(lib().ulysses_cache_read, idx, stream, tensors,
            (pk, pv, pks, pvs, tab, cols, _flat(cu_seqlens, _I32, "cu_seqlens"), at, k.data_ptr(), v.data_ptr(), ks, kh,
             vs, vh, T, B, n_pages, page, H, D, _code(dtype, "k"), held))
    return k, v


@functools.lru_cache(maxsize=256)
def _evict_bytes(*sizes):
    return lib().ulysses_cache_evict_workspace(*sizes)


def cache_evict_workspace(k_cache, page_table):
    """Workspace for cache_evict on tensors of these shapes (uint8, on their
    device)."""
    n = _evict_bytes(page_table.shape[0], k_cache.shape[1], page_table.shape[1], k_cache.shape[2])
    return torch.empty(n, dtype=torch.uint8, device=k_cache.device)


def cache_evict(k_cache, v_cache, weights, page_table, seq_lens, keep, recent=0, k_scale=None, v_scale=None, out=None,
                workspace=None, stream=None):
    """Take the tokens with the least attention weight out of the paged cache.

    Of a sequence's n = seq_lens[b] tokens min(n, keep[b]) stay (keep int32 [B];
    negative: all), for each kv head its own: the last `recent` of them for
    their age, and of those before the ones of greatest weight (the lower
    position first among equals, NaN above everything).  They close up in their
    order to positions 0, 1, ..., in place, with their scales and weights; the
    places behind are left as they were, and pages that hold none of them are
    the caller's again.  The sequences of a call must not share pages.  Returns
    the new lengths int32 [B] (out: into this tensor, which may be seq_lens or keep).
    workspace: cache_evict_workspace(), for calls that do not overlap on the
    GPU; made per call if not given.  A sequence with a bad length or page is
    left as it is, and raises in check()."""
    if _fast is not None and stream is None:
        r = _fast.cache_evict(k_cache, v_cache, weights, page_table, seq_lens, keep, recent, k_scale, v_scale, out, workspace)
        if r is not None:
            return r if type(r) is not int else _ck(r)
    pk, pv, pks, pvs, sh, held = _cache(k_cache, v_cache, k_scale, v_scale)
    n_pages, H, page, D = sh
    B = seq_lens.numel()
    idx = _device_of((k_cache, v_cache, weights, page_table, seq_lens, keep, k_scale, v_scale, out, workspace))
    pw = _weights(weights, sh)
    tab, cols = _batch_table(page_table, B, "seq_lens")
    if keep.numel() != B:
        raise ValueError("keep must have B entries")
    recent = max(min(recent, (1 << 31) - 1), -1)           # as many as there are; any number below 0 is refused
    if out is None:
        out = _empty(seq_lens, (B,), _I32, stream)
    elif out.numel() != B:
        raise ValueError("out must have B entries")
    if workspace is None:
        n = _evict_bytes(B, H, cols, page)
        if n:
            workspace = _empty(k_cache, (n,), _U8, stream)
    ws, n = (None, 0) if workspace is None else (_flat(workspace, _U8, "workspace"), workspace.numel())
    _launch(lib().ulysses_cache_evict, idx, stream,
            (k_cache, v_cache, weights, page_table, seq_lens, keep, k_scale, v_scale, out, workspace),
            (pk, pv, pks, pvs, pw, tab, cols, _flat(seq_lens, _I32, "seq_lens"), _flat(keep, _I32, "keep"), recent,
             _flat(out, _I32, "out"), B, n_pages, page, H, D, held, ws, n))
    return out


# --------------------------------------------------------------- single-token attention

@functools.lru_cache(maxsize=256)
def _decode_bytes(weights, *sizes):
    return (lib().ulysses_attn_decode_weights_workspace if weights else lib().ulysses_attn_decode_workspace)(*sizes)


def attn_decode_workspace(q, k_cache, page_table, layout="seq", weights=False):
    """Workspace for attn_decode on tensors of these shapes (uint8, on their
    device; empty where the call needs none).  weights: for calls with
    weights, which keep the scores of every position of the table there."""
    _, _, B, H_q, D = _rows3(q, layout, "q")
    n = _decode_bytes(bool(weights), B, H_q, k_cache.shape[1], D, page_table.shape[1], k_cache.shape[2], _code(q.dtype, "q"),
                      E2M1 if k_cache.dtype is _U8 else _code(k_cache.dtype, "k_cache"))
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def attn_decode(q, k_cache, v_cache, page_table, seq_lens, k_scale=None, v_scale=None, scale=None, layout="seq",
                workspace=None, out=None, lse=None, stream=None, weights=None):
    """Attention of one new token per sequence over the paged cache.

    q: [B, H_q, D] ("seq") or [H_q, B, D] ("head", as qkv_proj gives it), any
    strides with D contiguous; bf16 (bf16, e4m3 or 4-bit cache) or fp32 (fp32,
    e4m3 or 4-bit cache).  The keys of sequence b are its first seq_lens[b]
    (int32 [B]) cached positions; length 0 gives O = 0, LSE = -inf.  Returns (O
    shaped as q, LSE [B, H_q] fp32).  weights (cache_weights()): each key's
    attention weight, summed over the query heads of its kv head, is added to
    its slot's.  workspace: attn_decode_workspace(), for calls that do not
    overlap on the GPU; made per call if not given."""
    if _fast is not None and stream is None:
        r = _fast.attn_decode(q, k_cache, v_cache, page_table, seq_lens, k_scale, v_scale, scale, layout, workspace, out,
                              lse, weights)
        if r is not None:
            return r if type(r) is not int else _ck(r)
    qb, qh, B, H_q, D = _rows3(q, layout, "q")
    pk, pv, pks, pvs, sh, dc = _cache(k_cache, v_cache, k_scale, v_scale)
    n_pages, H_kv, page, Dc = sh
    if D != Dc or seq_lens.numel() != B:
        raise ValueError("attn_decode: q, cache and seq_lens differ in D or B")
    tensors = (q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, workspace, out, lse, weights)
    idx = _device_of(tensors)
    tab, cols = _batch_table(page_table, B, "q")
    dt = q.dtype
    dq = _code(dt, "q")
    if out is None:
        out = _empty(q, q.shape, dt, stream)
        ob, oh = (H_q * D, D) if layout == "seq" else (D, B * D)
    elif out.shape != q.shape or out.dtype is not dt:
        raise ValueError("attn_decode: out must have q's shape and dtype")
    else:
        ob, oh, _, _, _ = _rows3(out, layout, "out")
    if lse is None:
        lse = _empty(q, (B, H_q), _F32, stream)
        pl = lse.data_ptr()
    elif lse.shape != (B, H_q):
        raise ValueError("attn_decode: lse must be [B, H_q]")
    else:
        pl = _flat(lse, _F32, "lse")
    if workspace is None:
        n = _decode_bytes(weights is not None, B, H_q, H_kv, D, cols, page, dq, dc)
        if n:
            workspace = _empty(q, (n,), _U8, stream)
    ws, n = (None, 0) if workspace is None else (_flat(workspace, _U8, "workspace"), workspace.numel())
    args = (q.data_ptr(), qb, qh, pk, pv, pks, pvs, tab, cols, _flat(seq_lens, _I32, "seq_lens"), out.data_ptr(), ob, oh, pl)
    sizes = (B, H_q, H_kv, D, n_pages, page, scale or 0.0, dq, dc, ws, n)
    # again, for a given stream: with what was made here since their devices were looked at
    tensors = (q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, workspace, out, lse, weights)
    if weights is None:
        _launch(lib().ulysses_attn_decode, idx, stream, tensors, (*args, *sizes))
    else:
        _launch(lib().ulysses_attn_decode_weights, idx, stream, tensors, (*args, _weights(weights, sh), *sizes))
    return out, lse
