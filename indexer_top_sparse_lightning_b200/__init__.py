"""DSA sparse-attention step on B200: fused Lightning Indexer + Top-K and
Sparse Flash Attention over the MLA latent cache.

The computation runs in ``libdsa.so`` (hand-written sm_100a CUDA kernels behind
the C ABI of ``include/dsa.h``).  This module only marshals torch tensors into
that ABI: it checks dtypes and shapes, allocates outputs with torch, and
passes raw device pointers plus the current CUDA stream.  There is no
fallback: if the library is missing, importing the entry points raises.

Entry points (same names as the C ABI):
    indexer_topk(batch, q_idx, w, k_cache, K, k_scale=None, q_scale=None) -> (idx, score)
    sparse_mla_attn(batch, q, kv_cache, idx, sm_scale, kv_scale=None) -> (out, lse)
    dsa_decode(batch, q_idx, w, k_cache, q, kv_cache, K, sm_scale, k_scale=None, q_scale=None)
        -> (idx, score, out, lse)

    indexer_prolog(batch, x, w_proj, k_gamma, eps, k_cache, k_scale=None, mx=False)
        -> (q_idx, q_scale or None, w)   (also writes the tokens' keys into k_cache / k_scale;
        w_proj row-major, or prolog_pack_weights(w_proj, H_I, D_I) for weight streaming)
    dsa_qk_norm_rope(batch, inv_freq, q, k, q_gamma=None, k_gamma=None, k_cache=None, ...) -> q_out
        (per-head norm and rotation of queries and keys; keys go into the paged cache)
    dsa_chunk_attn(batch, q, kv_cache, sm_scale, kv_scale=None) -> (out, lse)
        (dense causal attention of the new tokens over the paged latent cache)
    dsa_attn_weight(batch, q, kv_cache, sm_scale, lse, weight, decay=1.0, kv_scale=None) -> weight
        (the attention weight that each cached position draws, accumulated)
    dsa_cache_evict(batch, weight, keep, new_table, arrays, new_arrays, sink=0, recent=0, new_weight=None) -> (idx, len)
        (keeps the positions with the most weight; their rows move to new pages)

Key formats: bf16 keys (k_scale None); e4m3 keys (uint8) with fp32 k_scale
[nblk, 64, D_I/64]; MXFP8 queries and keys when q_scale is given: q_idx and
k_cache hold e4m3 codes (uint8), q_scale [T, H_I, D_I/32] and k_scale
[nblk, 64, D_I/32] hold uint8 exponents (one power-of-two scale per 32 elements).
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from dataclasses import dataclass
from typing import Optional

import torch

__all__ = ["Batch", "Workspace", "indexer_topk", "sparse_mla_attn", "dsa_decode", "indexer_prolog",
           "prolog_pack_weights", "PackedWeights", "dsa_qk_norm_rope", "dsa_chunk_attn", "dsa_attn_weight", "dsa_cache_evict", "get_status", "status_workspace",
           "DsaError", "library_path", "load_library"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libdsa.so")
_lib = None

KEY_BF16 = 0
KEY_FP8_E4M3 = 1
KEY_MXFP8 = 2
Q_BF16 = 0
Q_MXFP8 = 1
KV_BF16 = 0
KV_FP8 = 1


DSA_ERR_CUDA = 4   # dsa_status code of a failed CUDA runtime / driver call


class DsaError(RuntimeError):
    def __init__(self, code: int, where: str, detail: str = ""):
        self.code = int(code)
        if not detail and self.code == DSA_ERR_CUDA:
            detail = last_error()
        super().__init__(f"{where}: {status_str(code)} (code {code})" + (f": {detail}" if detail else ""))


class _Batch(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_tokens", ctypes.c_int32),
                ("seq_lens", ctypes.c_void_p), ("cu_q", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("max_blocks_per_seq", ctypes.c_int32),
                ("num_blocks", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
                ("max_q_per_seq", ctypes.c_int32)]


class _Indexer(ctypes.Structure):
    _fields_ = [("q_idx", ctypes.c_void_p), ("w", ctypes.c_void_p), ("k_cache", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("key_dtype", ctypes.c_int32), ("H_I", ctypes.c_int32),
                ("D_I", ctypes.c_int32), ("K", ctypes.c_int32), ("q_dtype", ctypes.c_int32),
                ("q_scale", ctypes.c_void_p)]


class _Attn(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("kv_cache", ctypes.c_void_p), ("H", ctypes.c_int32),
                ("sm_scale", ctypes.c_float), ("kv_dtype", ctypes.c_int32), ("kv_scale", ctypes.c_void_p)]


class _Prolog(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("w_proj", ctypes.c_void_p), ("k_gamma", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("d_model", ctypes.c_int32), ("H_I", ctypes.c_int32),
                ("D_I", ctypes.c_int32), ("key_dtype", ctypes.c_int32), ("q_dtype", ctypes.c_int32),
                ("w_layout", ctypes.c_int32)]


class _Rope(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_stride_t", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("k_stride_t", ctypes.c_int64), ("H", ctypes.c_int32),
                ("D", ctypes.c_int32), ("q_gamma", ctypes.c_void_p), ("k_gamma", ctypes.c_void_p),
                ("q_norm", ctypes.c_int32), ("k_norm", ctypes.c_int32), ("eps", ctypes.c_float),
                ("inv_freq", ctypes.c_void_p), ("rope_dim", ctypes.c_int32), ("rope_off", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("positions", ctypes.c_void_p), ("kv_dtype", ctypes.c_int32)]


class _CacheArray(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("row_bytes", ctypes.c_int64)]


class _Evict(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("weight_stride", ctypes.c_int64), ("new_weight", ctypes.c_void_p),
                ("new_weight_stride", ctypes.c_int64), ("keep", ctypes.c_int32), ("sink", ctypes.c_int32),
                ("recent", ctypes.c_int32), ("new_table", ctypes.c_void_p), ("new_max_blocks", ctypes.c_int32),
                ("new_num_blocks", ctypes.c_int32), ("arrays", ctypes.POINTER(_CacheArray)),
                ("n_arrays", ctypes.c_int32)]


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libdsa.so (built in-tree by ``python -m indexer_top_sparse_lightning_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with "
                          "`python -m indexer_top_sparse_lightning_b200.build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(_LIB_PATH)
    P = ctypes.POINTER
    lib.dsa_workspace_size.argtypes = [P(_Batch), P(_Indexer), P(_Attn)]
    lib.dsa_workspace_size.restype = ctypes.c_size_t
    lib.indexer_topk.argtypes = [P(_Batch), P(_Indexer), ctypes.c_void_p, ctypes.c_void_p,
                                 ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.indexer_topk.restype = ctypes.c_int
    lib.sparse_mla_attn.argtypes = [P(_Batch), P(_Attn), ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.sparse_mla_attn.restype = ctypes.c_int
    lib.sparse_mla_attn_static.argtypes = [P(_Batch), P(_Attn), ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p]
    lib.sparse_mla_attn_static.restype = ctypes.c_int
    lib.dsa_decode.argtypes = [P(_Batch), P(_Indexer), P(_Attn), ctypes.c_void_p, ctypes.c_void_p,
                               ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                               ctypes.c_void_p]
    lib.dsa_decode.restype = ctypes.c_int
    lib.dsa_get_status.argtypes = [ctypes.c_void_p, ctypes.c_void_p, P(ctypes.c_int32)]
    lib.dsa_get_status.restype = ctypes.c_int
    lib.dsa_decode_launch_count.argtypes = [P(_Batch), P(_Indexer), P(_Attn)]
    lib.dsa_decode_launch_count.restype = ctypes.c_int32
    lib.dsa_prolog_workspace_size.argtypes = [P(_Batch), P(_Prolog)]
    lib.dsa_prolog_workspace_size.restype = ctypes.c_size_t
    lib.indexer_prolog.argtypes = [P(_Batch), P(_Prolog), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                   ctypes.c_void_p]
    lib.indexer_prolog.restype = ctypes.c_int
    lib.dsa_prolog_packed_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
    lib.dsa_prolog_packed_bytes.restype = ctypes.c_size_t
    lib.indexer_prolog_pack.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.c_int32, ctypes.c_void_p]
    lib.indexer_prolog_pack.restype = ctypes.c_int
    # (argument blocks of these are packed bytes, or structures by reference)
    lib.dsa_qk_norm_rope.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p]
    lib.dsa_qk_norm_rope.restype = ctypes.c_int
    lib.dsa_chunk_scratch_size.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.dsa_chunk_scratch_size.restype = ctypes.c_size_t
    lib.dsa_chunk_attn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                   ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.dsa_chunk_attn.restype = ctypes.c_int
    lib.dsa_weight_scratch_size.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.dsa_weight_scratch_size.restype = ctypes.c_size_t
    lib.dsa_attn_weight.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_float,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.dsa_attn_weight.restype = ctypes.c_int
    lib.dsa_evict_scratch_size.argtypes = [ctypes.c_void_p]
    lib.dsa_evict_scratch_size.restype = ctypes.c_size_t
    lib.dsa_cache_evict.argtypes = [ctypes.c_void_p, P(_Evict), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_size_t, ctypes.c_void_p]
    lib.dsa_cache_evict.restype = ctypes.c_int
    lib.dsa_status_str.argtypes = [ctypes.c_int32]
    lib.dsa_status_str.restype = ctypes.c_char_p
    lib.dsa_version.restype = ctypes.c_char_p
    lib.dsa_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_str(code: int) -> str:
    return load_library().dsa_status_str(int(code)).decode()


def last_error() -> str:
    """Text of the last failure the library recorded on this thread ("" if none)."""
    return load_library().dsa_last_error().decode()


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _check(t, name, dtype, ndim=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if shape is not None:
        for i, s in enumerate(shape):
            if s is not None and t.shape[i] != s:
                raise ValueError(f"{name} dim {i} must be {s}, got {tuple(t.shape)}")


@dataclass
class Batch:
    """Sequences of one step: device seq_lens [B], cu_q [B+1], block_table [B, max_blocks]
    (int32) plus the host-side bounds the launcher sizes its grids with."""
    seq_lens: "object"
    cu_q: "object"
    block_table: "object"
    num_blocks: int
    max_seq_len: int
    max_q_per_seq: int

    @classmethod
    def from_tensors(cls, seq_lens, cu_q, block_table, num_blocks, max_seq_len=None, max_q_per_seq=None):
        for t, n in ((seq_lens, "seq_lens"), (cu_q, "cu_q"), (block_table, "block_table")):
            _check(t, n, torch.int32)
        if max_seq_len is None:
            max_seq_len = int(seq_lens.max().item())
        if max_q_per_seq is None:
            max_q_per_seq = int((cu_q[1:] - cu_q[:-1]).max().item())
        return cls(seq_lens, cu_q, block_table, int(num_blocks), int(max_seq_len), int(max_q_per_seq))

    @property
    def B(self) -> int:
        return int(self.seq_lens.shape[0])

    def c(self, T: int) -> _Batch:
        return _Batch(self.B, int(T), _ptr(self.seq_lens), _ptr(self.cu_q), _ptr(self.block_table),
                      int(self.block_table.shape[1]), self.num_blocks, self.max_seq_len, self.max_q_per_seq)


def _indexer_struct(q_idx, w, k_cache, k_scale, K, q_scale=None):
    if q_scale is not None:
        # MXFP8 queries and keys
        _check(q_idx, "q_idx", torch.uint8, 3)
        T, H_I, D_I = q_idx.shape
        _check(q_scale, "q_scale", torch.uint8, 3, (T, H_I, D_I // 32))
        _check(k_cache, "k_cache", torch.uint8, 3, (None, 64, D_I))
        if k_scale is None:
            raise ValueError("MXFP8 queries need MXFP8 keys (k_scale)")
        _check(k_scale, "k_scale", torch.uint8, 3, (k_cache.shape[0], 64, D_I // 32))
        dt, qt = KEY_MXFP8, Q_MXFP8
    else:
        _check(q_idx, "q_idx", torch.bfloat16, 3)
        T, H_I, D_I = q_idx.shape
        qt = Q_BF16
        if k_scale is None:
            _check(k_cache, "k_cache", torch.bfloat16, 3, (None, 64, D_I))
            dt = KEY_BF16
        else:
            _check(k_cache, "k_cache", torch.uint8, 3, (None, 64, D_I))
            _check(k_scale, "k_scale", torch.float32, 3, (k_cache.shape[0], 64, D_I // 64))
            dt = KEY_FP8_E4M3
    _check(w, "w", torch.float32, 2, (T, H_I))
    return _Indexer(_ptr(q_idx), _ptr(w), _ptr(k_cache), _ptr(k_scale), dt, H_I, D_I, int(K), qt,
                    _ptr(q_scale)), T


def _attn_struct(q, kv_cache, sm_scale, kv_scale=None):
    _check(q, "q", torch.bfloat16, 3, (None, None, 576))
    if kv_scale is None:
        _check(kv_cache, "kv_cache", torch.bfloat16, 3, (None, 64, 576))
        kt = KV_BF16
    else:
        # FP8 latent cache: e4m3 codes and one fp32 scale per 128-element tile of a row
        _check(kv_cache, "kv_cache", torch.uint8, 3, (None, 64, 576))
        _check(kv_scale, "kv_scale", torch.float32, 3, (kv_cache.shape[0], 64, 5))
        kt = KV_FP8
    return _Attn(_ptr(q), _ptr(kv_cache), int(q.shape[1]), float(sm_scale), kt, _ptr(kv_scale)), int(q.shape[0])


class Workspace:
    """Caller-owned, zero-filled device workspace (grows on demand).  The
    kernels leave it zero-filled after every successful call."""

    def __init__(self, device=None):
        self.device = torch.device("cuda") if device is None else torch.device(device)
        self.buf = None

    def get(self, nbytes: int):
        if self.buf is None or self.buf.numel() < nbytes:
            self.buf = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=self.device)
        return self.buf

    def reset(self):
        if self.buf is not None:
            self.buf.zero_()


_default_ws = {}


def _workspace(ws, device):
    if ws is not None:
        return ws
    device = torch.device(device)
    key = device.index if device.index is not None else torch.cuda.current_device()
    if key not in _default_ws:
        _default_ws[key] = Workspace(torch.device("cuda", key))
    return _default_ws[key]


def indexer_topk(batch: Batch, q_idx, w, k_cache, K: int, k_scale=None, q_scale=None, *, out_idx=None, out_score=None,
                 want_score: bool = True, workspace: Optional[Workspace] = None, stream=None):
    """Fused Lightning Indexer + Top-K.  Returns (idx [T,K] int32, score [T,K] fp32 or None)."""
    lib = load_library()
    ix, T = _indexer_struct(q_idx, w, k_cache, k_scale, K, q_scale)
    cb = batch.c(T)
    if out_idx is None:
        out_idx = torch.empty((T, K), dtype=torch.int32, device=q_idx.device)
    if out_score is None and want_score:
        out_score = torch.empty((T, K), dtype=torch.float32, device=q_idx.device)
    ws = _workspace(workspace, q_idx.device)
    need = lib.dsa_workspace_size(ctypes.byref(cb), ctypes.byref(ix), None)
    if need == 0:
        raise DsaError(2, "dsa_workspace_size")
    buf = ws.get(need)
    rc = lib.indexer_topk(ctypes.byref(cb), ctypes.byref(ix), _ptr(out_idx), _ptr(out_score), _ptr(buf),
                          buf.numel(), _stream(stream))
    if rc != 0:
        raise DsaError(rc, "indexer_topk")
    return out_idx, out_score


def sparse_mla_attn(batch: Batch, q, kv_cache, idx, sm_scale: float, *, kv_scale=None, out=None, lse=None,
                    want_lse: bool = True, workspace: Optional[Workspace] = None, stream=None):
    """Sparse Flash Attention over the selected latent rows (bf16 cache, or an FP8 cache of e4m3
    codes with kv_scale).  Returns (out [T,H,512] bf16, lse [T,H] fp32)."""
    lib = load_library()
    at, T = _attn_struct(q, kv_cache, sm_scale, kv_scale)
    _check(idx, "idx", torch.int32, 2, (T, None))
    K = int(idx.shape[1])
    cb = batch.c(T)
    if out is None:
        out = torch.empty((T, q.shape[1], 512), dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((T, q.shape[1]), dtype=torch.float32, device=q.device)
    ws = _workspace(workspace, q.device)
    need = lib.dsa_workspace_size(ctypes.byref(cb), None, ctypes.byref(at))
    if need == 0:
        raise DsaError(2, "dsa_workspace_size")
    buf = ws.get(need)
    rc = lib.sparse_mla_attn(ctypes.byref(cb), ctypes.byref(at), _ptr(idx), K, _ptr(out), _ptr(lse),
                             _ptr(buf), buf.numel(), _stream(stream))
    if rc != 0:
        raise DsaError(rc, "sparse_mla_attn")
    return out, lse


def sparse_mla_attn_static(batch: Batch, q, kv_cache, idx, sm_scale: float, *, out=None, lse=None,
                           want_lse: bool = True, stream=None):
    """sparse_mla_attn without a workspace: the library's fixed scratch is used
    (calls on one device must not overlap).  Returns (out, lse)."""
    lib = load_library()
    at, T = _attn_struct(q, kv_cache, sm_scale)
    _check(idx, "idx", torch.int32, 2, (T, None))
    K = int(idx.shape[1])
    cb = batch.c(T)
    if out is None:
        out = torch.empty((T, q.shape[1], 512), dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((T, q.shape[1]), dtype=torch.float32, device=q.device)
    rc = lib.sparse_mla_attn_static(ctypes.byref(cb), ctypes.byref(at), _ptr(idx), K, _ptr(out), _ptr(lse),
                                    _stream(stream))
    if rc != 0:
        raise DsaError(rc, "sparse_mla_attn_static", last_error())
    return out, lse


def dsa_decode(batch: Batch, q_idx, w, k_cache, q, kv_cache, K: int, sm_scale: float, k_scale=None, q_scale=None, *,
               kv_scale=None, out_idx=None, out_score=None, out=None, lse=None, want_score=False, want_lse=False,
               workspace: Optional[Workspace] = None, stream=None):
    """Whole step (indexer + Top-K + sparse attention) on one stream.
    Returns (idx, score or None, out, lse or None)."""
    lib = load_library()
    ix, T = _indexer_struct(q_idx, w, k_cache, k_scale, K, q_scale)
    at, T2 = _attn_struct(q, kv_cache, sm_scale, kv_scale)
    if T2 != T:
        raise ValueError("q_idx and q disagree on the number of tokens")
    cb = batch.c(T)
    dev = q.device
    if out_idx is None:
        out_idx = torch.empty((T, K), dtype=torch.int32, device=dev)
    if out_score is None and want_score:
        out_score = torch.empty((T, K), dtype=torch.float32, device=dev)
    if out is None:
        out = torch.empty((T, q.shape[1], 512), dtype=torch.bfloat16, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((T, q.shape[1]), dtype=torch.float32, device=dev)
    ws = _workspace(workspace, dev)
    need = lib.dsa_workspace_size(ctypes.byref(cb), ctypes.byref(ix), ctypes.byref(at))
    if need == 0:
        raise DsaError(2, "dsa_workspace_size")
    buf = ws.get(need)
    rc = lib.dsa_decode(ctypes.byref(cb), ctypes.byref(ix), ctypes.byref(at), _ptr(out_idx), _ptr(out_score),
                        _ptr(out), _ptr(lse), _ptr(buf), buf.numel(), _stream(stream))
    if rc != 0:
        raise DsaError(rc, "dsa_decode")
    return out_idx, out_score, out, lse


_prolog_ws = {}


def prolog_workspace(device=None) -> Workspace:
    """The default workspace of indexer_prolog on a device (kept apart from the
    other entry points' workspace: its partial-tile region is scratch)."""
    device = torch.device("cuda") if device is None else torch.device(device)
    key = device.index if device.index is not None else torch.cuda.current_device()
    if key not in _prolog_ws:
        _prolog_ws[key] = Workspace(torch.device("cuda", key))
    return _prolog_ws[key]


class PackedWeights:
    """Prolog weights in the tile-packed layout (see prolog_pack_weights)."""

    def __init__(self, data, H_I: int, D_I: int, d_model: int):
        self.data, self.H_I, self.D_I, self.d_model = data, int(H_I), int(D_I), int(d_model)


def prolog_pack_weights(w_proj, H_I: int, D_I: int, stream=None) -> PackedWeights:
    """Tile-packed copy of the row-major prolog weights w_proj [H_I*D_I + D_I + H_I, d] (bf16):
    each 128-row x 64-column block contiguous (done once, when the weights are loaded)."""
    lib = load_library()
    _check(w_proj, "w_proj", torch.bfloat16, 2, (H_I * D_I + D_I + H_I, None))
    d = int(w_proj.shape[1])
    n = lib.dsa_prolog_packed_bytes(int(H_I), int(D_I), d)
    if n == 0:
        raise DsaError(1, "dsa_prolog_packed_bytes")
    out = torch.empty(n // 2, dtype=torch.bfloat16, device=w_proj.device)
    rc = lib.indexer_prolog_pack(_ptr(w_proj), _ptr(out), int(H_I), int(D_I), d, _stream(stream))
    if rc != 0:
        raise DsaError(rc, "indexer_prolog_pack")
    return PackedWeights(out, H_I, D_I, d)


def indexer_prolog(batch: Batch, x, w_proj, k_gamma, eps: float, k_cache, k_scale=None, mx: bool = False, *,
                   H_I: Optional[int] = None, q_out=None, q_scale_out=None, w_out=None,
                   workspace: Optional[Workspace] = None, stream=None):
    """Indexer prolog: projects the step's hidden states x [T, d] with the stacked rows
    w_proj [H_I*D_I + D_I + H_I, d] (bf16), RMS-normalizes the keys (k_gamma [D_I] fp32,
    eps) and writes them into the tokens' rows of the paged key cache (format given by
    k_cache / k_scale as for indexer_topk; MXFP8 when mx).  Returns (q_idx [T, H_I, D_I]
    bf16 or e4m3 codes, q_scale [T, H_I, D_I/32] uint8 or None, w [T, H_I] fp32)."""
    lib = load_library()
    _check(x, "x", torch.bfloat16, 2)
    _check(k_gamma, "k_gamma", torch.float32, 1)
    T, d = x.shape
    D_I = int(k_gamma.shape[0])
    if isinstance(w_proj, PackedWeights):
        if w_proj.D_I != D_I or w_proj.d_model != d:
            raise ValueError("packed weights were made for another D_I or d_model")
        H_I, w_ptr, layout = w_proj.H_I, _ptr(w_proj.data), 1
    else:
        _check(w_proj, "w_proj", torch.bfloat16, 2, (None, x.shape[1]))
        n_out = int(w_proj.shape[0])
        H_I = (n_out - D_I) // (D_I + 1) if H_I is None else int(H_I)
        if H_I * D_I + D_I + H_I != n_out:
            raise ValueError(f"w_proj has {n_out} rows; H_I*D_I + D_I + H_I rows are needed")
        w_ptr, layout = _ptr(w_proj), 0
    if mx:
        _check(k_cache, "k_cache", torch.uint8, 3, (None, 64, D_I))
        if k_scale is None:
            raise ValueError("MXFP8 keys need k_scale")
        _check(k_scale, "k_scale", torch.uint8, 3, (k_cache.shape[0], 64, D_I // 32))
        kt, qt = KEY_MXFP8, Q_MXFP8
    elif k_scale is None:
        _check(k_cache, "k_cache", torch.bfloat16, 3, (None, 64, D_I))
        kt, qt = KEY_BF16, Q_BF16
    else:
        _check(k_cache, "k_cache", torch.uint8, 3, (None, 64, D_I))
        _check(k_scale, "k_scale", torch.float32, 3, (k_cache.shape[0], 64, D_I // 64))
        kt, qt = KEY_FP8_E4M3, Q_BF16
    dev = x.device
    if q_out is None:
        q_out = torch.empty((T, H_I, D_I), dtype=torch.uint8 if mx else torch.bfloat16, device=dev)
    if mx and q_scale_out is None:
        q_scale_out = torch.empty((T, H_I, D_I // 32), dtype=torch.uint8, device=dev)
    if w_out is None:
        w_out = torch.empty((T, H_I), dtype=torch.float32, device=dev)
    pr = _Prolog(_ptr(x), w_ptr, _ptr(k_gamma), float(eps), int(d), H_I, D_I, kt, qt, layout)
    cb = batch.c(T)
    ws = workspace if workspace is not None else prolog_workspace(dev)
    need = lib.dsa_prolog_workspace_size(ctypes.byref(cb), ctypes.byref(pr))
    if need == 0:
        raise DsaError(2, "dsa_prolog_workspace_size")
    buf = ws.get(need)
    rc = lib.indexer_prolog(ctypes.byref(cb), ctypes.byref(pr), _ptr(q_out), _ptr(q_scale_out), _ptr(w_out),
                            _ptr(k_cache), _ptr(k_scale), _ptr(buf), buf.numel(), _stream(stream))
    if rc != 0:
        raise DsaError(rc, "indexer_prolog")
    return q_out, q_scale_out, w_out


_status_ws = {}
_status_lock = threading.Lock()


def status_workspace(device=None) -> Workspace:
    """The default status area of the dsa_ operators over the paged cache on a
    device: read it with get_status(status_workspace(device)).  It keeps its address for
    the life of the process, so captured graphs may hold it."""
    key = device if isinstance(device, int) else None if device is None else torch.device(device).index
    if key is None:
        key = torch.cuda.current_device()
    if key not in _status_ws:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the default status area is not there yet: call status_workspace() before the capture")
        with _status_lock:
            # (another thread may have been first: the area that it was given stays)
            if key not in _status_ws:
                ws = Workspace(torch.device("cuda", key))
                ws.get(256)
                # zeroed before any stream can use it
                torch.cuda.synchronize(ws.device)
                _status_ws[key] = ws
    return _status_ws[key]


def _status(ws: Optional[Workspace], dev: int) -> int:
    """Pointer of a call's status area, on the device that is current."""
    if ws is None:
        ws = _status_ws.get(dev) or status_workspace(dev)
    t = ws.get(256)
    if t.get_device() != dev:
        raise ValueError(f"the workspace is on {t.device}, the tensors on cuda:{dev}")
    return t.data_ptr()


class _On:
    """The device of a call's tensors (by index) made current, and its stream (the device's
    current one by default), so that outputs and scratch are allocated for the stream that
    uses them.  Entering it gives the stream's handle."""
    __slots__ = ("dev", "stream", "left")

    def __init__(self, dev: int, stream):
        self.dev, self.stream, self.left = dev, stream, ()

    def __enter__(self):
        if self.stream is not None:
            if self.stream.device.index != self.dev:
                raise ValueError(f"the stream is on {self.stream.device}, the tensors on cuda:{self.dev}")
            self.left = (torch.cuda.device(self.dev), torch.cuda.stream(self.stream))
        elif torch._C._cuda_getDevice() != self.dev:
            self.left = (torch.cuda.device(self.dev),)
        for c in self.left:
            c.__enter__()
        return torch._C._cuda_getCurrentRawStream(self.dev)

    def __exit__(self, *exc):
        for c in reversed(self.left):
            c.__exit__(*exc)


def _dense(t, name, dtype, shape, dev: int) -> int:
    """Pointer of a dense tensor of this type, shape and device index; raises what is wrong with another."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev >= 0 \
            and t.is_contiguous():
        return t.data_ptr()
    _check(t, name, dtype, len(shape), shape)
    raise ValueError(f"{name} is on {t.device}, other tensors of the call on cuda:{dev}")


def _packer(struct_type):
    """pack() of a ctypes structure's fields, in their order: a third of the time of an instance."""
    code = {ctypes.c_void_p: "P", ctypes.c_int64: "q", ctypes.c_int32: "i", ctypes.c_float: "f"}
    packed = struct.Struct("@" + "".join(code[t] for _, t in struct_type._fields_) + "0P")
    assert packed.size == ctypes.sizeof(struct_type)
    return packed.pack


_pack_batch, _pack_rope, _pack_attn = _packer(_Batch), _packer(_Rope), _packer(_Attn)


def _vector(t, name, dtype, dev: int):
    """(pointer, length) of a dense vector."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == 1 and t.get_device() == dev >= 0 \
            and t.is_contiguous():
        return t.data_ptr(), t.numel()
    _check(t, name, dtype, 1)
    raise ValueError(f"{name} is on {t.device}, other tensors of the call on cuda:{dev}")


def _batch_args(batch: Batch, T: int, dev: int):
    """(argument block, number of sequences) of a batch, its tensors checked."""
    i32, table = torch.int32, batch.block_table
    lens, B = _vector(batch.seq_lens, "seq_lens", i32, dev)
    cu, n = _vector(batch.cu_q, "cu_q", i32, dev)
    if n != B + 1:
        raise ValueError(f"cu_q dim 0 must be {B + 1}, got {n}")
    W = table.shape[1] if isinstance(table, torch.Tensor) and table.dim() == 2 else None
    tp = _dense(table, "block_table", i32, (B, W), dev)
    return _pack_batch(B, T, lens, cu, tp, W, batch.num_blocks, batch.max_seq_len, batch.max_q_per_seq), B


def _rows(t, name, ndim: int, dev: int):
    """Pointer, shape and strides of a bf16 CUDA tensor of dense, 16-byte aligned rows (other strides may be any)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.dim() == ndim and t.get_device() == dev >= 0):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype is not torch.bfloat16:
            raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
        if t.dim() != ndim:
            raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
        raise ValueError(f"{name} is on {t.device}, other tensors of the call on cuda:{dev}")
    shape, p = t.shape, t.data_ptr()
    if t.is_contiguous():
        # (not t.stride(): that of a dimension of one element may be anything)
        strides = (shape[1] * shape[2], shape[2], 1) if ndim == 3 else (shape[1], 1)
    else:
        # the stride of a dimension of one element is never used
        strides = [s if n > 1 else 0 for n, s in zip(shape, t.stride())]
        if (shape[-1] > 1 and strides[-1] != 1) or any(s % 8 for s in strides[:-1]):
            raise ValueError(f"{name} needs dense rows 16 bytes apart, got strides {t.stride()}")
    if p % 16:
        raise ValueError(f"{name} must be 16-byte aligned")
    return p, shape, strides


def dsa_qk_norm_rope(batch: Batch, inv_freq, q=None, k=None, *, q_gamma=None, k_gamma=None, eps: float = 1e-6,
                     rope_off: Optional[int] = None, interleaved: bool = False, positions=None, k_cache=None,
                     k_scale=None, q_out=None, workspace: Optional[Workspace] = None, stream=None):
    """Per-head RMS norm and position rotation of the step's queries q [T, H, D] and keys
    k [T, D] (bf16, rows may be strided) in one pass; the keys go into the tokens' rows of
    k_cache (bf16 [nblk, 64, D], or uint8 e4m3 codes of 576-element latent rows with k_scale
    [nblk, 64, 5]).  q_gamma / k_gamma (fp32) normalize as many leading elements as they
    have; inv_freq (fp32, or None) rotates twice its length from rope_off on (the row's end
    by default) by the tokens' places in their sequences, or by positions [T] int32.
    Returns q_out [T, H, D] (which may be q itself), or None without q."""
    lib = load_library()
    main = q if q is not None else k
    if main is None:
        raise ValueError("q or k is needed")
    dev = main.get_device() if isinstance(main, torch.Tensor) else -1
    f32 = torch.float32
    H = qp = kp = cp = sp = qn = kn = R = 0
    qs, ks, kt = (0, 0), (0,), KV_BF16
    qg = kg = fp = pp = 0
    if q is not None:
        qp, (T, H, D), qs = _rows(q, "q", 3, dev)
    if k is not None:
        kp, shape, ks = _rows(k, "k", 2, dev)
        if q is not None and shape != (T, D):
            raise ValueError(f"k {tuple(shape)} does not match q {tuple(q.shape)}")
        T, D = shape
        if k_scale is None:
            cp = _dense(k_cache, "k_cache", torch.bfloat16, (batch.num_blocks, 64, D), dev)
        else:
            kt = KV_FP8
            cp = _dense(k_cache, "k_cache", torch.uint8, (batch.num_blocks, 64, D), dev)
            sp = _dense(k_scale, "k_scale", f32, (batch.num_blocks, 64, 5), dev)
    if q_gamma is not None:
        qg, qn = _vector(q_gamma, "q_gamma", f32, dev)
    if k_gamma is not None:
        kg, kn = _vector(k_gamma, "k_gamma", f32, dev)
    if inv_freq is not None:
        fp, R = _vector(inv_freq, "inv_freq", f32, dev)
        R *= 2
    if positions is not None:
        pp = _dense(positions, "positions", torch.int32, (T,), dev)
    cb, _ = _batch_args(batch, T, dev)
    s = _pack_rope(qp, qs[0], qs[1], kp, ks[0], H, D, qg, kg, qn, kn, eps, fp, R,
                   D - R if rope_off is None else rope_off, bool(interleaved), pp, kt)
    with _On(dev, stream) as on:
        status = _status(workspace, dev)
        op = 0
        if q is not None:
            if q_out is None:
                q_out = torch.empty_like(q) if q.is_contiguous() else torch.empty(T, H, D, dtype=q.dtype, device=q.device)
                op = q_out.data_ptr()
            else:
                op = _dense(q_out, "q_out", torch.bfloat16, (T, H, D), dev)
                if op == qp and not q.is_contiguous():
                    raise ValueError("q_out may be q only when q is contiguous")
        rc = lib.dsa_qk_norm_rope(cb, s, op, cp, sp, status, on)
    if rc != 0:
        raise DsaError(rc, "dsa_qk_norm_rope")
    return q_out if q is not None else None


def _latent_attn(q, kv_cache, sm_scale, kv_scale, num_blocks: int):
    """(argument block, T, H, device index) of dense queries and the latent cache they attend to."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        _check(q, "q", torch.bfloat16, 3)
    T, H, _ = q.shape
    dev = q.get_device()
    qp = _dense(q, "q", torch.bfloat16, (T, H, 576), dev)
    if kv_scale is None:
        kt, sp = KV_BF16, 0
        cp = _dense(kv_cache, "kv_cache", torch.bfloat16, (num_blocks, 64, 576), dev)
    else:
        kt, sp = KV_FP8, _dense(kv_scale, "kv_scale", torch.float32, (num_blocks, 64, 5), dev)
        cp = _dense(kv_cache, "kv_cache", torch.uint8, (num_blocks, 64, 576), dev)
    return _pack_attn(qp, cp, H, sm_scale, kt, sp), T, H, dev


def dsa_chunk_attn(batch: Batch, q, kv_cache, sm_scale: float, *, kv_scale=None, out=None, lse=None,
                   want_lse: bool = True, workspace: Optional[Workspace] = None, stream=None):
    """Dense attention of the step's new tokens q [T, H, 576] over the paged latent cache
    (bf16, or FP8 codes with kv_scale): each sees all positions up to its own.  Returns
    (out [T, H, 512] bf16, lse [T, H] fp32 or None).  Scratch is allocated per call, on the
    call's stream; the status word is that of `workspace` (status_workspace() by default)."""
    lib = load_library()
    at, T, H, dev = _latent_attn(q, kv_cache, sm_scale, kv_scale, batch.num_blocks)
    cb, _ = _batch_args(batch, T, dev)
    with _On(dev, stream) as on:
        status = _status(workspace, dev)
        need = lib.dsa_chunk_scratch_size(cb, at)
        if need == 0:
            raise DsaError(2, "dsa_chunk_scratch_size")
        if out is None:
            out = torch.empty(T, H, 512, dtype=torch.bfloat16, device=q.device)
            op = out.data_ptr()
        else:
            op = _dense(out, "out", torch.bfloat16, (T, H, 512), dev)
        if lse is None and want_lse:
            lse = torch.empty(T, H, dtype=torch.float32, device=q.device)
            lp = lse.data_ptr()
        else:
            lp = None if lse is None else _dense(lse, "lse", torch.float32, (T, H), dev)
        scratch = torch.empty(need, dtype=torch.uint8, device=q.device)
        rc = lib.dsa_chunk_attn(cb, at, op, lp, status, scratch.data_ptr(), need, on)
    if rc != 0:
        raise DsaError(rc, "dsa_chunk_attn")
    return out, lse


def dsa_attn_weight(batch: Batch, q, kv_cache, sm_scale: float, lse, weight, *, decay: float = 1.0, kv_scale=None,
                    workspace: Optional[Workspace] = None, stream=None):
    """Adds to weight [B, >= max_seq_len] fp32 (after scaling what it holds by decay) the softmax
    weight that the step's new tokens give to each cached position, over tokens and heads; lse
    [T, H] is the attention's.  Returns weight."""
    lib = load_library()
    at, T, H, dev = _latent_attn(q, kv_cache, sm_scale, kv_scale, batch.num_blocks)
    cb, B = _batch_args(batch, T, dev)
    lp = _dense(lse, "lse", torch.float32, (T, H), dev)
    n = weight.shape[1] if isinstance(weight, torch.Tensor) and weight.dim() == 2 else None
    wp = _dense(weight, "weight", torch.float32, (B, n), dev)
    with _On(dev, stream) as on:
        status = _status(workspace, dev)
        need = lib.dsa_weight_scratch_size(cb, at)
        if need == 0:
            raise DsaError(2, "dsa_weight_scratch_size")
        scratch = torch.empty(need, dtype=torch.uint8, device=q.device)
        rc = lib.dsa_attn_weight(cb, at, lp, wp, n, decay, status, scratch.data_ptr(), need, on)
    if rc != 0:
        raise DsaError(rc, "dsa_attn_weight")
    return weight


def dsa_cache_evict(batch: Batch, weight, keep: int, new_table, arrays, new_arrays, *, sink: int = 0, recent: int = 0,
                    new_weight=None, out_idx=None, out_len=None, workspace: Optional[Workspace] = None, stream=None):
    """Keeps `keep` positions of each sequence: the first `sink`, the last `recent`, then those
    with the largest weight [B, >= max_seq_len] fp32.  Copies their rows, in ascending order, from
    each of `arrays` ([num_blocks, 64, ...], any type: latent rows, index keys, their scales) to
    the pages new_table [B, n] int32 of the tensor at the same place in `new_arrays`
    ([new blocks, 64, ...], as many for each), and their weights to new_weight.  Returns (idx
    [B, keep] int32, -1 padded; len [B] int32)."""
    lib = load_library()
    dev = weight.get_device() if isinstance(weight, torch.Tensor) else -1
    n = weight.shape[1] if isinstance(weight, torch.Tensor) and weight.dim() == 2 else None
    cb, B = _batch_args(batch, max(1, batch.max_q_per_seq), dev)
    wp = _dense(weight, "weight", torch.float32, (B, n), dev)
    W = new_table.shape[1] if isinstance(new_table, torch.Tensor) and new_table.dim() == 2 else None
    tp = _dense(new_table, "new_table", torch.int32, (B, W), dev)
    if keep > 0x7FFFFFFF:
        raise ValueError(f"keep {keep} does not fit 32 bits")
    if keep < 0 or sink < 0 or recent < 0 or sink + recent > keep:
        raise ValueError(f"keep {keep} has no room for sink {sink} and recent {recent}")
    if len(arrays) != len(new_arrays):
        raise ValueError(f"{len(arrays)} arrays, {len(new_arrays)} new ones")
    old_blocks, new_blocks = batch.num_blocks, new_arrays[0].shape[0] if len(new_arrays) else 1
    copies = (_CacheArray * max(1, len(arrays)))()
    for i, (a, c) in enumerate(zip(arrays, new_arrays)):
        if not isinstance(a, torch.Tensor) or a.dim() < 2:
            raise ValueError(f"arrays[{i}] must be a tensor [num_blocks, 64, ...]")
        row, e = a.shape[2:], copies[i]
        e.src = _dense(a, f"arrays[{i}]", a.dtype, (old_blocks, 64) + row, dev)
        e.dst = _dense(c, f"new_arrays[{i}]", a.dtype, (new_blocks, 64) + row, dev)
        e.row_bytes = a.nbytes // (64 * old_blocks) if old_blocks else 0
    np_, nn = None, 0
    if new_weight is not None:
        nn = new_weight.shape[1] if isinstance(new_weight, torch.Tensor) and new_weight.dim() == 2 else None
        np_ = _dense(new_weight, "new_weight", torch.float32, (B, nn), dev)
    s = _Evict(wp, n, np_, nn, keep, sink, recent, tp, W, new_blocks, copies, len(arrays))
    with _On(dev, stream) as on:
        status = _status(workspace, dev)
        if out_idx is None:
            out_idx = torch.empty(B, keep, dtype=torch.int32, device=weight.device)
            ip = out_idx.data_ptr()
        else:
            ip = _dense(out_idx, "out_idx", torch.int32, (B, keep), dev)
        if out_len is None:
            out_len = torch.empty(B, dtype=torch.int32, device=weight.device)
            lp = out_len.data_ptr()
        else:
            lp = _dense(out_len, "out_len", torch.int32, (B,), dev)
        need = lib.dsa_evict_scratch_size(cb)
        scratch = torch.empty(max(need, 256), dtype=torch.uint8, device=weight.device)
        rc = lib.dsa_cache_evict(cb, ctypes.byref(s), ip, lp, status, scratch.data_ptr(), need, on)
    if rc != 0:
        raise DsaError(rc, "dsa_cache_evict")
    return out_idx, out_len


def decode_launch_count(batch: Batch, q_idx, w, k_cache, q, kv_cache, K: int, sm_scale: float,
                        k_scale=None, q_scale=None, kv_scale=None) -> int:
    """Kernel launches one dsa_decode call enqueues for these shapes."""
    lib = load_library()
    ix, T = _indexer_struct(q_idx, w, k_cache, k_scale, K, q_scale)
    at, _ = _attn_struct(q, kv_cache, sm_scale, kv_scale)
    cb = batch.c(T)
    n = lib.dsa_decode_launch_count(ctypes.byref(cb), ctypes.byref(ix), ctypes.byref(at))
    if n < 0:
        raise DsaError(2, "dsa_decode_launch_count")
    return int(n)


def get_status(workspace: Optional[Workspace] = None, device=None, stream=None) -> int:
    """Synchronize and read (and clear) the device status word of a workspace."""
    lib = load_library()
    ws = _workspace(workspace, device if device is not None else torch.device("cuda"))
    buf = ws.get(256)
    code = ctypes.c_int32(0)
    rc = lib.dsa_get_status(_ptr(buf), _stream(stream), ctypes.byref(code))
    if rc != 0:
        raise DsaError(rc, "dsa_get_status")
    return int(code.value)
