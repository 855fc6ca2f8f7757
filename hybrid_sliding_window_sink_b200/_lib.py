"""ctypes binding of libmimo_attn.so (include/mimo_attn.h): argument marshalling only.

Each function takes torch tensors, checks dtype / device / contiguity / shape,
passes raw device pointers and the current CUDA stream to the C entry point of
the same name, and raises ``MimoError`` on any status other than MIMO_OK. All
arithmetic happens in the library's CUDA kernels. The library must be built
(``python -m hybrid_sliding_window_sink_b200.build``); there is no fallback.
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmimo_attn.so")

MIMO_CACHE_RING = 0
MIMO_CACHE_LINEAR = 1
MIMO_OP_DECODE = 0
MIMO_OP_SPARSE = 1
STATUS = {0: "MIMO_OK", 1: "MIMO_ERR_NULL", 2: "MIMO_ERR_SHAPE", 3: "MIMO_ERR_UNSUPPORTED",
          4: "MIMO_ERR_ALIGN", 5: "MIMO_ERR_WORKSPACE", 6: "MIMO_ERR_CUDA", 7: "MIMO_ERR_DEVICE"}

#: Every symbol include/mimo_attn.h declares.
EXPORTS = ("mimo_attn_prefill", "mimo_attn_decode", "mimo_attn_sparse", "mimo_attn_sparse_noalloc",
           "mimo_attn_decode_mq", "mimo_attn_decode_mq_workspace_size", "mimo_attn_workspace_size",
           "mimo_attn_decode_fp8", "mimo_attn_sparse_fp8", "mimo_attn_prefill_chunk",
           "mimo_attn_cache_append", "mimo_attn_select_tokens", "mimo_attn_select_workspace_size",
           "mimo_attn_prefill_first", "mimo_attn_decode_paged", "mimo_attn_decode_paged_fp8", "mimo_attn_decode_paged_workspace_size",
           "mimo_attn_cache_append_paged", "mimo_attn_cache_append_paged_fp8", "mimo_attn_verify_drafts",
           "mimo_attn_check_indices", "mimo_attn_last_device_error", "mimo_attn_device_status",
           "mimo_status_string", "mimo_attn_version")


class MimoError(RuntimeError):
    def __init__(self, fn, status, lib=None):
        msg = STATUS.get(status, str(status))
        if lib is not None:
            msg += ": " + lib.mimo_status_string(status).decode()
        super().__init__(f"{fn} failed with {msg}")
        self.status = status


class MimoShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("seqlen", ctypes.c_int), ("n_q_heads", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim_qk", ctypes.c_int),
                ("head_dim_v", ctypes.c_int), ("softmax_scale", ctypes.c_float)]


class MimoPages(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("max_pages", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("page_stride_tokens", ctypes.c_longlong)]


_LIB = None
_CALL = None      # _call.so bound to the library _CALL_LIB, or False when it has not been built
_CALL_LIB = None


def lib():
    """Load libmimo_attn.so once; raise if it has not been built."""
    global _LIB
    if _LIB is None:
        _LIB = load(LIB_PATH)
    return _LIB


def _usual():
    """The C++ marshalling of the usual calls (csrc/binding.cpp), bound to the library in use, or
    False. Its functions return None for a call that is not usual, which the Python code then makes."""
    global _CALL, _CALL_LIB
    if _CALL_LIB is not _LIB or _LIB is None:
        L = lib()
        if _CALL is None:
            try:
                from . import _call as _CALL
            except ImportError:
                _CALL = False
        if _CALL:
            addresses = [ctypes.cast(getattr(L, "mimo_attn_" + f), ctypes.c_void_p).value for f in (
                "prefill_first", "decode_paged", "decode_paged_fp8", "decode_paged_workspace_size",
                "cache_append_paged", "cache_append_paged_fp8", "verify_drafts")]
            _CALL.bind(*addresses)
        _CALL_LIB = L
    return _CALL


def load(path):
    """Load one build of the library (the product build, or a test build such as the one
    with a short wait limit) and declare the argument types of every entry point."""
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m hybrid_sliding_window_sink_b200.build`")
    L = ctypes.CDLL(path)
    P, I, F, LL, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong, ctypes.c_size_t
    SP = ctypes.POINTER(MimoShape)
    L.mimo_attn_prefill.argtypes = [SP, P, P, P, P, I, F, I, P, P, P]
    L.mimo_attn_decode.argtypes = [SP, P, P, P, I, I, LL, P, P, P, P, P, SZ, P]
    L.mimo_attn_sparse.argtypes = [SP, P, P, P, I, LL, P, I, P, I, P, P, P, P, SZ, P]
    L.mimo_attn_sparse_noalloc.argtypes = [SP, P, P, P, I, LL, P, I, P, I, P, P, P, P]
    L.mimo_attn_decode_mq.argtypes = [SP, P, P, P, I, I, LL, P, I, I, P, P, P, P, SZ, P]
    L.mimo_attn_decode_mq_workspace_size.argtypes = [SP, I, I, I, I]
    L.mimo_attn_decode_mq_workspace_size.restype = SZ
    L.mimo_attn_prefill_chunk.argtypes = [SP, P, P, P, I, I, P, I, F, I, P, P, P]
    L.mimo_attn_cache_append.argtypes = [SP, P, P, I, F, I, I, P, P, I, LL, P]
    L.mimo_attn_select_tokens.argtypes = [SP, P, P, I, LL, P, I, I, P, P, SZ, P]
    L.mimo_attn_select_workspace_size.argtypes = [SP, I]
    L.mimo_attn_select_workspace_size.restype = SZ
    L.mimo_attn_decode_fp8.argtypes = [SP, P, P, P, P, P, I, I, LL, P, P, P, P, P, SZ, P]
    L.mimo_attn_sparse_fp8.argtypes = [SP, P, P, P, P, P, I, LL, P, I, P, I, P, P, P, P, SZ, P]
    L.mimo_attn_prefill_first.argtypes = [SP, P, P, P, I, I, P, I, I, F, I, P, P, P]
    PP = ctypes.POINTER(MimoPages)
    L.mimo_attn_decode_paged.argtypes = [SP, P, P, P, PP, P, I, I, P, P, P, P, SZ, P]
    L.mimo_attn_decode_paged_fp8.argtypes = [SP, P, P, P, P, P, PP, P, I, I, P, P, P, P, SZ, P]
    L.mimo_attn_decode_paged_workspace_size.argtypes = [SP, PP, I, I]
    L.mimo_attn_decode_paged_workspace_size.restype = SZ
    L.mimo_attn_cache_append_paged.argtypes = [SP, P, P, P, P, F, I, PP, P, P, P]
    L.mimo_attn_cache_append_paged_fp8.argtypes = [SP, P, P, P, P, F, I, PP, P, P, P, P, P]
    L.mimo_attn_verify_drafts.argtypes = [I, I, I, I, P, P, P, P, P, P, P, P]
    L.mimo_attn_workspace_size.argtypes = [SP, I, I, I, I, I]
    L.mimo_attn_workspace_size.restype = SZ
    L.mimo_attn_check_indices.argtypes = [SP, P, P, I, I, I, P, P]
    L.mimo_attn_last_device_error.argtypes = []
    L.mimo_attn_last_device_error.restype = ctypes.c_uint
    L.mimo_attn_device_status.argtypes = [P]
    L.mimo_attn_device_status.restype = I
    L.mimo_status_string.argtypes = [I]
    L.mimo_status_string.restype = ctypes.c_char_p
    L.mimo_attn_version.argtypes = []
    L.mimo_attn_version.restype = I
    for fn in ("mimo_attn_prefill", "mimo_attn_decode", "mimo_attn_sparse", "mimo_attn_sparse_noalloc",
               "mimo_attn_check_indices"):
        getattr(L, fn).restype = I
    return L


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _addr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn, status):
    if status != 0:
        raise MimoError(fn, status, _LIB)


def _need(t, name, dtype, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def make_shape(batch, seqlen, hq, hkv, dqk=192, dv=128, softmax_scale=0.0):
    return MimoShape(int(batch), int(seqlen), int(hq), int(hkv), int(dqk), int(dv),
                     float(softmax_scale))


def prefill(q, k, v, sink=None, *, window=128, rope_theta=1.0e4, rot_dims=64,
            softmax_scale=0.0, out=None, lse=None, want_lse=True, stream=None):
    """mimo_attn_prefill. q [B,n,Hq,192], k [B,n,Hkv,192], v [B,n,Hkv,128] bf16,
    sink [Hq] fp32 or None. Returns (out [B,n,Hq,128] bf16, lse [B,Hq,n] fp32 or None)."""
    _need(q, "q", torch.bfloat16, 4)
    _need(k, "k", torch.bfloat16, 4)
    _need(v, "v", torch.bfloat16, 4)
    B, n, hq, dqk = q.shape
    hkv = k.shape[2]
    if k.shape[:2] != (B, n) or v.shape[:3] != (B, n, hkv):
        raise ValueError("q, k, v batch / sequence / head shapes disagree")
    if sink is not None:
        _need(sink, "sink", torch.float32, 1)
        if sink.shape[0] != hq:
            raise ValueError("sink must have Hq entries")
    if out is None:
        out = torch.empty(B, n, hq, v.shape[3], dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, 4)
    if lse is None and want_lse:
        lse = torch.empty(B, hq, n, dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 3)
    shape = make_shape(B, n, hq, hkv, dqk, v.shape[3], softmax_scale)
    st = lib().mimo_attn_prefill(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(sink),
                                 int(window), float(rope_theta), int(rot_dims), _ptr(out),
                                 _ptr(lse), _stream(stream))
    _check("mimo_attn_prefill", st)
    return out, lse


def workspace_size(batch, hq, hkv, *, op, kind=MIMO_CACHE_LINEAR, capacity=1, recent=0, n_sel=0):
    shape = make_shape(batch, 1, hq, hkv)
    return int(lib().mimo_attn_workspace_size(ctypes.byref(shape), int(op), int(kind),
                                              int(capacity), int(recent), int(n_sel)))


def _workspace(ws, nbytes, device):
    if nbytes == 0:
        return ws
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if ws.numel() * ws.element_size() < nbytes:
        raise ValueError("workspace too small")
    return ws


def decode(q, k_cache, v_cache, lengths, sink=None, *, kind="ring", capacity=None,
           softmax_scale=0.0, out=None, lse=None, want_lse=True, workspace=None, stream=None):
    """mimo_attn_decode. q [B,Hq,192]; caches [B,stride,Hkv,192/128] bf16 (rotated K);
    lengths [B] int32. kind "ring" (slot p mod capacity) or "linear"."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(lengths, "lengths", torch.int32, 1)
    B, hq, dqk = q.shape
    _, stride, hkv, _ = k_cache.shape
    if v_cache.shape[:3] != (B, stride, hkv) or k_cache.shape[0] != B or lengths.shape[0] != B:
        raise ValueError("cache / lengths shapes disagree with q")
    cap = stride if capacity is None else int(capacity)
    kind_id = {"ring": MIMO_CACHE_RING, "linear": MIMO_CACHE_LINEAR}[kind]
    if sink is not None:
        _need(sink, "sink", torch.float32, 1)
    if out is None:
        out = torch.empty(B, hq, v_cache.shape[3], dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(B, hq, dtype=torch.float32, device=q.device)
    shape = make_shape(B, 1, hq, hkv, dqk, v_cache.shape[3], softmax_scale)
    nbytes = int(lib().mimo_attn_workspace_size(ctypes.byref(shape), MIMO_OP_DECODE, kind_id, cap, 0, 0))
    ws = _workspace(workspace, nbytes, q.device)
    st = lib().mimo_attn_decode(ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache), kind_id,
                                cap, stride, _ptr(lengths), _ptr(sink), _ptr(out), _ptr(lse),
                                _ptr(ws), nbytes, _stream(stream))
    _check("mimo_attn_decode", st)
    return out, lse


def prefill_chunk(q, k, v, sink=None, *, pos_offset, k_prefix_rotated=True, window=0,
                  rope_theta=1e4, rot_dims=64, softmax_scale=0.0, out=None, lse=None,
                  want_lse=True, stream=None):
    """mimo_attn_prefill_chunk. q [B,n,Hq,192] (the chunk); k, v [B,pos_offset+n,Hkv,·] (every
    key position; prefix K rotated when k_prefix_rotated). Returns (out [B,n,Hq,128],
    lse [B,Hq,n])."""
    _need(q, "q", torch.bfloat16, 4)
    _need(k, "k", torch.bfloat16, 4)
    _need(v, "v", torch.bfloat16, 4)
    B, n, hq, dqk = q.shape
    _, nk, hkv, _ = k.shape
    if nk != pos_offset + n or v.shape[:3] != (B, nk, hkv):
        raise ValueError("k / v must hold positions 0 .. pos_offset + n - 1")
    if sink is not None:
        _need(sink, "sink", torch.float32, 1)
    if out is None:
        out = torch.empty(B, n, hq, v.shape[3], dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(B, hq, n, dtype=torch.float32, device=q.device)
    shape = make_shape(B, n, hq, hkv, dqk, v.shape[3], softmax_scale)
    st = lib().mimo_attn_prefill_chunk(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), int(pos_offset),
                                       1 if k_prefix_rotated else 0, _ptr(sink), int(window),
                                       float(rope_theta), int(rot_dims), _ptr(out), _ptr(lse),
                                       _stream(stream))
    _check("mimo_attn_prefill_chunk", st)
    return out, lse


def cache_append(k_chunk, v_chunk, k_cache, v_cache, *, pos_offset, rope_theta=1e4, rot_dims=64,
                 kind="ring", capacity=None, stream=None):
    """mimo_attn_cache_append: writes the chunk's rotated K and its V into the caches in place."""
    _need(k_chunk, "k_chunk", torch.bfloat16, 4)
    _need(v_chunk, "v_chunk", torch.bfloat16, 4)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    B, n, hkv, dqk = k_chunk.shape
    stride = k_cache.shape[1]
    cap = stride if capacity is None else int(capacity)
    kind_id = {"ring": MIMO_CACHE_RING, "linear": MIMO_CACHE_LINEAR}[kind]
    shape = make_shape(B, n, hkv, hkv, dqk, v_chunk.shape[3])
    st = lib().mimo_attn_cache_append(ctypes.byref(shape), _ptr(k_chunk), _ptr(v_chunk), int(pos_offset),
                                      float(rope_theta), int(rot_dims), kind_id, _ptr(k_cache),
                                      _ptr(v_cache), cap, stride, _stream(stream))
    _check("mimo_attn_cache_append", st)
    return k_cache, v_cache


def select_tokens(q, k_cache, lengths, *, recent=128, n_sel=1024, capacity=None, out=None,
                  workspace=None, stream=None):
    """mimo_attn_select_tokens. q [B,Hq,192]; linear k_cache [B,stride,Hkv,192] (rotated K);
    lengths [B] int32. Returns sel_idx [B,Hkv,n_sel] int32 (sorted, as sparse() reads it)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(lengths, "lengths", torch.int32, 1)
    B, hq, dqk = q.shape
    _, stride, hkv, _ = k_cache.shape
    cap = stride if capacity is None else int(capacity)
    if out is None:
        out = torch.empty(B, hkv, n_sel, dtype=torch.int32, device=q.device)
    shape = make_shape(B, 1, hq, hkv, dqk)
    nbytes = int(lib().mimo_attn_select_workspace_size(ctypes.byref(shape), cap))
    ws = _workspace(workspace, nbytes, q.device)
    st = lib().mimo_attn_select_tokens(ctypes.byref(shape), _ptr(q), _ptr(k_cache), cap, stride,
                                       _ptr(lengths), int(recent), int(n_sel), _ptr(out), _ptr(ws),
                                       nbytes, _stream(stream))
    _check("mimo_attn_select_tokens", st)
    return out


def decode_mq(q, k_cache, v_cache, lengths, sink=None, *, kind="ring", window=128, capacity=None,
              softmax_scale=0.0, out=None, lse=None, want_lse=True, workspace=None, stream=None):
    """mimo_attn_decode_mq. q [B,T,Hq,192] (the T newest tokens of each sequence, rotated);
    caches [B,stride,Hkv,192/128] bf16 holding them; lengths [B] int32 including them.
    kind "ring" (slot p mod capacity, needs capacity >= window + T - 1) or "linear"."""
    _need(q, "q", torch.bfloat16, 4)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(lengths, "lengths", torch.int32, 1)
    B, T, hq, dqk = q.shape
    _, stride, hkv, _ = k_cache.shape
    if v_cache.shape[:3] != (B, stride, hkv) or k_cache.shape[0] != B or lengths.shape[0] != B:
        raise ValueError("cache / lengths shapes disagree with q")
    cap = stride if capacity is None else int(capacity)
    kind_id = {"ring": MIMO_CACHE_RING, "linear": MIMO_CACHE_LINEAR}[kind]
    if sink is not None:
        _need(sink, "sink", torch.float32, 1)
    if out is None:
        out = torch.empty(B, T, hq, v_cache.shape[3], dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(B, T, hq, dtype=torch.float32, device=q.device)
    shape = make_shape(B, 1, hq, hkv, dqk, v_cache.shape[3], softmax_scale)
    nbytes = int(lib().mimo_attn_decode_mq_workspace_size(ctypes.byref(shape), kind_id, cap, T,
                                                          int(window)))
    ws = _workspace(workspace, nbytes, q.device)
    st = lib().mimo_attn_decode_mq(ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache), kind_id,
                                   cap, stride, _ptr(lengths), T, int(window), _ptr(sink), _ptr(out),
                                   _ptr(lse), _ptr(ws), nbytes, _stream(stream))
    _check("mimo_attn_decode_mq", st)
    return out, lse


def _need_fp8(k8, v8, ks, vs):
    _need(k8, "k_cache", torch.uint8, 4)
    _need(v8, "v_cache", torch.uint8, 4)
    _need(ks, "k_scale", torch.float32, 3)
    _need(vs, "v_scale", torch.float32, 3)
    if ks.shape != k8.shape[:3] or vs.shape != v8.shape[:3] or k8.shape[:3] != v8.shape[:3]:
        raise ValueError("FP8 caches and scales disagree in shape")


def decode_fp8(q, k8, v8, k_scale, v_scale, lengths, sink=None, *, kind="ring", capacity=None,
               softmax_scale=0.0, out=None, lse=None, want_lse=True, workspace=None, stream=None):
    """mimo_attn_decode_fp8. q [B,Hq,192] bf16; k8/v8 [B,stride,Hkv,192/128] uint8 E4M3;
    k_scale/v_scale [B,stride,Hkv] fp32; value = e4m3(byte) * scale."""
    _need(q, "q", torch.bfloat16, 3)
    _need_fp8(k8, v8, k_scale, v_scale)
    _need(lengths, "lengths", torch.int32, 1)
    B, hq, dqk = q.shape
    _, stride, hkv, _ = k8.shape
    cap = stride if capacity is None else int(capacity)
    kind_id = {"ring": MIMO_CACHE_RING, "linear": MIMO_CACHE_LINEAR}[kind]
    if sink is not None:
        _need(sink, "sink", torch.float32, 1)
    if out is None:
        out = torch.empty(B, hq, v8.shape[3], dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(B, hq, dtype=torch.float32, device=q.device)
    shape = make_shape(B, 1, hq, hkv, dqk, v8.shape[3], softmax_scale)
    nbytes = int(lib().mimo_attn_workspace_size(ctypes.byref(shape), MIMO_OP_DECODE, kind_id, cap, 0, 0))
    ws = _workspace(workspace, nbytes, q.device)
    st = lib().mimo_attn_decode_fp8(ctypes.byref(shape), _ptr(q), _ptr(k8), _ptr(v8), _ptr(k_scale),
                                    _ptr(v_scale), kind_id, cap, stride, _ptr(lengths), _ptr(sink),
                                    _ptr(out), _ptr(lse), _ptr(ws), nbytes, _stream(stream))
    _check("mimo_attn_decode_fp8", st)
    return out, lse


def sparse_fp8(q, k8, v8, k_scale, v_scale, lengths, sel_idx, sink=None, *, recent=128,
               capacity=None, softmax_scale=0.0, out=None, lse=None, want_lse=True, workspace=None,
               stream=None):
    """mimo_attn_sparse_fp8: sparse() over FP8 linear caches with per-row scales."""
    _need(q, "q", torch.bfloat16, 3)
    _need_fp8(k8, v8, k_scale, v_scale)
    _need(lengths, "lengths", torch.int32, 1)
    _need(sel_idx, "sel_idx", torch.int32, 3)
    B, hq, dqk = q.shape
    _, stride, hkv, _ = k8.shape
    n_sel = sel_idx.shape[2]
    cap = stride if capacity is None else int(capacity)
    if sink is not None:
        _need(sink, "sink", torch.float32, 1)
    if out is None:
        out = torch.empty(B, hq, v8.shape[3], dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(B, hq, dtype=torch.float32, device=q.device)
    shape = make_shape(B, 1, hq, hkv, dqk, v8.shape[3], softmax_scale)
    nbytes = int(lib().mimo_attn_workspace_size(ctypes.byref(shape), MIMO_OP_SPARSE,
                                                MIMO_CACHE_LINEAR, cap, int(recent), n_sel))
    ws = _workspace(workspace, nbytes, q.device)
    st = lib().mimo_attn_sparse_fp8(ctypes.byref(shape), _ptr(q), _ptr(k8), _ptr(v8), _ptr(k_scale),
                                    _ptr(v_scale), cap, stride, _ptr(lengths), int(recent),
                                    _ptr(sel_idx), n_sel, _ptr(sink), _ptr(out), _ptr(lse), _ptr(ws),
                                    nbytes, _stream(stream))
    _check("mimo_attn_sparse_fp8", st)
    return out, lse


def sparse(q, k_cache, v_cache, lengths, sel_idx, sink=None, *, recent=128, capacity=None,
           softmax_scale=0.0, out=None, lse=None, want_lse=True, workspace=None, stream=None):
    """mimo_attn_sparse. q [B,Hq,192]; linear caches [B,stride,Hkv,·]; lengths [B] int32;
    sel_idx [B,Hkv,n_sel] int32 sorted unique in [0, L-recent)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(lengths, "lengths", torch.int32, 1)
    _need(sel_idx, "sel_idx", torch.int32, 3)
    B, hq, dqk = q.shape
    _, stride, hkv, _ = k_cache.shape
    if sel_idx.shape[:2] != (B, hkv):
        raise ValueError("sel_idx must be [B, Hkv, n_sel]")
    n_sel = sel_idx.shape[2]
    cap = stride if capacity is None else int(capacity)
    if sink is not None:
        _need(sink, "sink", torch.float32, 1)
    if out is None:
        out = torch.empty(B, hq, v_cache.shape[3], dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(B, hq, dtype=torch.float32, device=q.device)
    shape = make_shape(B, 1, hq, hkv, dqk, v_cache.shape[3], softmax_scale)
    nbytes = int(lib().mimo_attn_workspace_size(ctypes.byref(shape), MIMO_OP_SPARSE,
                                                MIMO_CACHE_LINEAR, cap, int(recent), n_sel))
    ws = _workspace(workspace, nbytes, q.device)
    st = lib().mimo_attn_sparse(ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache), cap,
                                stride, _ptr(lengths), int(recent), _ptr(sel_idx), n_sel, _ptr(sink),
                                _ptr(out), _ptr(lse), _ptr(ws), nbytes, _stream(stream))
    _check("mimo_attn_sparse", st)
    return out, lse


_raw_stream = torch._C._cuda_getCurrentRawStream   # of a device index, without a Stream object


class _On:
    """Makes device ``index`` current and yields the raw stream to launch on: the given stream
    (which must belong to that device), or the device's current one. Scratch and outputs
    allocated inside belong to that stream. Not used where the device is current already and no
    stream is given (see _here)."""

    __slots__ = ("ctx", "index")

    def __init__(self, index, stream):
        self.index = index
        if stream is not None and stream.device_index != index:
            raise ValueError(f"stream of device {stream.device_index} for tensors on device {index}")
        self.ctx = torch.cuda.device(index) if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        self.ctx.__enter__()
        return _raw_stream(self.index)

    def __exit__(self, *exc):
        return self.ctx.__exit__(*exc)


def _here(index, stream):
    return stream is None and index == torch.cuda.current_device()


def _need_at(t, name, dtype, shape, device, contiguous=True):
    """t is a tensor of that dtype, shape (None: any size) and device."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device:
        have = t.shape
        if have == shape or _fits(have, shape):
            if not contiguous or t.is_contiguous():
                return
            raise ValueError(f"{name} must be contiguous")
        want = tuple("*" if n is None else n for n in shape)
        raise ValueError(f"{name} must have shape {want}, got {tuple(have)}")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be on {device}, got {t.device}")


def _int(x, name):
    """x as an int that the C ABI can take (ctypes would drop its upper bits)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} = {x} does not fit in 32 bits")
    return x


@functools.lru_cache(maxsize=1024)
def _fits(have, shape):
    return len(have) == len(shape) and all(n is None or n == h for n, h in zip(shape, have))


def _cuda_device(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def prefill_first(q, k, v, sink=None, *, window, n_first, pos_offset=0, k_prefix_rotated=True, rope_theta=1e4,
                  rot_dims=64, softmax_scale=0.0, out=None, lse=None, want_lse=True, stream=None):
    """mimo_attn_prefill_first. q [B,n,Hq,192] at positions pos_offset on; k, v [B,pos_offset+n,Hkv,·]
    (prefix K rotated when k_prefix_rotated). A query sees its last ``window`` tokens and, before
    them, those of the first ``n_first`` (window <= 0: everything up to it). Returns (out [B,n,Hq,128] bf16, lse [B,Hq,n] fp32 or None)."""
    if out is None and lse is None and stream is None and (call := _usual()):
        got = call.prefill_first(q, k, v, sink, window, n_first, pos_offset, k_prefix_rotated, rope_theta, rot_dims,
                                 softmax_scale, want_lse)
        if got is not None:
            return got
    window, n_first = _int(window, "window"), _int(n_first, "n_first")
    pos_offset, rot_dims = _int(pos_offset, "pos_offset"), _int(rot_dims, "rot_dims")
    rope_theta, softmax_scale = float(rope_theta), float(softmax_scale)
    dev = _cuda_device(q, "q")
    _need_at(q, "q", torch.bfloat16, (None, None, None, 192), dev)
    B, n, hq, _ = q.shape
    _need_at(k, "k", torch.bfloat16, (B, pos_offset + n, None, 192), dev)
    hkv = k.shape[2]
    _need_at(v, "v", torch.bfloat16, (B, pos_offset + n, hkv, 128), dev)
    if sink is not None:
        _need_at(sink, "sink", torch.float32, (hq,), dev)
    if out is not None:
        _need_at(out, "out", torch.bfloat16, (B, n, hq, 128), dev)
    if lse is not None:
        _need_at(lse, "lse", torch.float32, (B, hq, n), dev)

    def launch(st):
        o = torch.empty((B, n, hq, 128), dtype=torch.bfloat16, device=dev) if out is None else out
        ls = torch.empty((B, hq, n), dtype=torch.float32, device=dev) if lse is None and want_lse else lse
        _check("mimo_attn_prefill_first", lib().mimo_attn_prefill_first(
            _shape_struct(B, n, hq, hkv, softmax_scale), q.data_ptr(), k.data_ptr(), v.data_ptr(), pos_offset,
            1 if k_prefix_rotated else 0, _addr(sink), window, n_first, rope_theta, rot_dims, o.data_ptr(), _addr(ls), st))
        return o, ls

    if _here(dev.index, stream):
        return launch(_raw_stream(dev.index))
    with _On(dev.index, stream) as st:
        return launch(st)


def _pool_stride(shape, strides, name):
    """Tokens between the pages of a pool [num_pages, page_size, Hkv(, D)] that is contiguous
    within a page."""
    if shape[0] < 1 or shape[1] < 1 or shape[2] < 1:
        raise ValueError("the pool holds no page")
    row = shape[2] * shape[3] if len(shape) == 4 else shape[2]
    inner = (row, shape[3], 1) if len(shape) == 4 else (row, 1)
    if strides[1:] != inner and any(s != w and d > 1 for s, w, d in zip(strides[1:], inner, shape[1:])):
        raise ValueError(f"{name} must be contiguous within a page")
    if shape[0] == 1:
        return shape[1]
    if strides[0] % row or strides[0] < shape[1] * row:
        raise ValueError(f"{name}: pages must not overlap and must lie whole tokens apart")
    return strides[0] // row


@functools.lru_cache(maxsize=1024)
def _pools_stride(kshape, kstrides, *rest):
    """Tokens between pages of pools of these shapes and strides (K, V, scales), the same in all."""
    stride = _pool_stride(kshape, kstrides, "k_pages")
    for name, shape, strides in zip(("v_pages", "k_scale", "v_scale"), rest[::2], rest[1::2]):
        if _pool_stride(shape, strides, name) != stride:
            raise ValueError("K, V and scale pools must have the same distance between pages")
    return stride


def _pages(k, v, table, scales=None):
    """mimo_pages of the pools k [num_pages, page_size, Hkv, 192], v [.., 128] and the scales
    [num_pages, page_size, Hkv]."""
    ks = k.shape
    if scales is None:
        stride = _pools_stride(ks, k.stride(), v.shape, v.stride())
    else:
        a, b = scales
        stride = _pools_stride(ks, k.stride(), v.shape, v.stride(), a.shape, a.stride(), b.shape, b.stride())
    return MimoPages(table.data_ptr(), _int(table.shape[1], "max_pages"), _int(ks[0], "num_pages"),
                     _int(ks[1], "page_size"), stride)


def _need_pools(k, v, scales, hkv, dev):
    """Checks the pools of one call."""
    dt = torch.bfloat16 if scales is None else torch.uint8
    _need_at(k, "k_pages", dt, (None, None, hkv, 192), dev, contiguous=False)
    n, page, hkv, _ = k.shape
    _need_at(v, "v_pages", dt, (n, page, hkv, 128), dev, contiguous=False)
    if scales is not None:
        _need_at(scales[0], "k_scale", torch.float32, (n, page, hkv), dev, contiguous=False)
        _need_at(scales[1], "v_scale", torch.float32, (n, page, hkv), dev, contiguous=False)


@functools.lru_cache(maxsize=1024)
def _shape_struct(batch, seqlen, hq, hkv, softmax_scale):
    """mimo_shape of these sizes (only ever read)."""
    for x, name in ((batch, "batch"), (seqlen, "tokens"), (hq, "query heads"), (hkv, "KV heads")):
        _int(x, name)
    return MimoShape(batch, seqlen, hq, hkv, 192, 128, softmax_scale)


@functools.lru_cache(maxsize=1024)
def _paged_workspace(index, batch, hq, hkv, max_pages, page_size, window, n_first):
    """Workspace bytes by sizes (and the device, which is current)."""
    return int(lib().mimo_attn_decode_paged_workspace_size(
        make_shape(batch, 1, hq, hkv), MimoPages(None, max_pages, 1, page_size, page_size), window, n_first))


def _decode_paged(q, k, v, scales, table, lengths, sink, window, n_first, softmax_scale, out, lse, want_lse,
                  workspace, stream):
    if out is None and lse is None and workspace is None and stream is None and (call := _usual()):
        ks, vs = (None, None) if scales is None else scales
        got = call.decode_paged(q, k, v, ks, vs, table, lengths, sink, window, n_first, softmax_scale, want_lse)
        if got is not None:
            return got
    window, n_first, softmax_scale = _int(window, "window"), _int(n_first, "n_first"), float(softmax_scale)
    dev = _cuda_device(q, "q")
    _need_at(q, "q", torch.bfloat16, (None, None, 192), dev)
    B, hq, _ = q.shape
    _need_pools(k, v, scales, None, dev)
    _need_at(table, "block_table", torch.int32, (B, None), dev)
    _need_at(lengths, "lengths", torch.int32, (B,), dev)
    if sink is not None:
        _need_at(sink, "sink", torch.float32, (hq,), dev)
    if out is not None:
        _need_at(out, "out", torch.bfloat16, (B, hq, 128), dev)
    if lse is not None:
        _need_at(lse, "lse", torch.float32, (B, hq), dev)
    if workspace is not None and (not isinstance(workspace, torch.Tensor) or workspace.device != dev
                                  or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    pages = _pages(k, v, table, scales)
    hkv = k.shape[2]

    def launch(st):
        o = torch.empty((B, hq, 128), dtype=torch.bfloat16, device=dev) if out is None else out
        ls = torch.empty((B, hq), dtype=torch.float32, device=dev) if lse is None and want_lse else lse
        nbytes = _paged_workspace(dev.index, B, hq, hkv, pages.max_pages, pages.page_size, window, n_first)
        ws = _workspace(workspace, nbytes, dev)
        shape = _shape_struct(B, 1, hq, hkv, softmax_scale)
        if scales is None:
            _check("mimo_attn_decode_paged", lib().mimo_attn_decode_paged(
                shape, q.data_ptr(), k.data_ptr(), v.data_ptr(), pages, lengths.data_ptr(), window, n_first,
                _addr(sink), o.data_ptr(), _addr(ls), _addr(ws), nbytes, st))
        else:
            _check("mimo_attn_decode_paged_fp8", lib().mimo_attn_decode_paged_fp8(
                shape, q.data_ptr(), k.data_ptr(), v.data_ptr(), scales[0].data_ptr(), scales[1].data_ptr(), pages,
                lengths.data_ptr(), window, n_first, _addr(sink), o.data_ptr(), _addr(ls), _addr(ws), nbytes, st))
        return o, ls

    if _here(dev.index, stream):
        return launch(_raw_stream(dev.index))
    with _On(dev.index, stream) as st:
        return launch(st)


def decode_paged(q, k_pages, v_pages, block_table, lengths, sink=None, *, window=0, n_first=0, softmax_scale=0.0,
                 out=None, lse=None, want_lse=True, workspace=None, stream=None):
    """mimo_attn_decode_paged. q [B,Hq,192]; k_pages [N,page,Hkv,192], v_pages [N,page,Hkv,128] bf16
    (rotated K; pages may lie further apart than their size); block_table [B,max_pages] and lengths
    [B] int32. The query sees the last ``window`` tokens and the first ``n_first`` ones (window <= 0:
    everything). Returns (out [B,Hq,128] bf16, lse [B,Hq] fp32 or None)."""
    return _decode_paged(q, k_pages, v_pages, None, block_table, lengths, sink, window, n_first, softmax_scale, out,
                         lse, want_lse, workspace, stream)


def decode_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, block_table, lengths, sink=None, *, window=0, n_first=0,
                     softmax_scale=0.0, out=None, lse=None, want_lse=True, workspace=None, stream=None):
    """mimo_attn_decode_paged_fp8: decode_paged() over E4M3 pages (uint8) with k_scale / v_scale
    [N,page,Hkv] fp32."""
    return _decode_paged(q, k_pages, v_pages, (k_scale, v_scale), block_table, lengths, sink, window, n_first,
                         softmax_scale, out, lse, want_lse, workspace, stream)


def decode_paged_workspace_size(batch, hq, hkv, *, max_pages, page_size, window=0, n_first=0):
    """Bytes of workspace the paged decodes need on the current device."""
    return _paged_workspace(torch.cuda.current_device(), _int(batch, "batch"), _int(hq, "hq"), _int(hkv, "hkv"),
                            _int(max_pages, "max_pages"), _int(page_size, "page_size"), _int(window, "window"),
                            _int(n_first, "n_first"))


def _append_paged(k_new, v_new, k, v, scales, table, positions, n_new, rope_theta, rot_dims, stream):
    if stream is None and (call := _usual()):
        ks, vs = (None, None) if scales is None else scales
        if call.append_paged(k_new, v_new, k, v, ks, vs, table, positions, n_new, rope_theta, rot_dims):
            return
    rope_theta, rot_dims = float(rope_theta), _int(rot_dims, "rot_dims")
    dev = _cuda_device(k_new, "k_new")
    _need_at(k_new, "k_new", torch.bfloat16, (None, None, None, 192), dev)
    B, n, hkv, _ = k_new.shape
    _need_at(v_new, "v_new", torch.bfloat16, (B, n, hkv, 128), dev)
    _need_pools(k, v, scales, hkv, dev)
    _need_at(table, "block_table", torch.int32, (B, None), dev)
    _need_at(positions, "positions", torch.int32, (B,), dev)
    if n_new is not None:
        _need_at(n_new, "n_new", torch.int32, (B,), dev)
    pages = _pages(k, v, table, scales)

    def launch(st):
        shape = _shape_struct(B, n, hkv, hkv, 0.0)
        if scales is None:
            _check("mimo_attn_cache_append_paged", lib().mimo_attn_cache_append_paged(
                shape, k_new.data_ptr(), v_new.data_ptr(), positions.data_ptr(), _addr(n_new), rope_theta, rot_dims,
                pages, k.data_ptr(), v.data_ptr(), st))
        else:
            _check("mimo_attn_cache_append_paged_fp8", lib().mimo_attn_cache_append_paged_fp8(
                shape, k_new.data_ptr(), v_new.data_ptr(), positions.data_ptr(), _addr(n_new), rope_theta, rot_dims,
                pages, k.data_ptr(), v.data_ptr(), scales[0].data_ptr(), scales[1].data_ptr(), st))

    if _here(dev.index, stream):
        launch(_raw_stream(dev.index))
    else:
        with _On(dev.index, stream) as st:
            launch(st)


def cache_append_paged(k_new, v_new, k_pages, v_pages, block_table, positions, *, n_new=None, rope_theta=1e4,
                       rot_dims=64, stream=None):
    """mimo_attn_cache_append_paged: writes the new tokens' rotated K [B,n,Hkv,192] and V [B,n,Hkv,128]
    into the pages, in place, from position positions[b] on (n_new [B]: only so many of them)."""
    _append_paged(k_new, v_new, k_pages, v_pages, None, block_table, positions, n_new, rope_theta, rot_dims, stream)
    return k_pages, v_pages


def cache_append_paged_fp8(k_new, v_new, k_pages, v_pages, k_scale, v_scale, block_table, positions, *, n_new=None,
                           rope_theta=1e4, rot_dims=64, stream=None):
    """mimo_attn_cache_append_paged_fp8: as cache_append_paged(), into E4M3 pages (uint8) and their
    scales [N,page,Hkv] fp32."""
    _append_paged(k_new, v_new, k_pages, v_pages, (k_scale, v_scale), block_table, positions, n_new, rope_theta,
                  rot_dims, stream)
    return k_pages, v_pages, k_scale, v_scale


def verify_drafts(target_probs, draft_tokens, uniforms, draft_probs=None, *, n_valid=None, n_accepted=None,
                  tokens=None, stream=None):
    """mimo_attn_verify_drafts. target_probs [B,T+1,V] fp32 or bf16, draft_tokens [B,T] int32, uniforms
    [B,T+1] fp32, draft_probs [B,T,V] (None: drafts by argmax), n_valid [B] int32 or None. Returns
    (n_accepted [B], tokens [B,T+1]) int32: the accepted drafts, the next token, then -1."""
    if n_accepted is None and tokens is None and stream is None and (call := _usual()):
        got = call.verify_drafts(target_probs, draft_tokens, uniforms, draft_probs, n_valid)
        if got is not None:
            return got
    dev = _cuda_device(target_probs, "target_probs")
    if target_probs.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"target_probs must be float32 or bfloat16, got {target_probs.dtype}")
    _need_at(target_probs, "target_probs", target_probs.dtype, (None, None, None), dev)
    B, T1, V = target_probs.shape
    T = T1 - 1
    if T < 0:
        raise ValueError("target_probs must have T + 1 rows per sequence")
    for x, name in ((B, "batch"), (T, "drafts"), (V, "vocabulary")):
        _int(x, name)
    _need_at(draft_tokens, "draft_tokens", torch.int32, (B, T), dev)
    _need_at(uniforms, "uniforms", torch.float32, (B, T1), dev)
    if draft_probs is not None:
        _need_at(draft_probs, "draft_probs", target_probs.dtype, (B, T, V), dev)
    if n_valid is not None:
        _need_at(n_valid, "n_valid", torch.int32, (B,), dev)
    if n_accepted is not None:
        _need_at(n_accepted, "n_accepted", torch.int32, (B,), dev)
    if tokens is not None:
        _need_at(tokens, "tokens", torch.int32, (B, T1), dev)

    def launch(st):
        acc = torch.empty((B,), dtype=torch.int32, device=dev) if n_accepted is None else n_accepted
        tok = torch.empty((B, T1), dtype=torch.int32, device=dev) if tokens is None else tokens
        _check("mimo_attn_verify_drafts", lib().mimo_attn_verify_drafts(
            B, T, V, 0 if target_probs.dtype == torch.float32 else 1, target_probs.data_ptr(), _addr(draft_probs),
            draft_tokens.data_ptr(), uniforms.data_ptr(), _addr(n_valid), acc.data_ptr(), tok.data_ptr(), st))
        return acc, tok

    if _here(dev.index, stream):
        return launch(_raw_stream(dev.index))
    with _On(dev.index, stream) as st:
        return launch(st)


def check_indices(lengths, sel_idx, *, hq, recent=128, capacity, stream=None):
    """mimo_attn_check_indices: number of (b, g) rows violating the sparse preconditions."""
    _need(lengths, "lengths", torch.int32, 1)
    _need(sel_idx, "sel_idx", torch.int32, 3)
    B, hkv, n_sel = sel_idx.shape
    shape = make_shape(B, 1, hq, hkv)
    cnt = torch.zeros(1, dtype=torch.int32, device=lengths.device)
    st = lib().mimo_attn_check_indices(ctypes.byref(shape), _ptr(lengths), _ptr(sel_idx), n_sel,
                                       int(recent), int(capacity), _ptr(cnt), _stream(stream))
    _check("mimo_attn_check_indices", st)
    return int(cnt.item())


def last_device_error():
    return int(lib().mimo_attn_last_device_error())
