"""ctypes binding of libspecverify (include/specverify.h).

Argument marshalling only: tensors become device pointers, the current torch
stream becomes the cudaStream_t.  Every step of the verification runs in the
library's CUDA kernels; there is no CPU fallback, and every call raises when
the library is missing or returns an error status.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

from ._build import LIBRARY

SV_OK, SV_EINVAL, SV_ECUDA, SV_ETIMEOUT, SV_EDATA, SV_EWORKSPACE, SV_EUNSUPPORTED, SV_ECORESIDENT = range(8)
SV_BF16, SV_FP32, SV_FP16 = 0, 1, 2
SV_TREE_MSS, SV_TREE_MSS_NOREPLACE, SV_TREE_NAIVE = 0, 1, 2
TREE_MODES = {"mss": SV_TREE_MSS, "noreplace": SV_TREE_MSS_NOREPLACE, "naive": SV_TREE_NAIVE}
SV_DERR_TOKEN, SV_DERR_NONFINITE, SV_DERR_MASS = 0x01, 0x02, 0x04
SV_DERR_TREE, SV_DERR_TIMEOUT, SV_DERR_ARG = 0x08, 0x10, 0x20
SV_DERR_CHECK = 0x40
SV_DERR_PAGE = 0x80
SV_MAX_K, SV_MAX_B, SV_MAX_V, SV_MAX_TOPK = 32, 1024, 1 << 20, 64
SV_MAX_TREE_NODES, SV_MAX_TREE_B = 64, 1024
SV_MAX_KV_T, SV_MAX_KV_HEADS = 65536, 256
SV_MAX_ROTATE_D, SV_MAX_GIVEN = 256, 1024

# every symbol include/specverify.h declares
EXPORTS = ("sv_chain_workspace_bytes", "sv_tree_workspace_bytes", "sv_workspace_init",
           "sv_verify_chain", "sv_verify_tree", "sv_get_error", "sv_selftest_wait_timeout",
           "sv_verify_chain_noalloc", "sv_noalloc_get_error", "sv_tree_mask", "sv_row_stats",
           "sv_kv_write", "sv_kv_read", "sv_kv_attention_workspace_bytes", "sv_kv_attention",
           "sv_stream_capture_id", "sv_rotate", "sv_kv_append", "sv_token_logprobs",
           "sv_status_string", "sv_version")
SV_MIN_WORKSPACE_BYTES = 8192
SV_NOALLOC_SCRATCH_BYTES = 8 << 20

_P = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64


class SvChainArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("K", _i32), ("V", _i32), ("dtype", _i32),
                ("target_logits", _P), ("target_row_stride", _i64),
                ("draft_logits", _P), ("draft_row_stride", _i64),
                ("draft_tokens", _P), ("num_drafts", _P), ("temperature", _P),
                ("top_k", _P), ("max_top_k", _i32), ("uniforms", _P),
                ("out_tokens", _P), ("out_len", _P), ("accept_len", _P),
                ("p_at_draft", _P), ("q_at_draft", _P)]


class SvTreeArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("N", _i32), ("M", _i32), ("V", _i32), ("max_depth", _i32),
                ("dtype", _i32), ("mode", _i32),
                ("target_logits", _P), ("target_row_stride", _i64),
                ("draft_logits", _P), ("draft_row_stride", _i64),
                ("node_tokens", _P), ("parent", _P), ("q_row", _P), ("num_nodes", _P),
                ("temperature", _P), ("top_k", _P), ("max_top_k", _i32),
                ("u_accept", _P), ("u_sample", _P), ("out_tokens", _P), ("out_len", _P),
                ("accept_len", _P), ("accepted_nodes", _P)]


class SvTreeMaskArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("N", _i32), ("words", _i32), ("parent", _P), ("num_nodes", _P),
                ("mask", _P), ("depth", _P)]


class SvKvCache(ctypes.Structure):
    _fields_ = [("num_pages", _i32), ("page_size", _i32), ("Hkv", _i32), ("D", _i32),
                ("k", _P), ("v", _P), ("page_stride", _i64), ("head_stride", _i64),
                ("k_scale", _P), ("v_scale", _P), ("page_table", _P), ("slots", _i32)]


class SvKvWriteArgs(ctypes.Structure):
    _fields_ = [("cache", SvKvCache), ("B", _i32), ("T", _i32), ("dtype", _i32),
                ("k_new", _P), ("v_new", _P),
                ("k_batch_stride", _i64), ("k_token_stride", _i64), ("k_head_stride", _i64),
                ("v_batch_stride", _i64), ("v_token_stride", _i64), ("v_head_stride", _i64),
                ("kv_len", _P), ("num_new", _P)]


class SvKvReadArgs(ctypes.Structure):
    _fields_ = [("cache", SvKvCache), ("B", _i32), ("T", _i32), ("dtype", _i32),
                ("k_out", _P), ("v_out", _P),
                ("out_batch_stride", _i64), ("out_token_stride", _i64), ("out_head_stride", _i64),
                ("start", _P), ("num", _P), ("rows", _P)]


class SvKvAttentionArgs(ctypes.Structure):
    _fields_ = [("cache", SvKvCache), ("B", _i32), ("T", _i32), ("Hq", _i32), ("dtype", _i32),
                ("q", _P), ("q_batch_stride", _i64), ("q_token_stride", _i64),
                ("q_head_stride", _i64), ("out", _P), ("lse", _P), ("kv_len", _P),
                ("num_new", _P), ("mask", _P), ("words", _i32), ("scale", ctypes.c_float)]


# (the structures of the round's calls, for calling the C ABI by hand: the functions below
# are given theirs by the compiled binding)
class SvRope(ctypes.Structure):
    _fields_ = [("dim", _i32), ("interleaved", _i32), ("scale", ctypes.c_float), ("freq", _P)]


class SvHeadNorm(ctypes.Structure):
    _fields_ = [("weight", _P), ("weight_dtype", _i32), ("eps", ctypes.c_float)]


class SvHeads(ctypes.Structure):
    _fields_ = [("x", _P), ("out", _P), ("heads", _i32), ("out_dtype", _i32),
                ("batch_stride", _i64), ("token_stride", _i64), ("head_stride", _i64),
                ("out_batch_stride", _i64), ("out_token_stride", _i64), ("out_head_stride", _i64),
                ("norm", SvHeadNorm)]


class SvRotateArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("T", _i32), ("D", _i32), ("dtype", _i32), ("q", SvHeads),
                ("k", SvHeads), ("start", _P), ("num", _P), ("offset", _P), ("rope", SvRope)]


class SvKvAppendArgs(ctypes.Structure):
    _fields_ = [("cache", SvKvCache), ("B", _i32), ("T", _i32), ("dtype", _i32), ("q", SvHeads),
                ("k_new", _P), ("v_new", _P),
                ("k_batch_stride", _i64), ("k_token_stride", _i64), ("k_head_stride", _i64),
                ("v_batch_stride", _i64), ("v_token_stride", _i64), ("v_head_stride", _i64),
                ("k_norm", SvHeadNorm), ("kv_len", _P), ("num_new", _P), ("offset", _P),
                ("rope", SvRope)]


class SvTokenLogprobsArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("N", _i32), ("R", _i32), ("M", _i32), ("V", _i32), ("dtype", _i32),
                ("logits", _P), ("batch_stride", _i64), ("row_stride", _i64), ("tokens", _P),
                ("num_rows", _P), ("rows", _P), ("temperature", _P), ("top", _i32),
                ("logprob", _P), ("entropy", _P), ("top_token", _P), ("top_logprob", _P)]


class SpecVerifyError(RuntimeError):
    def __init__(self, status: int, what: str = "", flags: int = 0):
        self.status = status
        self.flags = flags
        msg = sv_status_string(status) if _lib_or_none() else f"status {status}"
        super().__init__(f"{what}: {msg}" + (f" (device flags 0x{flags:x})" if flags else ""))


_lib_handle = None


def _lib_or_none():
    return _lib_handle


def lib(path: str | None = None):
    """Load libspecverify.so.  Raises if it has not been built."""
    global _lib_handle
    if _lib_handle is not None and path is None:
        return _lib_handle
    p = path or LIBRARY
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with __graft_entry__.build() "
                           "(nvcc, sm_103a); there is no CPU fallback")
    h = ctypes.CDLL(p)
    h.sv_chain_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32]
    h.sv_chain_workspace_bytes.restype = ctypes.c_size_t
    h.sv_tree_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
    h.sv_tree_workspace_bytes.restype = ctypes.c_size_t
    h.sv_workspace_init.argtypes = [_P, ctypes.c_size_t, _P]
    h.sv_workspace_init.restype = ctypes.c_int
    h.sv_verify_chain.argtypes = [ctypes.POINTER(SvChainArgs), _P, ctypes.c_size_t, _P]
    h.sv_verify_chain.restype = ctypes.c_int
    h.sv_verify_tree.argtypes = [ctypes.POINTER(SvTreeArgs), _P, ctypes.c_size_t, _P]
    h.sv_verify_tree.restype = ctypes.c_int
    h.sv_get_error.argtypes = [_P, _P, ctypes.POINTER(_i32)]
    h.sv_get_error.restype = ctypes.c_int
    h.sv_selftest_wait_timeout.argtypes = [_P, ctypes.c_size_t, _i64, _P]
    h.sv_selftest_wait_timeout.restype = ctypes.c_int
    h.sv_verify_chain_noalloc.argtypes = [ctypes.POINTER(SvChainArgs), _P]
    h.sv_verify_chain_noalloc.restype = ctypes.c_int
    h.sv_noalloc_get_error.argtypes = [_P, ctypes.POINTER(_i32)]
    h.sv_noalloc_get_error.restype = ctypes.c_int
    h.sv_tree_mask.argtypes = [ctypes.POINTER(SvTreeMaskArgs), _P, ctypes.c_size_t, _P]
    h.sv_tree_mask.restype = ctypes.c_int
    h.sv_row_stats.argtypes = [ctypes.POINTER(SvChainArgs), _P, _P, _P, ctypes.c_size_t, _P]
    h.sv_row_stats.restype = ctypes.c_int
    for f in ("sv_kv_write", "sv_kv_read", "sv_kv_attention", "sv_rotate", "sv_kv_append",
              "sv_token_logprobs"):
        getattr(h, f).argtypes = [_P, _P, ctypes.c_size_t, _P]  # the arguments come packed
        getattr(h, f).restype = ctypes.c_int
    h.sv_kv_attention_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32]
    h.sv_kv_attention_workspace_bytes.restype = ctypes.c_size_t
    h.sv_stream_capture_id.argtypes = [_P, ctypes.POINTER(ctypes.c_uint64)]
    h.sv_stream_capture_id.restype = ctypes.c_int
    h.sv_status_string.argtypes = [ctypes.c_int]
    h.sv_status_string.restype = ctypes.c_char_p
    h.sv_version.argtypes = []
    h.sv_version.restype = _i32
    if path is None:
        _lib_handle = h
    return h


# ---------------------------------------------------------------- marshalling

def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libspecverify takes device tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dtype_code(t) -> int:
    if t.dtype == torch.bfloat16:
        return SV_BF16
    if t.dtype == torch.float32:
        return SV_FP32
    raise ValueError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _row_stride(t, rows_per_req: int) -> int:
    """Element stride between consecutive rows of a [B][R][V] tensor whose
    rows are evenly spaced."""
    if t.stride(-1) != 1:
        raise ValueError("logit rows must be contiguous")
    if t.shape[0] > 1 and rows_per_req > 0 and t.stride(0) != rows_per_req * t.stride(1):
        raise ValueError("logit rows must be evenly spaced across requests")
    return t.stride(1)


def _check(t, dtype, shape, what):
    if t is None:
        return
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{what}: expected contiguous {dtype} {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")


def sv_status_string(status: int) -> str:
    return lib().sv_status_string(int(status)).decode()


def sv_version() -> int:
    return lib().sv_version()


def sv_chain_workspace_bytes(B: int, K: int, V: int, dtype: int, max_top_k: int = 0) -> int:
    return lib().sv_chain_workspace_bytes(B, K, V, dtype, max_top_k)


def sv_tree_workspace_bytes(B: int, N: int, M: int, V: int, dtype: int,
                            max_top_k: int = 0) -> int:
    return lib().sv_tree_workspace_bytes(B, N, M, V, dtype, max_top_k)


def sv_workspace_init(workspace: torch.Tensor, stream=None) -> None:
    st = lib().sv_workspace_init(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "sv_workspace_init")


# The current device, and the handle of a device's current stream (without a
# Stream object around it).
_current_device = torch._C._cuda_getDevice
current_raw_stream = torch._C._cuda_getCurrentRawStream


def sv_stream_capture_id(stream) -> int:
    """The id of the capture that a stream is part of, 0 outside captures."""
    out = ctypes.c_uint64(0)
    st = lib().sv_stream_capture_id(_stream(stream), ctypes.byref(out))
    if st != SV_OK:
        raise SpecVerifyError(st, "sv_stream_capture_id")
    return out.value


def sv_verify_chain(target_logits, draft_logits, draft_tokens, temperature, uniforms,
                    out_tokens, out_len, accept_len, workspace, num_drafts=None, top_k=None,
                    max_top_k: int = 0, p_at_draft=None, q_at_draft=None, stream=None) -> None:
    """Enqueue sv_verify_chain on the current (or given) stream."""
    B, K1, V = target_logits.shape
    K = K1 - 1
    a = SvChainArgs()
    a.B, a.K, a.V = B, K, V
    a.dtype = _dtype_code(target_logits)
    a.target_logits = _ptr(target_logits)
    a.target_row_stride = _row_stride(target_logits, K1)
    if draft_logits is not None:
        if draft_logits.dtype != target_logits.dtype or tuple(draft_logits.shape) != (B, K, V):
            raise ValueError("draft_logits must be [B][K][V] of the target's dtype")
        if draft_logits.numel() > 0:
            a.draft_logits = _ptr(draft_logits)
            a.draft_row_stride = _row_stride(draft_logits, K)
    _check(draft_tokens, torch.int32, (B, K), "draft_tokens")
    if draft_tokens is not None and draft_tokens.numel() == 0:
        draft_tokens = None
    _check(temperature, torch.float32, (B,), "temperature")
    _check(uniforms, torch.float32, (B, K + 1), "uniforms")
    _check(num_drafts, torch.int32, (B,), "num_drafts")
    _check(top_k, torch.int32, (B,), "top_k")
    _check(out_tokens, torch.int32, (B, K + 1), "out_tokens")
    _check(out_len, torch.int32, (B,), "out_len")
    _check(accept_len, torch.int32, (B,), "accept_len")
    _check(p_at_draft, torch.float32, (B, K), "p_at_draft")
    _check(q_at_draft, torch.float32, (B, K), "q_at_draft")
    a.draft_tokens = _ptr(draft_tokens)
    a.num_drafts = _ptr(num_drafts)
    a.temperature = _ptr(temperature)
    a.top_k = _ptr(top_k)
    a.max_top_k = max_top_k
    a.uniforms = _ptr(uniforms)
    a.out_tokens = _ptr(out_tokens)
    a.out_len = _ptr(out_len)
    a.accept_len = _ptr(accept_len)
    a.p_at_draft = _ptr(p_at_draft)
    a.q_at_draft = _ptr(q_at_draft)
    st = lib().sv_verify_chain(ctypes.byref(a), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "sv_verify_chain")


def sv_verify_tree(target_logits, draft_logits, node_tokens, parent, q_row, temperature,
                   u_accept, u_sample, out_tokens, out_len, accept_len, accepted_nodes,
                   workspace, max_depth: int, num_nodes=None, top_k=None, max_top_k: int = 0,
                   mode: int = SV_TREE_MSS, stream=None) -> None:
    """Enqueue sv_verify_tree on the current (or given) stream."""
    B, N, V = target_logits.shape
    a = SvTreeArgs()
    a.B, a.N, a.V, a.max_depth = B, N, V, max_depth
    a.M = draft_logits.shape[1] if draft_logits is not None else 1
    a.dtype = _dtype_code(target_logits)
    a.mode = mode
    a.target_logits = _ptr(target_logits)
    a.target_row_stride = _row_stride(target_logits, N)
    if draft_logits is not None:
        if draft_logits.dtype != target_logits.dtype or draft_logits.shape[0] != B \
                or draft_logits.shape[2] != V:
            raise ValueError("draft_logits must be [B][M][V] of the target's dtype")
        a.draft_logits = _ptr(draft_logits)
        a.draft_row_stride = _row_stride(draft_logits, a.M)
    for t, dt, shp, nm in [(node_tokens, torch.int32, (B, N), "node_tokens"),
                           (parent, torch.int32, (B, N), "parent"),
                           (q_row, torch.int32, (B, N), "q_row"),
                           (temperature, torch.float32, (B,), "temperature"),
                           (u_accept, torch.float32, (B, N), "u_accept"),
                           (u_sample, torch.float32, (B,), "u_sample"),
                           (num_nodes, torch.int32, (B,), "num_nodes"),
                           (top_k, torch.int32, (B,), "top_k"),
                           (out_tokens, torch.int32, (B, max_depth + 1), "out_tokens"),
                           (out_len, torch.int32, (B,), "out_len"),
                           (accept_len, torch.int32, (B,), "accept_len")]:
        _check(t, dt, shp, nm)
    if accepted_nodes.dtype != torch.int32 or accepted_nodes.shape[0] != B \
            or accepted_nodes.numel() < B * max_depth:
        raise ValueError("accepted_nodes: expected int32 [B][max_depth]")
    a.node_tokens, a.parent, a.q_row = _ptr(node_tokens), _ptr(parent), _ptr(q_row)
    a.num_nodes, a.temperature, a.top_k = _ptr(num_nodes), _ptr(temperature), _ptr(top_k)
    a.max_top_k = max_top_k
    a.u_accept, a.u_sample = _ptr(u_accept), _ptr(u_sample)
    a.out_tokens, a.out_len, a.accept_len = _ptr(out_tokens), _ptr(out_len), _ptr(accept_len)
    a.accepted_nodes = _ptr(accepted_nodes)
    st = lib().sv_verify_tree(ctypes.byref(a), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "sv_verify_tree")


def sv_get_error(workspace, stream=None) -> tuple[int, int]:
    """(status, device flags); synchronises the stream and clears the word."""
    flags = _i32(0)
    st = lib().sv_get_error(_ptr(workspace), _stream(stream), ctypes.byref(flags))
    return st, flags.value


def sv_selftest_wait_timeout(workspace, limit_ns: int, stream=None) -> int:
    return lib().sv_selftest_wait_timeout(_ptr(workspace),
                                          workspace.numel() * workspace.element_size(),
                                          int(limit_ns), _stream(stream))


# ------------------------------------------------ allocation-free chain call

def sv_verify_chain_noalloc(target_logits, draft_logits, draft_tokens, temperature, uniforms,
                            out_tokens, out_len, accept_len, num_drafts=None, top_k=None,
                            max_top_k: int = 0, p_at_draft=None, q_at_draft=None,
                            stream=None) -> None:
    """Enqueue sv_verify_chain_noalloc: the chain verification with the
    library's own per-device scratch (no workspace argument)."""
    B, K1, V = target_logits.shape
    K = K1 - 1
    a = SvChainArgs()
    a.B, a.K, a.V = B, K, V
    a.dtype = _dtype_code(target_logits)
    a.target_logits = _ptr(target_logits)
    a.target_row_stride = _row_stride(target_logits, K1)
    if draft_logits is not None:
        if draft_logits.dtype != target_logits.dtype or tuple(draft_logits.shape) != (B, K, V):
            raise ValueError("draft_logits must be [B][K][V] of the target's dtype")
        if draft_logits.numel() > 0:
            a.draft_logits = _ptr(draft_logits)
            a.draft_row_stride = _row_stride(draft_logits, K)
    if draft_tokens is not None and draft_tokens.numel() == 0:
        draft_tokens = None
    for t, dt, shp, nm in [(draft_tokens, torch.int32, (B, K), "draft_tokens"),
                           (temperature, torch.float32, (B,), "temperature"),
                           (uniforms, torch.float32, (B, K + 1), "uniforms"),
                           (num_drafts, torch.int32, (B,), "num_drafts"),
                           (top_k, torch.int32, (B,), "top_k"),
                           (out_tokens, torch.int32, (B, K + 1), "out_tokens"),
                           (out_len, torch.int32, (B,), "out_len"),
                           (accept_len, torch.int32, (B,), "accept_len"),
                           (p_at_draft, torch.float32, (B, K), "p_at_draft"),
                           (q_at_draft, torch.float32, (B, K), "q_at_draft")]:
        _check(t, dt, shp, nm)
    a.draft_tokens, a.num_drafts = _ptr(draft_tokens), _ptr(num_drafts)
    a.temperature, a.top_k, a.max_top_k = _ptr(temperature), _ptr(top_k), max_top_k
    a.uniforms = _ptr(uniforms)
    a.out_tokens, a.out_len, a.accept_len = _ptr(out_tokens), _ptr(out_len), _ptr(accept_len)
    a.p_at_draft, a.q_at_draft = _ptr(p_at_draft), _ptr(q_at_draft)
    st = lib().sv_verify_chain_noalloc(ctypes.byref(a), _stream(stream))
    if st == SV_EWORKSPACE:
        need = sv_chain_workspace_bytes(B, K, V, a.dtype, max_top_k)
        raise SpecVerifyError(st, f"sv_verify_chain_noalloc: the call needs {need} bytes of "
                                  f"scratch, more than SV_NOALLOC_SCRATCH_BYTES "
                                  f"({SV_NOALLOC_SCRATCH_BYTES}); use sv_verify_chain with a "
                                  "workspace")
    if st != SV_OK:
        raise SpecVerifyError(st, "sv_verify_chain_noalloc")


def sv_noalloc_get_error(stream=None) -> tuple[int, int]:
    """(status, device flags) of the allocation-free scratch of the current
    device; synchronises the stream; re-zeroes the scratch after an error."""
    flags = _i32(0)
    st = lib().sv_noalloc_get_error(_stream(stream), ctypes.byref(flags))
    return st, flags.value


# ------------------------------------------------- tree mask, row statistics

def sv_tree_mask(parent, mask, depth, workspace, num_nodes=None, stream=None) -> None:
    """Enqueue sv_tree_mask: ancestor bitmask rows mask [B][N][words] (int32
    storage of the uint32 words) and depths [B][N] of DFS-linearised trees."""
    B, N = parent.shape
    if mask.dim() != 3 or tuple(mask.shape[:2]) != (B, N):
        raise ValueError("mask: expected [B][N][words]")
    _check(parent, torch.int32, (B, N), "parent")
    _check(num_nodes, torch.int32, (B,), "num_nodes")
    _check(mask, torch.int32, (B, N, mask.shape[2]), "mask")
    _check(depth, torch.int32, (B, N), "depth")
    a = SvTreeMaskArgs()
    a.B, a.N, a.words = B, N, mask.shape[2]
    a.parent, a.num_nodes = _ptr(parent), _ptr(num_nodes)
    a.mask, a.depth = _ptr(mask), _ptr(depth)
    st = lib().sv_tree_mask(ctypes.byref(a), _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _stream(stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "sv_tree_mask")


def sv_row_stats(target_logits, draft_logits, temperature, alpha, expected, workspace,
                 num_drafts=None, top_k=None, max_top_k: int = 0, stream=None) -> None:
    """Enqueue sv_row_stats: alpha [B][K] = sum min(p_i, q_i) per position
    and expected [B] tokens per round."""
    B, K1, V = target_logits.shape
    K = K1 - 1
    a = SvChainArgs()
    a.B, a.K, a.V = B, K, V
    a.dtype = _dtype_code(target_logits)
    a.target_logits = _ptr(target_logits)
    a.target_row_stride = _row_stride(target_logits, K1)
    if K > 0:
        if draft_logits is None or draft_logits.dtype != target_logits.dtype \
                or tuple(draft_logits.shape) != (B, K, V):
            raise ValueError("draft_logits must be [B][K][V] of the target's dtype")
        a.draft_logits = _ptr(draft_logits)
        a.draft_row_stride = _row_stride(draft_logits, K)
    _check(temperature, torch.float32, (B,), "temperature")
    _check(num_drafts, torch.int32, (B,), "num_drafts")
    _check(top_k, torch.int32, (B,), "top_k")
    _check(alpha, torch.float32, (B, K), "alpha")
    _check(expected, torch.float32, (B,), "expected")
    a.temperature, a.num_drafts, a.top_k = _ptr(temperature), _ptr(num_drafts), _ptr(top_k)
    a.max_top_k = max_top_k
    st = lib().sv_row_stats(ctypes.byref(a), _ptr(alpha), _ptr(expected), _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _stream(stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "sv_row_stats")


# ------------------------------------------------- 8-bit key/value cache
#
# These calls are made once a layer and round, so their marshalling counts:
# the arguments are packed in one go (struct.pack in the C layout of the
# ctypes structures above), and each tensor's facts are read once.

_KV_DTYPES = {torch.bfloat16: SV_BF16, torch.float32: SV_FP32, torch.float16: SV_FP16}
_PACK_CODES = {_i32: "i", _i64: "q", _P: "P", ctypes.c_float: "f"}


def _packer(cls) -> struct.Struct:
    """struct.Struct of a ctypes structure (an embedded one ends on its own
    alignment)."""
    def fmt(c):
        return "".join(fmt(t) + "0q" if issubclass(t, ctypes.Structure) else _PACK_CODES[t]
                       for _, t in c._fields_)
    packer = struct.Struct("@" + fmt(cls) + "0q")
    assert packer.size == ctypes.sizeof(cls)
    return packer


_pack_write, _pack_read = _packer(SvKvWriteArgs).pack, _packer(SvKvReadArgs).pack
_pack_attention = _packer(SvKvAttentionArgs).pack


def _wrong_device(t, dev: int) -> None:
    raise ValueError(f"expected tensors of one device, got one on {t.device} beside a workspace "
                     f"on {'cpu' if dev < 0 else f'cuda:{dev}'}")


def _addr(t, dtype, shape, what: str, dev: int) -> int:
    """Address of a contiguous tensor of the given type, shape and device (0
    for None)."""
    if t is None:
        return 0
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: expected contiguous {dtype} {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != dev:
        _wrong_device(t, dev)
    return t.data_ptr()


def _kv_cache(cache: dict, page_table, B: int, dev: int) -> tuple:
    """The fields of an sv_kv_cache, from the cache's tensors (k, v
    [pages][Hkv][P][D] e4m3, k_scale, v_scale [pages][Hkv] fp32) and the page
    table [B][slots]."""
    k, v = cache["k"], cache["v"]
    shape = k.shape
    if k.dtype != torch.float8_e4m3fn or len(shape) != 4:
        raise ValueError(f"cache k: expected float8_e4m3fn [pages][heads][page][D], got {k.dtype} "
                         f"{tuple(shape)}")
    pages, H, P, D = shape
    if v.dtype != k.dtype or v.shape != shape:
        raise ValueError("cache v: expected k's dtype, shape and strides")
    st, v_st = k.stride(), v.stride()
    if v_st != st:
        # the stride of a dimension of size 1 says nothing
        if any(a != b for a, b, n in zip(st, v_st, shape) if n > 1):
            raise ValueError("cache v: expected k's dtype, shape and strides")
    if st[3] != 1 or st[2] != D:
        raise ValueError("cache: the tokens of a page and head must be contiguous")
    if k.get_device() != dev or v.get_device() != dev:
        _wrong_device(v if k.get_device() == dev else k, dev)
    ks = _addr(cache["k_scale"], torch.float32, (pages, H), "k_scale", dev)
    vs = _addr(cache["v_scale"], torch.float32, (pages, H), "v_scale", dev)
    if page_table.dim() != 2:
        raise ValueError(f"page_table: expected contiguous int32 [{B}][slots]")
    slots = page_table.shape[1]
    table = _addr(page_table, torch.int32, (B, slots), "page_table", dev)
    return (pages, P, H, D, k.data_ptr(), v.data_ptr(), st[0] if pages > 1 else 0,
            st[1] if H > 1 else P * D, ks, vs, table, slots)


def _rows4(t, shape, what: str, dev: int) -> tuple:
    """(address, batch, token and head stride) of a [B][T][heads][D] tensor
    with contiguous D; the stride of a dimension of size 1, which says nothing,
    is 0."""
    if t.shape != shape or t.stride(3) != 1:
        raise ValueError(f"{what}: expected {tuple(shape)} with contiguous rows, got "
                         f"{tuple(t.shape)}")
    if t.dtype not in _KV_DTYPES:
        raise ValueError(f"{what}: expected bfloat16, float16 or float32, got {t.dtype}")
    if t.get_device() != dev:
        _wrong_device(t, dev)
    B, T, H, _ = shape
    batch, token, head, _ = t.stride()
    return t.data_ptr(), batch if B > 1 else 0, token if T > 1 else 0, head if H > 1 else 0


def _kv_call(name: str, packed: bytes, workspace, dev: int, stream) -> None:
    # The library launches on the current device.
    if dev < 0:
        raise ValueError("libspecverify takes device tensors")
    if dev != _current_device():
        raise ValueError(f"{name}: the tensors are on cuda:{dev}, the current device is "
                         f"cuda:{_current_device()}")
    if stream is None:
        stream = current_raw_stream(dev)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    st = getattr(_lib_handle or lib(), name)(packed, workspace.data_ptr(), workspace.nbytes, stream)
    if st != SV_OK:
        raise SpecVerifyError(st, name)


def sv_kv_write(cache: dict, page_table, kv_len, k_new, v_new, workspace, num_new=None,
                stream=None) -> None:
    """Enqueue sv_kv_write: quantise k_new, v_new [B][T][Hkv][D] into the
    cache at positions kv_len[b] .. of each request."""
    B, T = k_new.shape[:2]
    dev = workspace.get_device()
    c = _kv_cache(cache, page_table, B, dev)
    shape = (B, T, c[2], c[3])
    k, *k_strides = _rows4(k_new, shape, "k_new", dev)
    v, *v_strides = _rows4(v_new, shape, "v_new", dev)
    if v_new.dtype != k_new.dtype:
        raise ValueError("v_new: expected k_new's dtype")
    length = _addr(kv_len, torch.int32, (B,), "kv_len", dev)
    num = _addr(num_new, torch.int32, (B,), "num_new", dev)
    _kv_call("sv_kv_write", _pack_write(*c, B, T, _KV_DTYPES[k_new.dtype], k, v, *k_strides,
                                        *v_strides, length, num), workspace, dev, stream)


def sv_kv_read(cache: dict, page_table, start, num, k_out, v_out, workspace, rows=None,
               stream=None) -> None:
    """Enqueue sv_kv_read: the values at positions start[b] + t, or start[b]
    + rows[b][t], into k_out, v_out [B][T][Hkv][D] (rows t >= num[b] zero)."""
    B, T = k_out.shape[:2]
    dev = workspace.get_device()
    c = _kv_cache(cache, page_table, B, dev)
    shape = (B, T, c[2], c[3])
    k, *strides = _rows4(k_out, shape, "k_out", dev)
    v, *v_strides = _rows4(v_out, shape, "v_out", dev)
    if v_strides != strides or v_out.dtype != k_out.dtype:
        raise ValueError("v_out: expected k_out's dtype and strides")
    first = _addr(start, torch.int32, (B,), "start", dev)
    count = _addr(num, torch.int32, (B,), "num", dev)
    which = _addr(rows, torch.int32, (B, T), "rows", dev)
    _kv_call("sv_kv_read", _pack_read(*c, B, T, _KV_DTYPES[k_out.dtype], k, v, *strides, first,
                                      count, which), workspace, dev, stream)


@functools.lru_cache(maxsize=1024)
def sv_kv_attention_workspace_bytes(B: int, T: int, Hq: int, Hkv: int, D: int) -> int:
    return lib().sv_kv_attention_workspace_bytes(B, T, Hq, Hkv, D)


def sv_kv_attention(q, cache: dict, page_table, kv_len, out, workspace, scale: float,
                    num_new=None, mask=None, lse=None, stream=None) -> None:
    """Enqueue sv_kv_attention: q [B][T][Hq][D] over the cache into out (the
    same shape, contiguous) and, optionally, lse [B][T][Hq] fp32."""
    shape = q.shape
    B, T, Hq, D = shape
    dev = workspace.get_device()
    c = _kv_cache(cache, page_table, B, dev)
    if D != c[3] or q.dtype == torch.float32:
        raise ValueError(f"q: expected bfloat16 or float16 [B][T][Hq][{c[3]}], got {q.dtype} "
                         f"{tuple(shape)}")
    qp, *strides = _rows4(q, shape, "q", dev)
    o = _addr(out, q.dtype, shape, "out", dev)
    ls = _addr(lse, torch.float32, (B, T, Hq), "lse", dev)
    length = _addr(kv_len, torch.int32, (B,), "kv_len", dev)
    num = _addr(num_new, torch.int32, (B,), "num_new", dev)
    words = 0
    if mask is not None:
        if mask.dim() != 3:
            raise ValueError("mask: expected [B][T][words]")
        words = mask.shape[2]
    m = _addr(mask, torch.int32, (B, T, words), "mask", dev)
    _kv_call("sv_kv_attention", _pack_attention(*c, B, T, Hq, _KV_DTYPES[q.dtype], qp, *strides,
                                                o, ls, length, num, m, words, scale),
             workspace, dev, stream)


# --------------------- norms and positions of queries and keys, log probabilities
#
# A model makes these calls in every layer or step and they take a dozen tensors
# each, so their marshalling is compiled (csrc/native.cpp).  Results that are not
# given are allocated there.

_native_module = None
_entries: dict = {}


def _native():
    global _native_module
    if _native_module is None:
        try:
            from . import _native as module
        except ImportError as e:
            raise RuntimeError("the compiled binding is missing: build it with "
                               "__graft_entry__.build()") from e
        _native_module = module
    return _native_module


def _entry(name: str) -> int:
    """The address of an entry point of the loaded library."""
    h = _lib_handle or lib()
    known = _entries.get(name)
    if known is None or known[0] is not h:
        known = _entries[name] = (h, ctypes.cast(getattr(h, name), ctypes.c_void_p).value)
    return known[1]


def _launched(name: str, result):
    if result.__class__ is int:
        raise SpecVerifyError(result, name)
    return result


def _raw_stream(stream):
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def sv_rotate(q, q_out, workspace, k=None, k_out=None, start=None, num=None, offset=None,
              rope=None, q_weight=None, k_weight=None, eps=None, stream=None) -> tuple:
    """Enqueue sv_rotate: norms and rotations of q and k [B][T][heads][D] into
    q_out and k_out (None: new tensors; Ellipsis: in place).  Returns both."""
    if stream is not None:
        stream = _raw_stream(stream)
    return _launched("sv_rotate", (_native_module or _native()).rotate(
        _entry("sv_rotate"), workspace, stream, q, q_out, k, k_out, start, num, offset, rope,
        q_weight, k_weight, eps))


def sv_kv_append(cache: dict, page_table, kv_len, k_new, v_new, workspace, q=None, q_out=None,
                 num_new=None, offset=None, rope=None, q_weight=None, k_weight=None, eps=None,
                 stream=None, q_dtype=None) -> tuple:
    """Enqueue sv_kv_append: keys normed, rotated and, with the values,
    quantised into the cache; queries normed and rotated into q_out (None: a new
    tensor of q_dtype, q's own by default).  Returns (q_out,)."""
    if stream is not None:
        stream = _raw_stream(stream)
    return _launched("sv_kv_append", (_native_module or _native()).kv_append(
        _entry("sv_kv_append"), workspace, stream, cache, page_table, kv_len, q, q_out, q_dtype,
        k_new, v_new, num_new, offset, rope, q_weight, k_weight, eps))


def sv_token_logprobs(logits, workspace, R=None, tokens=None, num_rows=None, rows=None,
                      temperature=None, top: int = 0, logprobs=None, entropy=None,
                      top_tokens=None, top_logprobs=None, stream=None,
                      allocate: bool = False) -> tuple:
    """Enqueue sv_token_logprobs on logits [B][N][V]: tokens and logprobs
    [B][R] or [B][R][M], entropy [B][R], top_tokens and top_logprobs
    [B][R][top] (allocate: new tensors for all that is asked for).  Returns
    logprobs, entropy, top_tokens and top_logprobs."""
    if stream is not None:
        stream = _raw_stream(stream)
    return _launched("sv_token_logprobs", (_native_module or _native()).token_logprobs(
        _entry("sv_token_logprobs"), workspace, stream, logits, R, tokens, num_rows, rows,
        temperature, top, allocate, logprobs, entropy, top_tokens, top_logprobs))
