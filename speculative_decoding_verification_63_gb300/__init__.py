"""GB300 (sm_103a) speculative-sampling verification step.

The computation runs in libspecverify.so (hand-written CUDA for sm_103a,
C ABI in include/specverify.h).  This package holds the ctypes binding
(_binding), the build (_build), the seeded synthetic workloads (workloads)
and a thin convenience layer that allocates outputs and workspaces with
torch and calls the C ABI.  There is no CPU fallback: without the built
library every call raises.
"""
from __future__ import annotations

import threading

import torch

from ._binding import (  # noqa: F401
    EXPORTS, SV_BF16, SV_DERR_ARG, SV_DERR_CHECK, SV_DERR_MASS, SV_DERR_NONFINITE, SV_DERR_TIMEOUT,
    SV_DERR_TOKEN, SV_DERR_TREE, SV_ECORESIDENT, SV_EDATA, SV_EINVAL, SV_ETIMEOUT, SV_EUNSUPPORTED,
    SV_EWORKSPACE, SV_FP32, SV_MAX_B, SV_MAX_K, SV_MAX_TOPK, SV_MAX_TREE_B,
    SV_MAX_TREE_NODES, SV_MAX_V, SV_OK, SpecVerifyError, lib, sv_chain_workspace_bytes,
    sv_get_error, sv_selftest_wait_timeout, sv_status_string, sv_tree_workspace_bytes,
    sv_verify_chain, sv_verify_tree, sv_version, sv_workspace_init,
    SV_NOALLOC_SCRATCH_BYTES, sv_noalloc_get_error, sv_verify_chain_noalloc,
    SV_TREE_MSS, SV_TREE_MSS_NOREPLACE, SV_TREE_NAIVE, TREE_MODES, SV_MIN_WORKSPACE_BYTES,
    sv_tree_mask, sv_row_stats, SV_FP16, SV_DERR_PAGE, SV_MAX_KV_HEADS, SV_MAX_KV_T,
    sv_kv_attention, sv_kv_attention_workspace_bytes, sv_kv_read, sv_kv_write,
    sv_stream_capture_id, current_raw_stream)
from ._build import build_library  # noqa: F401

_ws_lock = threading.Lock()
_ws_cache: dict = {}
_ws_kept: list = []   # buffers that a larger one replaced: captured graphs may name them
_ws_graph: dict = {}  # those of the capture under way: its id and its buffers
# Calls that hold more than the error word in their workspace and are at home
# on several streams at once (a prompt on one, decoding on another).
_WS_PER_STREAM = ("kv_attention",)


def workspace(nbytes: int, device=None, key=None) -> torch.Tensor:
    """A zeroed, 256-byte aligned device workspace of at least nbytes,
    cached per (device, key), and for key "kv_attention" per current stream
    too.  Calls sharing one workspace must not overlap on the GPU.  A cached
    buffer stays allocated when a larger one takes its place, so a graph
    captured with it stays valid.

    While the current stream is being captured, a buffer that does not exist
    yet, and always one of "kv_attention", belongs to the graph: it comes from
    the graph's memory and is zeroed by the graph, once, ahead of the first
    call that uses it.  (To read the error word of such a call, get the
    workspace inside the capture and keep it.)"""
    if not isinstance(device, torch.device) or device.index is None:
        device = torch.device(device if device is not None else "cuda")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
    if key in _WS_PER_STREAM:
        stream = current_raw_stream(device.index)
        capturing = torch.cuda.is_current_stream_capturing()
        buf = None if capturing else _ws_cache.get((device, key, stream))
        if buf is None or buf.numel() < nbytes:
            buf = _make_workspace(nbytes, device, (device, key, stream), stream, capturing)
    else:
        buf = _ws_cache.get((device, key))
        if buf is None or buf.numel() < nbytes:
            stream = current_raw_stream(device.index)
            capturing = torch.cuda.is_current_stream_capturing()
            buf = _make_workspace(nbytes, device, (device, key), stream, capturing)
    return buf


def _make_workspace(nbytes: int, device, k, stream: int, capturing: bool) -> torch.Tensor:
    with _ws_lock:
        if capturing:
            return _graph_workspace(nbytes, device, (k, stream), stream)
        old = _ws_cache.get(k)
        if old is not None and old.numel() >= nbytes:
            return old  # another thread's, meanwhile
        if old is not None:
            _ws_kept.append(old)
        # (sizes are rounded up to a power of two: all that a growing one
        # leaves behind is smaller than the last)
        buf = _new_workspace(1 << (max(nbytes, 256) - 1).bit_length(), device, stream)
        if len(k) == 2:  # any stream may be the next to use it: zeroed by then
            torch.cuda.current_stream(device).synchronize()
        _ws_cache[k] = buf
        return buf


def _new_workspace(nbytes: int, device, stream: int) -> torch.Tensor:
    buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if buf.data_ptr() % 256:
        raise RuntimeError("torch returned a workspace that is not 256-byte aligned")
    sv_workspace_init(buf, stream)
    return buf


def _graph_workspace(nbytes: int, device, k, stream: int) -> torch.Tensor:
    """The buffer k of the capture that the current stream is part of.  Kept
    here until the next capture begins; the memory is the graph's."""
    capture = sv_stream_capture_id(stream)
    if _ws_graph.get("capture") != capture:
        _ws_graph.clear()
        _ws_graph["capture"] = capture
    buf = _ws_graph.get(k)
    if buf is None or buf.numel() < nbytes:
        buf = _ws_graph[k] = _new_workspace(max(nbytes, 256), device, stream)
    return buf


def dtype_code(t: torch.Tensor) -> int:
    return SV_BF16 if t.dtype == torch.bfloat16 else SV_FP32


def verify_chain(target_logits, draft_logits, draft_tokens, temperature, uniforms,
                 num_drafts=None, top_k=None, max_top_k: int | None = None,
                 with_probs: bool = False, ws: torch.Tensor | None = None) -> dict:
    """Chain verification of a batch on the current stream (asynchronous).

    target_logits [B][K+1][V] and draft_logits [B][K][V] (bf16 or fp32),
    draft_tokens [B][K] int32, temperature [B] fp32 (0 = greedy), uniforms
    [B][K+1] fp32; optional num_drafts [B] int32 and top_k [B] int32.
    Returns device tensors out_tokens [B][K+1], out_len [B], accept_len [B]
    (and p_at_draft, q_at_draft [B][K] when with_probs)."""
    B, K1, V = target_logits.shape
    K = K1 - 1
    dev = target_logits.device
    if max_top_k is None:
        max_top_k = 0 if top_k is None else SV_MAX_TOPK
    out = dict(out_tokens=torch.empty((B, K1), dtype=torch.int32, device=dev),
               out_len=torch.empty(B, dtype=torch.int32, device=dev),
               accept_len=torch.empty(B, dtype=torch.int32, device=dev))
    if with_probs:
        out["p_at_draft"] = torch.empty((B, K), dtype=torch.float32, device=dev)
        out["q_at_draft"] = torch.empty((B, K), dtype=torch.float32, device=dev)
    need = sv_chain_workspace_bytes(B, K, V, dtype_code(target_logits), max_top_k)
    if need == 0:
        raise SpecVerifyError(SV_EINVAL, "verify_chain (sizes)")
    if ws is None:
        ws = workspace(need, dev, "chain")
    sv_verify_chain(target_logits, draft_logits, draft_tokens, temperature, uniforms,
                    out["out_tokens"], out["out_len"], out["accept_len"], ws,
                    num_drafts=num_drafts, top_k=top_k, max_top_k=max_top_k,
                    p_at_draft=out.get("p_at_draft"), q_at_draft=out.get("q_at_draft"))
    return out


def verify_tree(target_logits, draft_logits, node_tokens, parent, q_row, temperature,
                u_accept, u_sample, max_depth: int, num_nodes=None,
                ws: torch.Tensor | None = None, mode: str = "mss") -> dict:
    """Token-tree verification on the current stream: VerifyGreedy for
    temperature 0, otherwise the stochastic rule `mode` ("mss", "noreplace"
    for children drawn without replacement, or "naive" sampling).
    Returns out_tokens [B][max_depth+1], out_len, accept_len and
    accepted_nodes [B][max_depth] (device tensors)."""
    B, N, V = target_logits.shape
    M = draft_logits.shape[1] if draft_logits is not None else 1
    dev = target_logits.device
    out = dict(out_tokens=torch.empty((B, max_depth + 1), dtype=torch.int32, device=dev),
               out_len=torch.empty(B, dtype=torch.int32, device=dev),
               accept_len=torch.empty(B, dtype=torch.int32, device=dev),
               accepted_nodes=torch.empty((B, max(max_depth, 1)), dtype=torch.int32,
                                          device=dev))
    need = sv_tree_workspace_bytes(B, N, M, V, dtype_code(target_logits), 0)
    if need == 0:
        raise SpecVerifyError(SV_EINVAL, "verify_tree (sizes)")
    if ws is None:
        ws = workspace(need, dev, "tree")
    sv_verify_tree(target_logits, draft_logits, node_tokens, parent, q_row, temperature,
                   u_accept, u_sample, out["out_tokens"], out["out_len"], out["accept_len"],
                   out["accepted_nodes"], ws, max_depth=max_depth, num_nodes=num_nodes,
                   mode=TREE_MODES[mode])
    if max_depth == 0:
        out["accepted_nodes"] = out["accepted_nodes"][:, :0]
    return out


def tree_mask(parent, num_nodes=None, words: int | None = None,
              ws: torch.Tensor | None = None) -> dict:
    """Tree-attention mask and depth position ids of DFS-linearised trees
    (parent [B][N] int32 on the device).  Returns mask [B][N][words] (the
    uint32 words in int32 storage: bit j of row i set iff j is i or an
    ancestor of i) and depth [B][N] (device tensors)."""
    B, N = parent.shape
    W = (N + 31) // 32 if words is None else words
    dev = parent.device
    out = dict(mask=torch.empty((B, N, W), dtype=torch.int32, device=dev),
               depth=torch.empty((B, N), dtype=torch.int32, device=dev))
    if ws is None:
        ws = workspace(SV_MIN_WORKSPACE_BYTES, dev, "mask")
    sv_tree_mask(parent, out["mask"], out["depth"], ws, num_nodes=num_nodes)
    return out


def row_stats(target_logits, draft_logits, temperature, num_drafts=None, top_k=None,
              ws: torch.Tensor | None = None, max_top_k: int | None = None) -> dict:
    """Per-position acceptance rates alpha [B][K] (sum min(p_i, q_i), over
    the top-k sets of filtered requests) and the expected tokens per round
    [B] of a chain batch (device tensors)."""
    B, K1, V = target_logits.shape
    K = K1 - 1
    dev = target_logits.device
    if max_top_k is None:
        max_top_k = 0 if top_k is None else SV_MAX_TOPK
    out = dict(alpha=torch.empty((B, K), dtype=torch.float32, device=dev),
               expected=torch.empty(B, dtype=torch.float32, device=dev))
    if ws is None:
        ws = workspace(sv_chain_workspace_bytes(max(B, 1), K, V, dtype_code(target_logits),
                                                max_top_k), dev, "chain")
    sv_row_stats(target_logits, draft_logits, temperature, out["alpha"], out["expected"], ws,
                 num_drafts=num_drafts, top_k=top_k, max_top_k=max_top_k)
    return out


def kv_cache(num_pages: int, page_size: int, num_heads: int, head_dim: int,
             device=None) -> dict:
    """An empty 8-bit key/value cache: e4m3 codes k, v [num_pages][num_heads]
    [page_size][head_dim] and power-of-two scales k_scale, v_scale
    [num_pages][num_heads] (device tensors).  Which pages a request holds is
    the caller's page table [B][slots] int32 (slot i: tokens i * page_size ..)."""
    dev = torch.device(device if device is not None else "cuda")
    shape = (num_pages, num_heads, page_size, head_dim)
    return dict(k=torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn),
                v=torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn),
                k_scale=torch.ones(shape[:2], dtype=torch.float32, device=dev),
                v_scale=torch.ones(shape[:2], dtype=torch.float32, device=dev))


def kv_write(cache: dict, page_table, kv_len, k_new, v_new, num_new=None,
             ws: torch.Tensor | None = None) -> None:
    """Quantise a round's keys and values k_new, v_new [B][T][heads][D] (bf16,
    fp16 or fp32) into the cache: token t < num_new[b] goes to position
    kv_len[b] + t of request b."""
    if ws is None:
        ws = workspace(SV_MIN_WORKSPACE_BYTES, k_new.device, "kv")
    sv_kv_write(cache, page_table, kv_len, k_new, v_new, ws, num_new=num_new)


def kv_read(cache: dict, page_table, start, num, T: int, rows=None, dtype=torch.bfloat16,
            ws: torch.Tensor | None = None) -> dict:
    """Read tokens back as values: row t < num[b] is position start[b] + t, or
    start[b] + rows[b][t]; later rows are zero.  Returns k and v
    [B][T][heads][D] (device tensors)."""
    _, H, _, D = cache["k"].shape
    dev = page_table.device
    k = torch.empty((page_table.shape[0], T, H, D), dtype=dtype, device=dev)
    out = dict(k=k, v=torch.empty_like(k))
    if ws is None:
        ws = workspace(SV_MIN_WORKSPACE_BYTES, dev, "kv")
    sv_kv_read(cache, page_table, start, num, out["k"], out["v"], ws, rows=rows)
    return out


def kv_attention(q, cache: dict, page_table, kv_len, num_new=None, mask=None,
                 scale: float | None = None, with_lse: bool = False,
                 ws: torch.Tensor | None = None) -> dict:
    """Attention of a round's queries q [B][T][heads][D] (bf16 or fp16) over
    the cache, which holds kv_len[b] earlier tokens and the round's own (see
    kv_write): causal among the round's tokens, or by the rows of a tree mask
    [B][T][words] (tree_mask).  scale defaults to 1 / sqrt(D).  Returns out
    [B][T][heads][D] and, when with_lse, lse [B][T][heads] (device tensors).
    Without ws the current stream's own workspace serves (a captured call's,
    the graph's: workspace()), so calls on several streams may overlap; calls
    that are given one ws must not."""
    B, T, Hq, D = q.shape
    out = dict(out=torch.empty_like(q, memory_format=torch.contiguous_format))
    if with_lse:
        out["lse"] = torch.empty((B, T, Hq), dtype=torch.float32, device=q.device)
    if ws is None:
        need = sv_kv_attention_workspace_bytes(B, T, Hq, cache["k"].shape[1], D)
        if need == 0:
            raise SpecVerifyError(SV_EINVAL, "kv_attention (sizes)")
        ws = workspace(need, q.device, "kv_attention")
    sv_kv_attention(q, cache, page_table, kv_len, out["out"], ws,
                    scale=D ** -0.5 if scale is None else scale, num_new=num_new, mask=mask,
                    lse=out.get("lse"))
    return out


def kv_commit(cache: dict, page_table, kv_len, accept_len, accepted_nodes,
              ws: torch.Tensor | None = None) -> None:
    """Keep a tree round's accepted path: the tokens of accepted_nodes[b][0 ..
    accept_len[b]) (verify_tree's results), which kv_write put at kv_len[b] +
    node, move to kv_len[b] + 1 .. behind the root.  The request then holds
    kv_len + 1 + accept_len tokens.  (A chain round needs nothing moved: it
    holds kv_len + 1 + accept_len tokens as it is.)"""
    T = accepted_nodes.shape[1]
    if T == 0:
        return
    path = kv_read(cache, page_table, kv_len, accept_len, T, rows=accepted_nodes, ws=ws)
    kv_write(cache, page_table, kv_len + 1, path["k"], path["v"], num_new=accept_len, ws=ws)


def check_device_errors(ws: torch.Tensor) -> None:
    """Synchronise and raise if the last calls on `ws` recorded a device
    error (the workspace is re-initialised in that case)."""
    st, flags = sv_get_error(ws)
    if st != SV_OK:
        sv_workspace_init(ws)
        raise SpecVerifyError(st, "device", flags)
