"""GB300-native fused scaled-dot-product attention.

``O = softmax(attn_scale * Q K^T + causal mask) V`` plus the per-row
log-sum-exp, dense BHSD or packed THD, and its backward, computed by
hand-written sm_103a kernels behind the C ABI in ``include/sdpa.h``.

This package is the thin Python side: ``_lib`` mirrors the C entry points
one to one, and the helpers below allocate outputs with torch and call them
(those of the paged key/value cache through the compiled ``csrc/calls.cpp``).
PyTorch only provides device memory and streams.
"""
from __future__ import annotations

import math
from typing import NamedTuple

from ._lib import (SDPA_BF16, SDPA_FP16, SDPA_FP8_E4M3, sdpa_fwd_fp8, sdpa_varlen_fwd_fp8,  # noqa: F401
                   SDPA_MASK_CAUSAL, SDPA_MASK_CAUSAL_BOTTOM_RIGHT,
                   SDPA_MASK_NONE, SdpaError, calls, dtype_code, load, sdpa_bwd, sdpa_bwd_ex,
                   sdpa_bwd_ex_workspace_size, sdpa_bwd_noalloc, sdpa_bwd_workspace_size,
                   sdpa_check_device_error, sdpa_fwd, sdpa_fwd_ex, sdpa_last_error,
                   sdpa_selftest_wait_timeout,
                   sdpa_last_backward_variant, sdpa_set_backward_grid_limit,
                   sdpa_cache_accept, sdpa_cache_append, sdpa_cache_plan, sdpa_tree_fwd,
                   sdpa_tree_fwd_workspace_size,
                   sdpa_set_backward_variant,
                   sdpa_set_forward_variant, sdpa_set_kernel_timer, sdpa_varlen_bwd,
                   sdpa_varlen_bwd_ex, sdpa_varlen_bwd_ex_workspace_size,
                   sdpa_varlen_bwd_workspace_size, sdpa_varlen_fwd, sdpa_varlen_fwd_ex, sdpa_version)

__all__ = ["attention", "attention_varlen", "attention_bwd", "attention_varlen_bwd",
           "sdpa_fwd", "sdpa_varlen_fwd", "sdpa_bwd", "sdpa_varlen_bwd", "sdpa_bwd_noalloc",
           "sdpa_fwd_ex", "sdpa_varlen_fwd_ex", "sdpa_bwd_ex", "sdpa_varlen_bwd_ex",
           "sdpa_bwd_workspace_size", "sdpa_varlen_bwd_workspace_size",
           "sdpa_bwd_ex_workspace_size", "sdpa_varlen_bwd_ex_workspace_size", "sdpa_last_error",
           "sdpa_check_device_error", "sdpa_selftest_wait_timeout", "sdpa_set_forward_variant",
           "sdpa_set_backward_variant", "sdpa_last_backward_variant",
           "sdpa_set_backward_grid_limit", "sdpa_set_kernel_timer",
           "sdpa_version", "SdpaError", "load", "SDPA_MASK_NONE", "SDPA_MASK_CAUSAL",
           "SDPA_MASK_CAUSAL_BOTTOM_RIGHT", "SDPA_FP8_E4M3", "sdpa_fwd_fp8", "sdpa_varlen_fwd_fp8",
           "attention_fp8", "attention_tree", "attention_tree_workspace", "cache_plan", "CachePlan",
           "cache_append", "cache_accept", "sdpa_cache_plan", "sdpa_cache_append",
           "sdpa_cache_accept", "sdpa_tree_fwd", "sdpa_tree_fwd_workspace_size"]

_MASK_NAMES = {"none": SDPA_MASK_NONE, "top_left": SDPA_MASK_CAUSAL,
               "bottom_right": SDPA_MASK_CAUSAL_BOTTOM_RIGHT}


def _mask_code(causal, mask) -> int:
    """`mask` (an SDPA_MASK_* value or "none" / "top_left" / "bottom_right")
    overrides the plain `causal` flag when given."""
    if mask is None:
        return SDPA_MASK_CAUSAL if causal else SDPA_MASK_NONE
    return _MASK_NAMES[mask] if isinstance(mask, str) else int(mask)


def _default_scale(d: int, scale):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def attention(q, k, v, *, scale=None, causal=False, mask=None, window_left=-1, stream=None):
    """Dense forward. q [b,h,s_q,d], k/v [b,h_kv,s_kv,d] (CUDA, contiguous) -> (o, lse).

    h_kv may divide h (grouped key/value heads); `mask` and `window_left`
    select the masks of include/sdpa.h (sdpa_mask)."""
    import torch
    b, h, s_q, d = q.shape
    h_kv, s_kv = k.shape[1], k.shape[2]
    m = _mask_code(causal, mask)
    o = torch.empty_like(q)
    lse = torch.empty((b, h, s_q), dtype=torch.float32, device=q.device)
    if h_kv == h and window_left < 0 and m != SDPA_MASK_CAUSAL_BOTTOM_RIGHT:
        sdpa_fwd(q, k, v, o, lse, b, h, s_q, s_kv, d, _default_scale(d, scale), m,
                 dtype_code(q), stream)
    else:
        sdpa_fwd_ex(q, k, v, o, lse, b, h, h_kv, s_q, s_kv, d, _default_scale(d, scale), m,
                    window_left, dtype_code(q), stream)
    return o, lse


def attention_varlen(q, k, v, cu_seqlens_q, cu_seqlens_kv, max_seqlen_q, max_seqlen_kv, *,
                     scale=None, causal=False, mask=None, window_left=-1, stream=None,
                     total_q=None, total_kv=None):
    """Packed forward. q [Tq,h,d], k/v [Tkv,h_kv,d], cu_seqlens int32 on the device.

    ``total_q``/``total_kv`` default to the tensors' first dimension; pass them
    when the buffers hold spare capacity past the packed total.
    """
    import torch
    tq = q.shape[0] if total_q is None else int(total_q)
    tkv = k.shape[0] if total_kv is None else int(total_kv)
    _, h, d = q.shape
    h_kv = k.shape[1]
    m = _mask_code(causal, mask)
    o = torch.empty_like(q)
    lse = torch.empty((q.shape[0], h), dtype=torch.float32, device=q.device)
    args = (cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q.numel() - 1, tq, tkv, int(max_seqlen_q),
            int(max_seqlen_kv))
    if h_kv == h and window_left < 0 and m != SDPA_MASK_CAUSAL_BOTTOM_RIGHT:
        sdpa_varlen_fwd(q, k, v, o, lse, *args, h, d, _default_scale(d, scale), m, dtype_code(q),
                        stream)
    else:
        sdpa_varlen_fwd_ex(q, k, v, o, lse, *args, h, h_kv, d, _default_scale(d, scale), m,
                           window_left, dtype_code(q), stream)
    return o, lse


def attention_bwd(q, k, v, o, dout, lse, *, scale=None, causal=False, mask=None, window_left=-1,
                  deterministic=False, stream=None, workspace=None):
    """Dense backward -> (dq, dk, dv).  Allocates the workspace unless one is given."""
    import torch
    b, h, s_q, d = q.shape
    h_kv, s_kv = k.shape[1], k.shape[2]
    m = _mask_code(causal, mask)
    plain = (h_kv == h and window_left < 0 and m != SDPA_MASK_CAUSAL_BOTTOM_RIGHT
             and not deterministic)
    ws_bytes = (sdpa_bwd_workspace_size(b, h, s_q, d) if plain
                else sdpa_bwd_ex_workspace_size(b, h, s_q, d, int(bool(deterministic))))
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if plain:
        sdpa_bwd(q, k, v, o, dout, lse, dq, dk, dv, b, h, s_q, s_kv, d, _default_scale(d, scale),
                 m, dtype_code(q), workspace, workspace.numel(), stream)
    else:
        sdpa_bwd_ex(q, k, v, o, dout, lse, dq, dk, dv, b, h, h_kv, s_q, s_kv, d,
                    _default_scale(d, scale), m, window_left, int(bool(deterministic)),
                    dtype_code(q), workspace, workspace.numel(), stream)
    return dq, dk, dv


def attention_varlen_bwd(q, k, v, o, dout, lse, cu_seqlens_q, cu_seqlens_kv, max_seqlen_q,
                         max_seqlen_kv, *, scale=None, causal=False, mask=None, window_left=-1,
                         deterministic=False, stream=None, workspace=None, total_q=None,
                         total_kv=None):
    """Packed backward -> (dq, dk, dv) in the packed layouts."""
    import torch
    tq = q.shape[0] if total_q is None else int(total_q)
    tkv = k.shape[0] if total_kv is None else int(total_kv)
    _, h, d = q.shape
    h_kv = k.shape[1]
    m = _mask_code(causal, mask)
    plain = (h_kv == h and window_left < 0 and m != SDPA_MASK_CAUSAL_BOTTOM_RIGHT
             and not deterministic)
    ws_bytes = (sdpa_varlen_bwd_workspace_size(tq, h, d) if plain
                else sdpa_varlen_bwd_ex_workspace_size(tq, h, d, int(bool(deterministic))))
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    args = (cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q.numel() - 1, tq, tkv, int(max_seqlen_q),
            int(max_seqlen_kv))
    if plain:
        sdpa_varlen_bwd(q, k, v, o, dout, lse, dq, dk, dv, *args, h, d, _default_scale(d, scale),
                        m, dtype_code(q), workspace, workspace.numel(), stream)
    else:
        sdpa_varlen_bwd_ex(q, k, v, o, dout, lse, dq, dk, dv, *args, h, h_kv, d,
                           _default_scale(d, scale), m, window_left, int(bool(deterministic)),
                           dtype_code(q), workspace, workspace.numel(), stream)
    return dq, dk, dv


def attention_fp8(q, k, v, descale_q, descale_k, descale_v, *, scale=None, causal=False, mask=None,
                  window_left=-1, out_dtype=None, scale_o=None, want_amax=True, stream=None):
    """Dense FP8 forward.  q [b,h,s_q,d], k/v [b,h_kv,s_kv,d] as torch.float8_e4m3fn (or
    uint8 codes) on the GPU; descales are 1-element fp32 CUDA tensors.  out_dtype:
    torch.bfloat16 (default), torch.float16 or torch.float8_e4m3fn (needs scale_o).
    -> (o, lse, amax) with amax a 1-element fp32 tensor (or None)."""
    import torch
    b, h, s_q, d = q.shape
    h_kv, s_kv = k.shape[1], k.shape[2]
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    code = {torch.bfloat16: SDPA_BF16, torch.float16: SDPA_FP16}.get(out_dtype, SDPA_FP8_E4M3)
    o = torch.empty((b, h, s_q, d), dtype=out_dtype, device=q.device)
    lse = torch.empty((b, h, s_q), dtype=torch.float32, device=q.device)
    amax = torch.empty(1, dtype=torch.float32, device=q.device) if want_amax else None
    sdpa_fwd_fp8(q, k, v, o, lse, descale_q, descale_k, descale_v, scale_o, amax, b, h, h_kv, s_q,
                 s_kv, d, _default_scale(d, scale), _mask_code(causal, mask), window_left, code,
                 stream)
    return o, lse, amax


# ------------------------------------------------------------------ paged key/value cache
# Checked and marshalled in csrc/calls.cpp: a decoding step is a few of these calls a layer.
# What a call allocates is memory of the stream that it runs on (`stream`, or the current one),
# kept until the current stream is through with it too.
class CachePlan(NamedTuple):
    """What cache_plan writes.  cu_new [b + 1] and kv_lens [b] go to attention_tree, slot_map
    [max_new] to cache_append; positions [max_new]; tree_mask [max_new, mask_words] or None;
    held [b] and ring_state [3] are the next plan's."""
    cu_new: object
    kv_lens: object
    slot_map: object
    positions: object
    tree_mask: object
    held: object
    ring_state: object


def cache_plan(ctx_lens, new_lens, held, ring_state, free_ring, block_table, page_size, max_new, *,
               parents=None, mask_words=0, out=None, stream=None):
    """Pages, slots, positions and tree masks of one step, from the requests' lengths.

    ctx_lens, new_lens, held [b]: tokens in the cache, tokens of this step (negative: the
    request has finished and gives its pages back) and pages a request holds.  ring_state [3]
    and free_ring [num_pages]: the free pages are free_ring[(ring_state[0] + i) % num_pages] for
    i < ring_state[1].  block_table [b, max_blocks] gets the new pages, free_ring the returned
    ones, both in place.  parents [max_new] (packed like the tokens; -1: child of the context's
    last token, below -1: padding) makes the new tokens of each request a tree.  All int32.
    out: an earlier CachePlan of the same sizes to write to (not the one whose held and
    ring_state are read).  -> CachePlan."""
    got = calls().cache_plan(ctx_lens, new_lens, held, ring_state, free_ring, block_table, page_size,
                             max_new, parents, mask_words, out, stream)
    return got if got is out else CachePlan(*got)


def cache_append(k, v, k_cache, v_cache, slot_map, *, scale_k=None, scale_v=None, stream=None):
    """Writes k, v [tokens, h_kv, d] to their slots of the caches [num_pages, h_kv, page_size, d]
    (a negative slot: not written).  Into an E4M3 cache goes the code of k * scale_k and
    v * scale_v (1-element fp32 CUDA tensors), saturated.  The tokens of k and v may be apart."""
    calls().cache_append(k, v, k_cache, v_cache, slot_map, scale_k, scale_v, stream)


def cache_accept(k_cache, v_cache, block_table, ctx_lens, new_lens, path, path_lens, *, out=None,
                 stream=None):
    """Keeps the accepted nodes of each request's verified tree: the rows of nodes path[b, j],
    j < path_lens[b] (ascending), move to the tree's first rows.  -> the new context lengths."""
    return calls().cache_accept(k_cache, v_cache, block_table, ctx_lens, new_lens, path, path_lens,
                                out, stream)


def attention_tree_workspace(q, k_cache, num_seqs, max_seqlen_q, max_seqlen_kv):
    """The workspace that attention_tree takes for requests of up to these lengths."""
    return calls().attention_tree_workspace(q, k_cache, num_seqs, max_seqlen_q, max_seqlen_kv)


def attention_tree(q, k_cache, v_cache, block_table, cu_seqlens_q, kv_lens, max_seqlen_q,
                   max_seqlen_kv, *, tree_mask=None, scale=None, descale_k=None, descale_v=None,
                   out=None, workspace=None, stream=None):
    """Attention of each request's new tokens over its cached keys and values -> (o, lse).

    q [total_q, h, d] (the tokens may be apart), caches [num_pages, h_kv, page_size, d] in q's
    type, or E4M3 with 1-element fp32 descales; block_table [b, max_blocks], cu_seqlens_q
    [b + 1], kv_lens [b] int32.  The last cu_seqlens_q[i + 1] - cu_seqlens_q[i] of a request's
    kv_lens[i] tokens are the new ones; each sees all tokens before them, and of the new ones
    those whose bits its tree_mask row names (without a mask: itself and the ones before it).
    max_seqlen_q (at most total_q) and max_seqlen_kv bound a request's new tokens and kv_lens.
    out: (o, lse) to write to; workspace: from attention_tree_workspace."""
    return calls().attention_tree(q, k_cache, v_cache, block_table, cu_seqlens_q, kv_lens,
                                  max_seqlen_q, max_seqlen_kv, tree_mask,
                                  _default_scale(k_cache.shape[-1], scale), descale_k, descale_v, out,
                                  workspace, stream)
