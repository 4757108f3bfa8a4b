"""Softmax attention for the layers that stand between the Lightning layers of
the hybrid model: argument marshalling over the C ABI, as in `_binding`.

A call runs on the device of `q` and on `stream` (default: that device's
current stream); what it allocates -- outputs that were not passed, and the
workspace -- belongs to that stream.
"""
from __future__ import annotations

import contextlib

import torch

from ._binding import D, _check, _need, _out_code, _ptr, _stream_handle, lib

SCALE = D ** -0.5


@contextlib.contextmanager
def _on(q, stream):
    """Run on q's device and `stream`; yields the stream's handle."""
    with torch.cuda.device(q.device):
        if stream is None:
            yield _stream_handle(torch.cuda.current_stream(q.device))
            return
        if stream.device != q.device:
            raise ValueError("stream must be on the device of q")
        with torch.cuda.stream(stream):
            yield _stream_handle(stream)


def _same_device(q, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != q.device:
            raise ValueError(f"{name} must be on the device of q")


def _need_qkv(q, k, v):
    """Shapes of packed q [T, H, d], k and v [T, Hkv, d]: (T, H, Hkv, d)."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must be [T, heads, d]")
    T, H, d = q.shape
    Hkv = k.shape[1]
    _need(q, "q", torch.bfloat16, (T, H, d))
    _need(k, "k", torch.bfloat16, (T, Hkv, d))
    _need(v, "v", torch.bfloat16, (T, Hkv, d))
    if Hkv == 0 or H == 0 or H % Hkv:
        raise ValueError("the heads of q must be a multiple of those of k and v")
    return T, H, Hkv, d


def _scale(scale):
    return SCALE if scale is None else float(scale)


def _workspace(workspace, nbytes, device):
    if workspace is None:
        return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace


def _outputs(q, out, lse, want_lse, out_dtype=torch.bfloat16):
    T, H, d = q.shape
    if out is None:
        out = torch.empty((T, H, d), dtype=out_dtype, device=q.device)
    _need(out, "out", out_dtype, (T, H, d))
    if lse is None and want_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, (T, H))
    return out, lse


def softmax_prefill_varlen(q, k, v, cu_seqlens, max_seqlen: int, scale=None, out=None, lse=None,
                           want_lse: bool = True, workspace=None, stream=None):
    """la_softmax_prefill_varlen: causal softmax attention of packed bf16
    q [T, H, d] over k, v [T, Hkv, d] (H a multiple of Hkv) with device int32
    cu_seqlens.  scale: factor of the scores, d**-0.5 by default.  Returns
    (out [T, H, d] bf16, lse [T, H] fp32 or None)."""
    T, H, Hkv, d = _need_qkv(q, k, v)
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    nseq = cu_seqlens.numel() - 1
    if nseq < 0:
        raise ValueError("cu_seqlens must hold nseq + 1 entries")
    _same_device(q, k=k, v=v, cu_seqlens=cu_seqlens, out=out, lse=lse, workspace=workspace)
    with _on(q, stream) as handle:
        out, lse = _outputs(q, out, lse, want_lse)
        workspace = _workspace(workspace, lib().la_softmax_prefill_varlen_workspace_size(nseq, T, H, Hkv, d), q.device)
        st = lib().la_softmax_prefill_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), nseq, T, int(max_seqlen), H,
                                             Hkv, d, _scale(scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                             workspace.numel() * workspace.element_size(), handle)
    _check(st, "la_softmax_prefill_varlen")
    return out, lse


def softmax_prefill_backward_varlen(q, k, v, out, lse, dout, cu_seqlens, max_seqlen: int, scale=None, dq=None, dk=None,
                                    dv=None, workspace=None, stream=None):
    """la_softmax_prefill_backward_varlen: gradients of softmax_prefill_varlen
    for dL/dout; out and lse are what that call returned, scale what it was
    given.  Returns (dq [T, H, d], dk, dv [T, Hkv, d]) in bf16."""
    T, H, Hkv, d = _need_qkv(q, k, v)
    _need(out, "out", torch.bfloat16, (T, H, d))
    _need(lse, "lse", torch.float32, (T, H))
    _need(dout, "dout", torch.bfloat16, (T, H, d))
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    nseq = cu_seqlens.numel() - 1
    if nseq < 0:
        raise ValueError("cu_seqlens must hold nseq + 1 entries")
    _same_device(q, k=k, v=v, out=out, lse=lse, dout=dout, cu_seqlens=cu_seqlens, dq=dq, dk=dk, dv=dv,
                 workspace=workspace)
    with _on(q, stream) as handle:
        grads = []
        for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
            if t is None:
                t = torch.empty_like(like)
            _need(t, name, torch.bfloat16, like.shape)
            grads.append(t)
        workspace = _workspace(workspace,
                               lib().la_softmax_prefill_backward_varlen_workspace_size(nseq, T, H, Hkv, d), q.device)
        st = lib().la_softmax_prefill_backward_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                                      _ptr(cu_seqlens), nseq, T, int(max_seqlen), H, Hkv, d,
                                                      _scale(scale), _ptr(grads[0]), _ptr(grads[1]), _ptr(grads[2]),
                                                      _ptr(workspace), workspace.numel() * workspace.element_size(),
                                                      handle)
    _check(st, "la_softmax_prefill_backward_varlen")
    return tuple(grads)


def _need_cache(q, k_cache, v_cache, page_table, cache_lens, n, Hkv, d):
    """A paged cache of n requests: (n_pages, page_size, max_pages)."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [n_pages, Hkv, page_size, d]")
    n_pages, _, page, _ = k_cache.shape
    _need(k_cache, "k_cache", torch.bfloat16, (n_pages, Hkv, page, d))
    _need(v_cache, "v_cache", torch.bfloat16, (n_pages, Hkv, page, d))
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [requests, max_pages]")
    _need(page_table, "page_table", torch.int32, (n, page_table.shape[1]))
    _need(cache_lens, "cache_lens", torch.int32, (n,))
    _same_device(q, k_cache=k_cache, v_cache=v_cache, page_table=page_table, cache_lens=cache_lens)
    return n_pages, page, page_table.shape[1]


def softmax_prefill_paged(q, k, v, cu_seqlens, max_seqlen: int, k_cache, v_cache, page_table, cache_lens, scale=None,
                          out=None, lse=None, want_lse: bool = True, workspace=None, stream=None):
    """la_softmax_prefill_paged: the packed new tokens q [T, H, d], k, v
    [T, Hkv, d] of each sequence are written behind its cache_lens[i] cached
    ones and attend to all of them, causally among themselves.  k_cache,
    v_cache: bf16 [n_pages, Hkv, page_size, d], updated in place; page_table:
    device int32 [nseq, max_pages]; cache_lens: device int32 [nseq], lengths
    before the call.  Returns (out, lse or None)."""
    T, H, Hkv, d = _need_qkv(q, k, v)
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    nseq = cu_seqlens.numel() - 1
    if nseq < 0:
        raise ValueError("cu_seqlens must hold nseq + 1 entries")
    n_pages, page, max_pages = _need_cache(q, k_cache, v_cache, page_table, cache_lens, nseq, Hkv, d)
    _same_device(q, k=k, v=v, cu_seqlens=cu_seqlens, out=out, lse=lse, workspace=workspace)
    with _on(q, stream) as handle:
        out, lse = _outputs(q, out, lse, want_lse)
        workspace = _workspace(workspace, lib().la_softmax_prefill_paged_workspace_size(nseq, T, H, Hkv, d), q.device)
        st = lib().la_softmax_prefill_paged(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), nseq, T, int(max_seqlen), H,
                                            Hkv, d, _scale(scale), _ptr(k_cache), _ptr(v_cache), n_pages, page,
                                            _ptr(page_table), max_pages, _ptr(cache_lens), _ptr(out), _ptr(lse),
                                            _ptr(workspace), workspace.numel() * workspace.element_size(), handle)
    _check(st, "la_softmax_prefill_paged")
    return out, lse


def softmax_decode_paged(q, k, v, k_cache, v_cache, page_table, cache_lens, scale=None, out=None,
                         out_dtype=torch.bfloat16, lse=None, want_lse: bool = True, workspace=None, stream=None):
    """la_softmax_decode_paged: one new token per request, q [B, H, d], k, v
    [B, Hkv, d], written behind the cache_lens[b] cached ones (-1: no request,
    the row's outputs are left as they are).  The cache as for
    softmax_prefill_paged.  Returns (out [B, H, d] bf16 or fp32, lse [B, H] or
    None)."""
    B, H, Hkv, d = _need_qkv(q, k, v)
    n_pages, page, max_pages = _need_cache(q, k_cache, v_cache, page_table, cache_lens, B, Hkv, d)
    _same_device(q, k=k, v=v, out=out, lse=lse, workspace=workspace)
    with _on(q, stream) as handle:
        out, lse = _outputs(q, out, lse, want_lse, out_dtype if out is None else out.dtype)
        code = _out_code(out.dtype)
        workspace = _workspace(workspace, lib().la_softmax_decode_paged_workspace_size(B, H, Hkv, d), q.device)
        st = lib().la_softmax_decode_paged(_ptr(q), _ptr(k), _ptr(v), B, H, Hkv, d, _scale(scale), _ptr(k_cache),
                                           _ptr(v_cache), n_pages, page, _ptr(page_table), max_pages,
                                           _ptr(cache_lens), _ptr(out), code, _ptr(lse), _ptr(workspace),
                                           workspace.numel() * workspace.element_size(), handle)
    _check(st, "la_softmax_decode_paged")
    return out, lse


def cache_copy_pages(k_cache, v_cache, src, dst, stream=None):
    """la_cache_copy_pages: page src[i] is copied to page dst[i] in both
    tensors [n_pages, Hkv, page_size, d]; src, dst: device int32 [n]."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [n_pages, Hkv, page_size, d]")
    _need(k_cache, "k_cache", torch.bfloat16)
    _need(v_cache, "v_cache", torch.bfloat16, k_cache.shape)
    _need(src, "src", torch.int32, (src.numel(),))
    _need(dst, "dst", torch.int32, (src.numel(),))
    _same_device(k_cache, v_cache=v_cache, src=src, dst=dst)
    n_pages, Hkv, page, d = k_cache.shape
    with _on(k_cache, stream) as handle:
        st = lib().la_cache_copy_pages(_ptr(k_cache), _ptr(v_cache), n_pages, page, Hkv, d, _ptr(src), _ptr(dst),
                                       src.numel(), handle)
    _check(st, "la_cache_copy_pages")
