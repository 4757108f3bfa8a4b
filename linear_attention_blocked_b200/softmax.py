"""Softmax attention for the layers that stand between the Lightning layers of
the hybrid model: argument marshalling over the C ABI, as in `_binding`.

A call runs on the device of `q` and on `stream` (default: that device's
current stream); what it allocates -- outputs that were not passed, and the
workspace -- belongs to that stream.

A decode step of one request takes some seven microseconds on the GPU, so the
marshalling is kept short.  Calls of the plain kind (no stream or workspace
passed, everything on the current device and as documented) go through a small
compiled module where it is built; the others, and those with something wrong,
through the Python code here, which checks everything and says what is wrong.
"""
from __future__ import annotations

import functools
import importlib.machinery
import importlib.util
import os

import torch

from . import _build
from ._binding import D, LA_BF16, LA_FP32, LA_OK, LAError, _need, lib

SCALE = D ** -0.5
_BF16, _FP32, _INT32 = torch.bfloat16, torch.float32, torch.int32
_raw_stream = torch._C._cuda_getCurrentRawStream


def _load_marshal():
    path = _build.marshal_path()
    if not os.path.exists(path) or not os.path.exists(_build.LIB_PATH):
        return None
    try:
        loader = importlib.machinery.ExtensionFileLoader("_marshal", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_marshal", loader))
        loader.exec_module(module)
        return module
    except ImportError:
        return None


_marshal = False  # not looked for yet


def _module():
    """The compiled module, or None."""
    global _marshal
    if _marshal is False:
        _marshal = _load_marshal()
    return _marshal


def _fits(t, name, dtype, shape, dev):
    """t is a contiguous tensor of this dtype and shape on CUDA device dev, or raise."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.get_device() == dev):
        _need(t, name, dtype, shape)
        raise ValueError(f"{name} must be on the device of q")


def _like(t, name, ref, dev):
    """t, or, for None, an uninitialised tensor like the contiguous `ref`."""
    if t is None:
        return torch.empty_like(ref)
    _fits(t, name, ref.dtype, ref.shape, dev)
    return t


def _rows(lse, want, q, T, H, dev):
    """The lse [T, H] to write, or None."""
    if lse is not None:
        _fits(lse, "lse", _FP32, (T, H), dev)
    elif want:
        lse = q.new_empty((T, H), dtype=_FP32)
    return lse


def _dims(q, k, v):
    """Packed q [T, H, d], k and v [T, Hkv, d]: (T, H, Hkv, d, device)."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must be [T, heads, d]")
    T, H, d = q.shape
    Hkv = k.shape[1]
    dev = q.get_device()
    _need(q, "q", _BF16)
    _fits(k, "k", _BF16, (T, Hkv, d), dev)
    _fits(v, "v", _BF16, (T, Hkv, d), dev)
    if Hkv == 0 or H == 0 or H % Hkv:
        raise ValueError("the heads of q must be a multiple of those of k and v")
    return T, H, Hkv, d, dev


def _sequences(cu_seqlens, max_seqlen, dev):
    """Number of sequences, with max_seqlen a length."""
    if not 0 <= max_seqlen <= 0x7FFFFFFF:
        raise ValueError("max_seqlen must be a length")
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must hold nseq + 1 entries")
    _fits(cu_seqlens, "cu_seqlens", _INT32, cu_seqlens.shape, dev)
    return cu_seqlens.shape[0] - 1


def _cache(k_cache, v_cache, page_table, cache_lens, n, Hkv, d, dev):
    """A paged cache of n requests: (n_pages, page_size, max_pages)."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [n_pages, Hkv, page_size, d]")
    n_pages, _, page, _ = k_cache.shape
    _fits(k_cache, "k_cache", _BF16, (n_pages, Hkv, page, d), dev)
    _fits(v_cache, "v_cache", _BF16, (n_pages, Hkv, page, d), dev)
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [requests, max_pages]")
    max_pages = page_table.shape[1]
    _fits(page_table, "page_table", _INT32, (n, max_pages), dev)
    _fits(cache_lens, "cache_lens", _INT32, (n,), dev)
    return n_pages, page, max_pages


@functools.lru_cache(maxsize=4096)
def _size(name, *shape):
    return int(getattr(lib(), name)(*shape))


def _scratch(workspace, nbytes, q, dev):
    """The workspace's (tensor, address, bytes)."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = q.new_empty(nbytes, dtype=torch.uint8)
        return workspace, workspace.data_ptr(), nbytes
    if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError("workspace must be a contiguous CUDA tensor on the device of q")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _on_stream(call):
    """call(*args, handle=..., **kw) on the device of its first tensor and on
    `stream`."""
    @functools.wraps(call)
    def run(first, *args, stream=None, **kw):
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise ValueError(f"the tensors of {call.__name__} must be CUDA tensors")
        dev = first.get_device()
        if stream is None and torch.cuda.current_device() == dev:
            return call(first, *args, handle=_raw_stream(dev), **kw)
        if stream is not None and stream.device != first.device:
            raise ValueError("stream must be on the device of the tensors")
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            return call(first, *args, handle=_raw_stream(dev), **kw)
    return run


def _done(status, where):
    if status != LA_OK:
        raise LAError(status, where)


def _short(result, where):
    """What the compiled module returned: results, a status, or None."""
    if result.__class__ is int:
        raise LAError(result, where)
    return result


@_on_stream
def _softmax_prefill_varlen(q, k, v, cu_seqlens, max_seqlen, scale, out, lse, want_lse, workspace, *, handle):
    T, H, Hkv, d, dev = _dims(q, k, v)
    nseq = _sequences(cu_seqlens, max_seqlen, dev)
    out = _like(out, "out", q, dev)
    lse = _rows(lse, want_lse, q, T, H, dev)
    ws, at, nbytes = _scratch(workspace, _size("la_softmax_prefill_varlen_workspace_size", nseq, T, H, Hkv, d), q, dev)
    _done(lib().la_softmax_prefill_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), nseq, T,
                                          max_seqlen, H, Hkv, d, SCALE if scale is None else scale, out.data_ptr(),
                                          None if lse is None else lse.data_ptr(), at, nbytes, handle),
          "la_softmax_prefill_varlen")
    return out, lse


@_on_stream
def _softmax_prefill_backward_varlen(q, k, v, out, lse, dout, cu_seqlens, max_seqlen, scale, dq, dk, dv, workspace, *,
                                     handle):
    T, H, Hkv, d, dev = _dims(q, k, v)
    _fits(out, "out", _BF16, (T, H, d), dev)
    _fits(lse, "lse", _FP32, (T, H), dev)
    _fits(dout, "dout", _BF16, (T, H, d), dev)
    nseq = _sequences(cu_seqlens, max_seqlen, dev)
    dq, dk, dv = _like(dq, "dq", q, dev), _like(dk, "dk", k, dev), _like(dv, "dv", v, dev)
    ws, at, nbytes = _scratch(workspace,
                              _size("la_softmax_prefill_backward_varlen_workspace_size", nseq, T, H, Hkv, d), q, dev)
    _done(lib().la_softmax_prefill_backward_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                                   lse.data_ptr(), dout.data_ptr(), cu_seqlens.data_ptr(), nseq, T,
                                                   max_seqlen, H, Hkv, d, SCALE if scale is None else scale,
                                                   dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), at, nbytes,
                                                   handle), "la_softmax_prefill_backward_varlen")
    return dq, dk, dv


@_on_stream
def _softmax_prefill_paged(q, k, v, cu_seqlens, max_seqlen, k_cache, v_cache, page_table, cache_lens, scale, out, lse,
                           want_lse, workspace, *, handle):
    T, H, Hkv, d, dev = _dims(q, k, v)
    nseq = _sequences(cu_seqlens, max_seqlen, dev)
    n_pages, page, max_pages = _cache(k_cache, v_cache, page_table, cache_lens, nseq, Hkv, d, dev)
    out = _like(out, "out", q, dev)
    lse = _rows(lse, want_lse, q, T, H, dev)
    nbytes = _size("la_softmax_prefill_paged_workspace_size", nseq, T, H, Hkv, d, page, max_pages)
    ws, at, nbytes = _scratch(workspace, nbytes, q, dev)
    _done(lib().la_softmax_prefill_paged(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), nseq, T,
                                         max_seqlen, H, Hkv, d, SCALE if scale is None else scale, k_cache.data_ptr(),
                                         v_cache.data_ptr(), n_pages, page, page_table.data_ptr(), max_pages,
                                         cache_lens.data_ptr(), out.data_ptr(),
                                         None if lse is None else lse.data_ptr(), at, nbytes, handle),
          "la_softmax_prefill_paged")
    return out, lse


@_on_stream
def _softmax_decode_paged(q, k, v, k_cache, v_cache, page_table, cache_lens, scale, out, out_dtype, lse, want_lse,
                          workspace, *, handle):
    B, H, Hkv, d, dev = _dims(q, k, v)
    n_pages, page, max_pages = _cache(k_cache, v_cache, page_table, cache_lens, B, Hkv, d, dev)
    dtype = out_dtype if out is None else out.dtype
    if dtype is not _BF16 and dtype is not _FP32:
        raise TypeError("out dtype must be torch.bfloat16 or torch.float32")
    if out is None and dtype is _FP32:
        out = q.new_empty((B, H, d), dtype=_FP32)
    elif out is None or dtype is _BF16:
        out = _like(out, "out", q, dev)
    else:
        _fits(out, "out", _FP32, (B, H, d), dev)
    lse = _rows(lse, want_lse, q, B, H, dev)
    nbytes = _size("la_softmax_decode_paged_workspace_size", B, H, Hkv, d, page, max_pages)
    ws, at, nbytes = _scratch(workspace, nbytes, q, dev)
    _done(lib().la_softmax_decode_paged(q.data_ptr(), k.data_ptr(), v.data_ptr(), B, H, Hkv, d,
                                        SCALE if scale is None else scale, k_cache.data_ptr(), v_cache.data_ptr(),
                                        n_pages, page, page_table.data_ptr(), max_pages, cache_lens.data_ptr(),
                                        out.data_ptr(), LA_BF16 if dtype is _BF16 else LA_FP32,
                                        None if lse is None else lse.data_ptr(), at, nbytes, handle),
          "la_softmax_decode_paged")
    return out, lse


@_on_stream
def _cache_copy_pages(k_cache, v_cache, src, dst, *, handle):
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [n_pages, Hkv, page_size, d]")
    dev = k_cache.get_device()
    n_pages, Hkv, page, d = k_cache.shape
    _need(k_cache, "k_cache", _BF16)
    _fits(v_cache, "v_cache", _BF16, k_cache.shape, dev)
    n = src.numel() if isinstance(src, torch.Tensor) else 0
    _fits(src, "src", _INT32, (n,), dev)
    _fits(dst, "dst", _INT32, (n,), dev)
    _done(lib().la_cache_copy_pages(k_cache.data_ptr(), v_cache.data_ptr(), n_pages, page, Hkv, d, src.data_ptr(),
                                    dst.data_ptr(), n, handle), "la_cache_copy_pages")


def softmax_prefill_varlen(q, k, v, cu_seqlens, max_seqlen: int, scale=None, out=None, lse=None, want_lse: bool = True,
                           workspace=None, stream=None):
    """la_softmax_prefill_varlen: causal softmax attention of packed bf16
    q [T, H, d] over k, v [T, Hkv, d] (H a multiple of Hkv) with device int32
    cu_seqlens.  scale: factor of the scores, d**-0.5 by default; stream: the
    device's current one by default.  Returns (out [T, H, d] bf16, lse [T, H]
    fp32 or None)."""
    if stream is None and workspace is None and _module() is not None:
        done = _short(_marshal.prefill_varlen(q, k, v, cu_seqlens, max_seqlen, SCALE if scale is None else scale, out,
                                              lse, want_lse), "la_softmax_prefill_varlen")
        if done is not None:
            return done
    return _softmax_prefill_varlen(q, k, v, cu_seqlens, max_seqlen, scale, out, lse, want_lse, workspace, stream=stream)


def softmax_prefill_backward_varlen(q, k, v, out, lse, dout, cu_seqlens, max_seqlen: int, scale=None, dq=None, dk=None,
                                    dv=None, workspace=None, stream=None):
    """la_softmax_prefill_backward_varlen: gradients of softmax_prefill_varlen
    for dL/dout; out and lse are what that call returned (not joined with results
    over other keys), scale what it was given.  Returns (dq [T, H, d], dk, dv
    [T, Hkv, d]) in bf16."""
    if stream is None and workspace is None and _module() is not None:
        done = _short(_marshal.prefill_backward_varlen(q, k, v, out, lse, dout, cu_seqlens, max_seqlen,
                                                       SCALE if scale is None else scale, dq, dk, dv),
                      "la_softmax_prefill_backward_varlen")
        if done is not None:
            return done
    return _softmax_prefill_backward_varlen(q, k, v, out, lse, dout, cu_seqlens, max_seqlen, scale, dq, dk, dv,
                                            workspace, stream=stream)


def softmax_prefill_paged(q, k, v, cu_seqlens, max_seqlen: int, k_cache, v_cache, page_table, cache_lens, scale=None,
                          out=None, lse=None, want_lse: bool = True, workspace=None, stream=None):
    """la_softmax_prefill_paged: the packed new tokens q [T, H, d], k, v
    [T, Hkv, d] of each sequence are written behind its cache_lens[i] cached
    ones and attend to all of them, causally among themselves.  k_cache,
    v_cache: bf16 [n_pages, Hkv, page_size, d], updated in place; page_table:
    device int32 [nseq, max_pages]; cache_lens: device int32 [nseq], lengths
    before the call.  Returns (out, lse or None)."""
    if stream is None and workspace is None and _module() is not None:
        done = _short(_marshal.prefill_paged(q, k, v, cu_seqlens, max_seqlen, k_cache, v_cache, page_table, cache_lens,
                                             SCALE if scale is None else scale, out, lse, want_lse),
                      "la_softmax_prefill_paged")
        if done is not None:
            return done
    return _softmax_prefill_paged(q, k, v, cu_seqlens, max_seqlen, k_cache, v_cache, page_table, cache_lens, scale, out,
                                  lse, want_lse, workspace, stream=stream)


def softmax_decode_paged(q, k, v, k_cache, v_cache, page_table, cache_lens, scale=None, out=None,
                         out_dtype=torch.bfloat16, lse=None, want_lse: bool = True, workspace=None, stream=None):
    """la_softmax_decode_paged: one new token per request, q [B, H, d], k, v
    [B, Hkv, d], written behind the cache_lens[b] cached ones (-1: no request,
    the row's outputs are left as they are).  The cache as for
    softmax_prefill_paged.  Returns (out [B, H, d] bf16 or fp32, lse [B, H] or
    None)."""
    if stream is None and workspace is None and _module() is not None:
        dtype = out.dtype if isinstance(out, torch.Tensor) else out_dtype
        if dtype is not _BF16 and dtype is not _FP32:
            raise TypeError("out dtype must be torch.bfloat16 or torch.float32")
        done = _short(_marshal.decode_paged(q, k, v, k_cache, v_cache, page_table, cache_lens,
                                            SCALE if scale is None else scale, out, dtype is _FP32, lse, want_lse),
                      "la_softmax_decode_paged")
        if done is not None:
            return done
    return _softmax_decode_paged(q, k, v, k_cache, v_cache, page_table, cache_lens, scale, out, out_dtype, lse,
                                 want_lse, workspace, stream=stream)


def cache_copy_pages(k_cache, v_cache, src, dst, stream=None):
    """la_cache_copy_pages: page src[i] is copied to page dst[i] in both
    tensors [n_pages, Hkv, page_size, d]; src, dst: device int32 [n]."""
    if stream is None and _module() is not None:
        if _short(_marshal.copy_pages(k_cache, v_cache, src, dst), "la_cache_copy_pages") is not None:
            return
    _cache_copy_pages(k_cache, v_cache, src, dst, stream=stream)
