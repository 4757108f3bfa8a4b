"""Argument errors of the softmax-attention entry points, which need no GPU: each
call below fails its checks before anything is launched."""
import ctypes

import pytest

import linear_attention_blocked_b200 as la
from linear_attention_blocked_b200 import _build

V = ctypes.c_void_p
A = 0x10000           # never dereferenced
FAR = 1 << 40
INVALID, UNSUPPORTED, WORKSPACE = la.LA_ERR_INVALID_ARGUMENT, la.LA_ERR_UNSUPPORTED, la.LA_ERR_WORKSPACE
BIG = 300000          # tokens that need a workspace


@pytest.fixture(scope="module")
def L():
    _build.build()
    return la.lib()


def prefill(L, q=A, k=FAR, v=2 * FAR, cu=3 * FAR, nseq=1, T=128, longest=128, H=8, Hkv=2, d=128, scale=0.1, out=4 * FAR,
            lse=5 * FAR, ws=6 * FAR, n=1 << 40):
    return L.la_softmax_prefill_varlen(V(q), V(k), V(v), V(cu), nseq, T, longest, H, Hkv, d, scale, V(out), V(lse),
                                       V(ws), n, None)


def backward(L, q=A, k=FAR, v=2 * FAR, out=3 * FAR, lse=4 * FAR, dout=5 * FAR, cu=6 * FAR, nseq=1, T=128, longest=128,
             H=8, Hkv=2, d=128, scale=0.1, dq=7 * FAR, dk=8 * FAR, dv=9 * FAR, ws=10 * FAR, n=1 << 40):
    return L.la_softmax_prefill_backward_varlen(V(q), V(k), V(v), V(out), V(lse), V(dout), V(cu), nseq, T, longest, H,
                                                Hkv, d, scale, V(dq), V(dk), V(dv), V(ws), n, None)


def chunk(L, q=A, k=FAR, v=2 * FAR, cu=3 * FAR, nseq=1, T=128, longest=128, H=8, Hkv=2, d=128, scale=0.1, kc=4 * FAR,
          vc=5 * FAR, n_pages=10, page=16, table=6 * FAR, max_pages=5, lens=7 * FAR, out=8 * FAR, lse=9 * FAR,
          ws=10 * FAR, n=1 << 40):
    return L.la_softmax_prefill_paged(V(q), V(k), V(v), V(cu), nseq, T, longest, H, Hkv, d, scale, V(kc), V(vc), n_pages,
                                      page, V(table), max_pages, V(lens), V(out), V(lse), V(ws), n, None)


def decode(L, q=A, k=FAR, v=2 * FAR, B=4, H=8, Hkv=2, d=128, scale=0.1, kc=4 * FAR, vc=5 * FAR, n_pages=10, page=16,
           table=6 * FAR, max_pages=5, lens=7 * FAR, out=8 * FAR, dtype=0, lse=9 * FAR, ws=10 * FAR, n=1 << 40):
    return L.la_softmax_decode_paged(V(q), V(k), V(v), B, H, Hkv, d, scale, V(kc), V(vc), n_pages, page, V(table),
                                     max_pages, V(lens), V(out), dtype, V(lse), V(ws), n, None)


@pytest.mark.parametrize("call", [prefill, backward, chunk, decode])
def test_shapes_scale_and_pointers(L, call):
    assert call(L, d=64) == UNSUPPORTED
    assert call(L, H=7) == INVALID                  # not a multiple of Hkv
    assert call(L, H=0) == INVALID
    assert call(L, Hkv=0) == INVALID
    for scale in (0.0, -0.1, float("nan"), float("inf")):
        assert call(L, scale=scale) == INVALID
    for name in ("q", "k", "v", "out"):
        assert call(L, **{name: 0}) == INVALID
        assert call(L, **{name: A + 8}) == INVALID  # not 16-byte aligned
    assert call(L, lse=4 * FAR + 2) == INVALID


@pytest.mark.parametrize("call", [prefill, backward, chunk])
def test_sequences(L, call):
    assert call(L, nseq=-1) == INVALID
    assert call(L, T=-1) == INVALID
    assert call(L, longest=-1) == INVALID
    assert call(L, nseq=0) == INVALID               # tokens without a sequence
    assert call(L, nseq=0, T=0) == la.LA_OK
    assert call(L, cu=0) == INVALID
    assert call(L, cu=3 * FAR + 2) == INVALID


def test_overlaps(L):
    assert prefill(L, out=A) == INVALID
    assert prefill(L, out=FAR + 64) == INVALID
    assert prefill(L, lse=2 * FAR) == INVALID
    assert prefill(L, lse=4 * FAR + 4) == INVALID
    for name in ("dq", "dk", "dv"):
        for other in (A, FAR, 2 * FAR, 3 * FAR, 4 * FAR, 5 * FAR):
            assert backward(L, **{name: other}) == INVALID
    assert backward(L, dk=7 * FAR) == INVALID
    assert backward(L, ws=9 * FAR) == INVALID
    for call in (chunk, decode):
        assert call(L, out=4 * FAR) == INVALID      # over the cache
        assert call(L, q=5 * FAR) == INVALID
        assert call(L, k=4 * FAR) == INVALID
        assert call(L, vc=4 * FAR + 4096) == INVALID


@pytest.mark.parametrize("call", [chunk, decode])
def test_caches(L, call):
    assert call(L, page=48) == UNSUPPORTED
    assert call(L, page=256) == UNSUPPORTED
    assert call(L, page=0) == INVALID
    assert call(L, n_pages=0) == INVALID
    assert call(L, max_pages=0) == INVALID
    for name in ("kc", "vc", "table", "lens"):
        assert call(L, **{name: 0}) == INVALID
    assert call(L, kc=4 * FAR + 8) == INVALID
    assert call(L, n_pages=1 << 30, page=128) == UNSUPPORTED
    assert call(L, max_pages=1 << 30, page=128) == UNSUPPORTED


def test_workspaces(L):
    size = L.la_softmax_prefill_varlen_workspace_size
    assert size(1, 128, 8, 2, 128) == 0             # few tiles: none needed
    need = size(1, BIG, 8, 2, 128)
    assert need > 0 and size(1, BIG, 8, 3, 128) == 0
    assert prefill(L, T=BIG, longest=BIG, n=need - 1) == WORKSPACE
    assert prefill(L, T=BIG, longest=BIG, ws=0) == WORKSPACE
    assert prefill(L, T=BIG, longest=BIG, ws=6 * FAR + 16, n=need) == INVALID
    need = L.la_softmax_prefill_backward_varlen_workspace_size(1, 128, 8, 2, 128)
    assert backward(L, n=need - 1) == WORKSPACE and backward(L, ws=0) == WORKSPACE
    need = L.la_softmax_prefill_paged_workspace_size(1, BIG, 8, 2, 128, 16, 1 << 15)
    assert chunk(L, T=BIG, longest=BIG, n=need - 1, n_pages=1 << 16, max_pages=1 << 15) == WORKSPACE
    size = L.la_softmax_decode_paged_workspace_size
    assert size(4, 8, 2, 128, 16, 5) == size(400, 8, 2, 128, 16, 5) == 0   # short rows: none needed
    need = size(400, 8, 2, 128, 128, 512)
    assert need > 0 and size(1, 8, 2, 128, 128, 4096) == need
    long = dict(B=400, page=128, max_pages=512)
    assert decode(L, n=need - 1, **long) == WORKSPACE and decode(L, ws=0, **long) == WORKSPACE


def test_decode_and_copies(L):
    assert decode(L, B=-1) == INVALID
    assert decode(L, B=0) == la.LA_OK
    assert decode(L, dtype=7) == INVALID

    def copy(kc=A, vc=FAR, n_pages=10, page=16, Hkv=2, d=128, src=2 * FAR, dst=3 * FAR, n=4):
        return L.la_cache_copy_pages(V(kc), V(vc), n_pages, page, Hkv, d, V(src), V(dst), n, None)
    assert copy(n=0) == la.LA_OK
    assert copy(n=-1) == INVALID
    assert copy(d=64) == UNSUPPORTED
    assert copy(page=24) == UNSUPPORTED
    assert copy(n_pages=0) == INVALID
    assert copy(Hkv=0) == INVALID
    assert copy(vc=A + 4096) == INVALID
    for name in ("kc", "vc", "src", "dst"):
        assert copy(**{name: 0}) == INVALID
    assert copy(src=2 * FAR + 1) == INVALID


def test_cpu_tensors_are_refused():
    import torch
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        la.softmax_prefill_varlen(q, q, q, cu, 4)
    with pytest.raises(ValueError):
        la.cache_copy_pages(q, q, cu, cu)
