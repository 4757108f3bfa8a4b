"""Softmax attention at the edges of what its calls allow: tensors of more than
2^31 elements, no tokens, thousands of sequences, values that are not finite,
calls that run at once."""
import pytest
import torch

import linear_attention_blocked_b200 as la
from softmax_util import BF16, Cache, attention64, check, gradients64, packed

pytestmark = pytest.mark.gpu
S = 128 ** -0.5


def test_tensors_beyond_32_bit_offsets():
    """q, out and their gradients of 2.3e9 elements; the last sequences checked."""
    n, count, H, Hkv = 141, 1000, 128, 16
    T = n * count
    assert T * H * 128 > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    q, dout = (torch.randn(T, H, 128, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    k, v = (torch.randn(T, Hkv, 128, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    cu = torch.arange(0, T + 1, n, dtype=torch.int32, device="cuda")
    out, lse = la.softmax_prefill_varlen(q, k, v, cu, n)
    dq, dk, dv = la.softmax_prefill_backward_varlen(q, k, v, out, lse, dout, cu, n)
    assert la.get_device_status() == la.LA_OK
    for i in (0, count // 2, count - 1):
        a = slice(i * n, (i + 1) * n)
        check(out[a], lse[a], attention64(q[a], k[a], v[a], 0, S), n, f"sequence {i}")
        for name, (want, bound) in gradients64(q[a], k[a], v[a], dout[a], S).items():
            got = {"q": dq, "k": dk, "v": dv}[name][a]
            assert ((got.double() - want).abs() <= bound).all(), (i, name)


def test_caches_beyond_32_bit_offsets():
    """A pool of 2.3e9 elements; the requests' pages lie at its end."""
    Hkv, page, pages = 64, 128, 2200
    assert pages * Hkv * page * 128 > 2 ** 31
    kc, vc = (torch.zeros(pages, Hkv, page, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    past, new = [300, 129], [40, 1]
    c = Cache(past, [60, 60], Hkv, page, 3, spare=0)
    shift = pages - c.n_pages
    kc[shift:], vc[shift:] = c.k, c.v
    valid = c.table < c.n_pages
    c.table[valid] += shift
    c.k, c.v, c.n_pages = kc, vc, pages
    q, k, v, cu, cu_dev = packed(new, 64, Hkv, 4)
    out, lse = la.softmax_prefill_paged(q, k, v, cu_dev, 40, kc, vc, c.table, c.lens)
    for b in range(2):
        a = slice(cu[b], cu[b + 1])
        ref = attention64(q[a], torch.cat([c.past[b][0], k[a]]), torch.cat([c.past[b][1], v[a]]), past[b], S)
        check(out[a], lse[a], ref, past[b] + new[b])
    c.lens += torch.tensor(new, dtype=torch.int32, device="cuda")
    q2, k2, v2, _, _ = packed([2], 64, Hkv, 5)
    out, lse = la.softmax_decode_paged(q2, k2, v2, kc, vc, c.table, c.lens)
    for b in range(2):
        n = past[b] + new[b]
        kk, vv = c.read(b, n + 1)
        assert torch.equal(kk[n], k2[b]) and torch.equal(vv[n], v2[b])
        check(out[b:b + 1], lse[b:b + 1], attention64(q2[b:b + 1], kk, vv, n, S), n + 1, p_step=2.0 ** -16)
    src = c.table[0, :1].clone()
    la.cache_copy_pages(kc, vc, src, torch.zeros_like(src))
    assert la.get_device_status() == la.LA_OK
    assert torch.equal(kc[0], kc[src.long()[0]]) and torch.equal(vc[0], vc[src.long()[0]])


def test_no_tokens():
    empty = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    kv = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    for seqs in (0, 1, 5):
        cu = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
        out, lse = la.softmax_prefill_varlen(empty, kv, kv, cu, 0)
        assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
        grads = la.softmax_prefill_backward_varlen(empty, kv, kv, out, lse, empty, cu, 0)
        assert [x.shape[0] for x in grads] == [0, 0, 0]
    c = Cache([20], [0], 2, 16, 1)
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    la.softmax_prefill_paged(empty, kv, kv, cu, 0, c.k, c.v, c.table, c.lens)
    out, _ = la.softmax_decode_paged(empty, kv, kv, c.k, c.v, c.table[:0], c.lens[:0])
    assert out.shape == (0, 8, 128)
    assert la.get_device_status() == la.LA_OK


def test_thousands_of_sequences():
    lens = [(i * 37) % 9 for i in range(6000)]
    q, k, v, cu, cu_dev = packed(lens, 4, 2, 9)
    g = torch.randn_like(q)
    out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, 8)
    got = la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu_dev, 8)
    assert la.get_device_status() == la.LA_OK
    for i in (0, 1, 2, 1023, 1024, 3000, 5997, 5998, 5999):
        a = slice(cu[i], cu[i + 1])
        if cu[i] == cu[i + 1]:
            continue
        check(out[a], lse[a], attention64(q[a], k[a], v[a], 0, S), 8)
        for x, (want, bound) in zip(got, gradients64(q[a], k[a], v[a], g[a], S).values()):
            assert ((x[a].double() - want).abs() <= bound).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite_show(bad):
    """A query, key or value that is not finite makes the rows that see it not
    finite, and no row of an earlier tile."""
    for which in range(3):
        x = list(packed([400], 4, 2, 13)[:3])
        cu = torch.tensor([0, 400], dtype=torch.int32, device="cuda")
        x[which][200, 1 if which else 2, 5] = bad
        out, _ = la.softmax_prefill_varlen(*x, cu, 400)
        hit = out[:, 2] if which else out[200:201, 2]
        assert torch.isfinite(out[:128]).all() and torch.isfinite(out[:, :2]).all()
        if which == 0:
            assert not torch.isfinite(hit).all()
        elif which == 1:
            # a key with an infinite score takes all weight or none; NaN reaches every later row
            assert bad == float("inf") or not torch.isfinite(hit[200:]).all(-1).any()
        else:
            assert not torch.isfinite(hit[200:, 5]).any()


def test_calls_at_once_on_two_streams():
    """The same calls on two streams, each with what it allocates itself, against
    one after the other."""
    lens = [700, 40, 300]
    sets = []
    for seed in (1, 2):
        q, k, v, cu, cu_dev = packed(lens, 16, 2, seed)
        c = Cache([500, 30, 900], [1, 1, 1], 2, 32, seed)
        sets.append((q, k, v, cu_dev, torch.randn_like(q), c))

    def all_calls(s, stream=None):
        q, k, v, cu_dev, g, c = s
        out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, 700, stream=stream)
        grads = la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu_dev, 700, stream=stream)
        dec = la.softmax_decode_paged(q[:3], k[:3], v[:3], c.k, c.v, c.table, c.lens, stream=stream)
        return [out, lse, *grads, *dec]
    want = [all_calls(s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for st in streams:
            st.wait_stream(torch.cuda.current_stream())
        got = [all_calls(s, st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            for a, b in zip(x, y):
                assert torch.equal(a, b)
    assert la.get_device_status() == la.LA_OK


def test_keys_whose_scores_are_all_minus_infinity():
    """The first keys of a row, more than a tile of them, score -inf: they have no
    weight, and the row is that of the keys behind them.  A row with no others has
    no result."""
    def lower(q, k, first):
        q[..., 0] = q[..., 0].abs() + 0.5
        k[:first, :, 0] = float("-inf")

    for lens, first, heads in (([400], 130, (8, 2)), ([3001], 1500, (2, 1))):
        q, k, v, _, cu = packed(lens, *heads, 21)
        lower(q, k, first)
        out, lse = la.softmax_prefill_varlen(q, k, v, cu, lens[0])
        check(out[first:], lse[first:], attention64(q[first:], k[first:], v[first:], 0, S), lens[0])
        assert torch.isnan(out[:first]).all() and (lse[:first] == float("-inf")).all()
    for new, past, first in ((20, 700, 300), (20, 5000, 4000)):
        c = Cache([past], [new + 1], 1, 32, 22)
        q, k, v, _, cu = packed([new], 8, 1, 23)
        lower(q, c.past[0][0], first)
        c.write(0, 0, *c.past[0])
        out, lse = la.softmax_prefill_paged(q, k, v, cu, new, c.k, c.v, c.table, c.lens)
        kk, vv = c.read(0, past + new)
        check(out, lse, attention64(q, kk[first:], vv[first:], past - first, S), past + new)
        c.lens += new
        dec, dlse = la.softmax_decode_paged(q[:1], k[:1], v[:1], c.k, c.v, c.table, c.lens)
        kk, vv = c.read(0, past + new + 1)
        check(dec, dlse, attention64(q[:1], kk[first:], vv[first:], past + new - first, S), past + new + 1,
              p_step=2.0 ** -16)
    assert la.get_device_status() == la.LA_OK


def test_tensors_aligned_to_16_bytes_only():
    """Every tensor 16 bytes behind a 32-byte boundary: the same bits."""
    def shifted(x):
        buf = torch.empty(x.numel() + 8, dtype=x.dtype, device="cuda")
        return buf[8:].view(x.shape).copy_(x)

    q, k, v, _, cu = packed([300, 5, 0, 129], 6, 2, 31)
    g = torch.randn_like(q)
    out, lse = la.softmax_prefill_varlen(q, k, v, cu, 300)
    want = la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu, 300)
    q2, k2, v2, g2 = (shifted(x) for x in (q, k, v, g))
    out2, _ = la.softmax_prefill_varlen(q2, k2, v2, cu, 300, out=shifted(torch.zeros_like(q)), lse=torch.empty_like(lse))
    got = la.softmax_prefill_backward_varlen(q2, k2, v2, out2, lse, g2, cu, 300, dq=shifted(torch.zeros_like(q)),
                                             dk=shifted(torch.zeros_like(k)), dv=shifted(torch.zeros_like(v)))
    assert la.get_device_status() == la.LA_OK
    assert all(x.data_ptr() % 32 == 16 for x in (out2, *got))
    for x, y in zip((out2, *got), (out, *want)):
        assert torch.equal(x, y)
