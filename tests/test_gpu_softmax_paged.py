"""Softmax attention on the paged cache against plain attention in 64 bits:
decode steps, prompt chunks, page copies, and the calls that are refused."""
import pytest
import torch

import linear_attention_blocked_b200 as la
from softmax_util import BF16, Cache, attention64, check, packed

pytestmark = pytest.mark.gpu
S = 128 ** -0.5
# the decode kernel's weights meet V as bf16 hi + lo: each p_ts within 2^-16
PAIR = 2.0 ** -16
FP32 = torch.finfo(torch.float32).eps / 2


def decode(past, H, Hkv, page, seed, out_dtype=torch.bfloat16, scale=None):
    B = len(past)
    c = Cache([max(n, 0) for n in past], [1] * B, Hkv, page, seed)
    c.lens = torch.tensor(past, dtype=torch.int32, device="cuda")
    q, k, v, _, _ = packed([B], H, Hkv, seed + 1)
    before_k, before_v = c.k.clone(), c.v.clone()
    out = torch.full(q.shape, 7.0, dtype=out_dtype, device="cuda")
    lse = torch.full((B, H), 7.0, device="cuda")
    la.softmax_decode_paged(q, k, v, c.k, c.v, c.table, c.lens, scale=scale, out=out, lse=lse)
    assert la.get_device_status() == la.LA_OK
    for b, n in enumerate(past):
        if n < 0:
            assert (out[b] == 7).all() and (lse[b] == 7).all()
            continue
        kk, vv = c.read(b, n + 1)
        assert torch.equal(kk[n], k[b]) and torch.equal(vv[n], v[b])     # the new token is cached
        ref = attention64(q[b:b + 1], torch.cat([c.past[b][0], k[b:b + 1]]), torch.cat([c.past[b][1], v[b:b + 1]]), n,
                          S if scale is None else scale)
        check(out[b:b + 1], lse[b:b + 1], ref, n + 1, f"past {n} H={H} Hkv={Hkv} page={page}", p_step=PAIR,
              out_step=BF16 if out_dtype == torch.bfloat16 else FP32)
        before_k[c.table[b, n // page], :, n % page] = k[b]
        before_v[c.table[b, n // page], :, n % page] = v[b]
    # nothing else in the pool has changed
    assert torch.equal(c.k.view(torch.int16), before_k.view(torch.int16))
    assert torch.equal(c.v.view(torch.int16), before_v.view(torch.int16))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", [(8, 1), (4, 4), (64, 8), (6, 2), (40, 2)], ids=str)
def test_decode_matches_plain_attention(heads, page):
    decode([0, 1, 15, 16, 62, 63, 64, 65, 127, 128, 500], *heads, page=page, seed=heads[0] + page)


@pytest.mark.parametrize("heads", [(16, 2), (64, 8), (40, 1)], ids=str)
@pytest.mark.parametrize("past", [[0], [5000], [17000], [3], [-1, 200, -1], [-1], [900, 17]], ids=str)
def test_decode_few_requests(past, heads):
    decode(past, *heads, 32, seed=3 + len(past))


def test_decode_fp32_output_and_scale():
    decode([700, 3, 64], 16, 2, 64, seed=5, out_dtype=torch.float32)
    decode([700, 3, 64], 16, 2, 64, seed=6, out_dtype=torch.float32, scale=0.5)


def test_decode_many_requests():
    decode([(37 * i) % 300 for i in range(333)], 8, 4, 16, seed=9)
    decode([-1 if i % 3 else i for i in range(150)], 4, 1, 64, seed=10)


def test_decode_repeats_bit_for_bit_and_in_a_graph():
    """Replays of a captured step with lengths advanced on the device, two
    graphs sharing one workspace, against the same steps run eagerly."""
    past, H, Hkv, page, steps = [200, 0, 63, 1000], 160, 40, 32, 6  # too many rows for a cluster each
    B = len(past)
    ca, cb = (Cache(past, [steps] * B, Hkv, page, 21) for _ in range(2))
    q, k, v, _, _ = packed([steps * B], H, Hkv, 22)
    want = []
    for s in range(steps):
        a = slice(s * B, (s + 1) * B)
        want.append(la.softmax_decode_paged(q[a].clone(), k[a].clone(), v[a].clone(), ca.k, ca.v, ca.table, ca.lens)[0])
        ca.lens += 1
    qs, ks, vs = q[:B].clone(), k[:B].clone(), v[:B].clone()
    ws = torch.empty(la.lib().la_softmax_decode_paged_workspace_size(B, H, Hkv, 128, page, cb.table.shape[1]), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(qs) for _ in range(2)]
    graphs = []
    for o in outs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            la.softmax_decode_paged(qs, ks, vs, cb.k, cb.v, cb.table, cb.lens, out=o, workspace=ws)
            cb.lens += 1
    for s in range(steps):
        a = slice(s * B, (s + 1) * B)
        for x, y in ((qs, q), (ks, k), (vs, v)):
            x.copy_(y[a])
        graphs[s % 2].replay()
        assert torch.equal(outs[s % 2], want[s]), s
    assert la.get_device_status() == la.LA_OK
    assert torch.equal(ca.k.view(torch.int16), cb.k.view(torch.int16))


@pytest.mark.parametrize("H,Hkv", [(8, 2), (16, 4), (16, 16)])
def test_decode_bad_pages_and_lengths(H, Hkv):
    past, page = [40, 40, 40, 40], 16
    c = Cache(past, [1] * 4, Hkv, page, 31)
    q, k, v, _, _ = packed([4], H, Hkv, 32)
    want, _ = la.softmax_decode_paged(q, k, v, c.k, c.v, c.table, c.lens)
    assert la.get_device_status() == la.LA_OK
    for bad in (-1, c.n_pages, 1 << 30, -(1 << 31)):
        for slot in (0, 2):  # a page of old tokens, and that of the new one
            table = c.table.clone()
            table[1, slot] = bad
            kc, vc = c.k.clone(), c.v.clone()
            kc[:], vc[:] = torch.nan_to_num(kc), torch.nan_to_num(vc)  # page 0 stands in: keep it finite
            got, _ = la.softmax_decode_paged(q, k, v, kc, vc, table, c.lens)
            assert la.get_device_status() == la.LA_ERR_INVALID_ARGUMENT
            for b in (0, 2, 3):
                assert torch.equal(got[b], want[b])
    lens = torch.tensor([40, -2, c.table.shape[1] * page, 40], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    la.softmax_decode_paged(q, k, v, c.k, c.v, c.table, lens, out=out)
    assert la.get_device_status() == la.LA_ERR_INVALID_ARGUMENT
    assert torch.equal(out[0], want[0]) and torch.equal(out[3], want[3])
    assert (out[1] == 7).all() and (out[2] == 7).all()
    assert la.get_device_status() == la.LA_OK


def chunk(new, past, H, Hkv, page, seed):
    c = Cache(past, new, Hkv, page, seed)
    q, k, v, cu, cu_dev = packed(new, H, Hkv, seed + 1)
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    la.softmax_prefill_paged(q, k, v, cu_dev, max(new), c.k, c.v, c.table, c.lens, out=out, lse=lse)
    assert la.get_device_status() == la.LA_OK
    for b, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
        kk, vv = c.read(b, past[b] + e - a)
        assert torch.equal(kk[past[b]:], k[a:e]) and torch.equal(vv[past[b]:], v[a:e])
        assert torch.equal(kk[:past[b]], c.past[b][0])
        if e > a:
            ref = attention64(q[a:e], torch.cat([c.past[b][0], k[a:e]]), torch.cat([c.past[b][1], v[a:e]]), past[b], S)
            check(out[a:e], lse[a:e], ref, past[b] + e - a, f"new {e - a} past {past[b]} page {page}")


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", [(8, 1), (3, 3), (64, 8)], ids=str)
def test_chunks_match_plain_attention(heads, page):
    chunk([1, 0, 130, 128, 61, 300], [0, 50, 127, 128, 500, 1001], *heads, page=page, seed=heads[0] + page)


def test_chunk_bad_lengths_refuse_the_call():
    c = Cache([10, 20], [5, 5], 2, 16, 41)
    q, k, v, cu, cu_dev = packed([5, 5], 4, 2, 42)
    kc = c.k.clone()
    for lens in ([-1, 20], [10, c.table.shape[1] * 16 - 4], [2 ** 31 - 1, 20]):
        out = torch.full_like(q, 7.0)
        la.softmax_prefill_paged(q, k, v, cu_dev, 5, c.k, c.v, c.table,
                                 torch.tensor(lens, dtype=torch.int32, device="cuda"), out=out)
        assert la.get_device_status() == la.LA_ERR_INVALID_ARGUMENT
        assert (out == 7).all() and torch.equal(c.k.view(torch.int16), kc.view(torch.int16))
    table = c.table.clone()
    table[0, 0] = c.n_pages
    kc, vc = torch.nan_to_num(c.k), torch.nan_to_num(c.v)
    want, _ = la.softmax_prefill_paged(q, k, v, cu_dev, 5, kc.clone(), vc.clone(), c.table, c.lens)
    got, _ = la.softmax_prefill_paged(q, k, v, cu_dev, 5, kc, vc, table, c.lens)
    assert la.get_device_status() == la.LA_ERR_INVALID_ARGUMENT
    assert torch.equal(got[5:], want[5:])


@pytest.mark.parametrize("page,Hkv", [(16, 1), (32, 3), (128, 8)])
def test_copied_pages(page, Hkv):
    g = torch.Generator(device="cuda").manual_seed(page)
    kc, vc = (torch.randn(50, Hkv, page, 128, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    ids = torch.randperm(50, generator=g, device="cuda").to(torch.int32)
    want_k, want_v = kc.clone(), vc.clone()
    src, dst = ids[:20].contiguous(), ids[20:40].contiguous()
    src[7] = src[3]  # a page may be copied twice
    want_k[dst.long()], want_v[dst.long()] = kc[src.long()], vc[src.long()]
    la.cache_copy_pages(kc, vc, src, dst)
    assert la.get_device_status() == la.LA_OK
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    la.cache_copy_pages(kc, vc, src[:0], dst[:0])
    bad = dst.clone()
    bad[2], bad[5] = 50, -1
    src[4] = 50
    kc2, vc2 = kc.clone(), vc.clone()
    la.cache_copy_pages(kc2, vc2, src, bad)
    assert la.get_device_status() == la.LA_ERR_INVALID_ARGUMENT
    keep = [i for i in range(20) if i not in (2, 4, 5)]
    kc[dst[keep].long()] = kc[src[keep].long()]
    assert torch.equal(kc2, kc)


@pytest.mark.parametrize("heads", [(8, 1), (16, 16), (24, 2)], ids=str)
def test_decode_in_every_form(heads):
    """The batch's size and the table's width choose between clusters per row and
    runs of tiles: widths and batches on both sides of each border."""
    for B, longest in [(1, 200), (1, 4500), (1, 33000), (2, 2100), (3, 9000), (5, 20000), (9, 3000), (17, 2500),
                       (40, 1500), (130, 300), (260, 90)]:
        past = [(longest * 7919 * (i + 1)) % (longest + 1) for i in range(B)]
        past[-1] = longest
        decode(past, *heads, page=128 if longest > 1000 else 32, seed=B)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("heads", [(8, 1), (1, 1), (6, 2), (16, 2)], ids=str)
def test_chunks_behind_long_caches(heads, page):
    """Few new tokens, many cached ones: equal runs of key tiles, cut items joined."""
    chunk([5], [9000], *heads, page=page, seed=50 + page)
    chunk([1, 0, 40, 130], [4000, 0, 2500, 1], *heads, page=page, seed=60 + page)
    chunk([257], [6001], *heads, page=page, seed=70 + page)
