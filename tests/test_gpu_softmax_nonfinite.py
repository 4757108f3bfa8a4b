"""Values that are not finite, in decode steps: what they reach and what they leave as
it is."""
import pytest
import torch

import linear_attention_blocked_b200 as la
from softmax_util import Cache, attention64, check, packed

pytestmark = pytest.mark.gpu
S = 128 ** -0.5
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("heads", [(8, 1), (16, 1), (6, 2), (40, 2)], ids=str)
@pytest.mark.parametrize("past", [[5], [300], [300, 70, 9], [40000], [1500] * 40], ids=lambda p: f"{len(p)}x{p[0]}")
def test_infinite_values_in_a_decode_step(past, heads, out_dtype):
    """An infinite value with a weight above zero makes the sum infinite, with its
    sign; values of both signs make it NaN; the other features are not touched."""
    B, Hkv = len(past), heads[1]
    c = Cache(past, [1] * B, Hkv, 128 if past[0] > 10000 else 16, 61)
    q, k, v, _, _ = packed([B], *heads, seed=62)
    for b, n in enumerate(past):
        # heavy and light weights, the first and the last cached token and the new one
        kk, vv = c.past[b]
        for at, feature, bad in ((0, 5, INF), (n - 1, 7, -INF), (n // 2, 9, INF), (n // 3, 9, -INF), (n // 2, 11, NAN),
                                 (n // 4, 13, -INF), (n // 5, 13, -INF)):
            vv[at, :, feature] = bad
        v[b, :, 6] = INF
        v[b, :, 8] = -INF
        c.write(b, 0, kk, vv)
    out, lse = la.softmax_decode_paged(q, k, v, c.k, c.v, c.table, c.lens, out_dtype=out_dtype)
    assert la.get_device_status() == la.LA_OK
    for feature, bad in ((5, INF), (6, INF), (7, -INF), (8, -INF), (13, -INF)):
        assert (out[..., feature] == bad).all(), (feature, out[..., feature])
    for feature in (9, 11):
        assert torch.isnan(out[..., feature]).all()
    for b, n in enumerate(past[:3]):
        vv = torch.cat([c.past[b][1], v[b:b + 1]]).nan_to_num(0.0, 0.0, 0.0)
        got = out[b:b + 1].clone()
        ref = attention64(q[b:b + 1], torch.cat([c.past[b][0], k[b:b + 1]]), vv, n, S)
        for feature in (5, 6, 7, 8, 9, 11, 13):
            got[..., feature] = 0
            ref[0][..., feature] = 0
        check(got, lse[b:b + 1], ref, n + 1, p_step=2.0 ** -16,
              out_step=torch.finfo(out_dtype).eps / 2)


@pytest.mark.parametrize("heads", [(8, 1), (16, 1)], ids=str)
def test_a_token_alone_and_as_a_chunk_agree_on_infinities(heads):
    c = Cache([700], [1], heads[1], 32, 63)
    kk, vv = c.past[0]
    vv[123, :, ::3] = INF
    vv[456, :, 1::3] = -INF
    c.write(0, 0, kk, vv)
    q, k, v, _, cu = packed([1], *heads, seed=64)
    a, _ = la.softmax_decode_paged(q, k, v, c.k, c.v, c.table, c.lens)
    b, _ = la.softmax_prefill_paged(q, k, v, cu, 1, c.k, c.v, c.table, c.lens)
    assert la.get_device_status() == la.LA_OK
    for x in (a, b):
        assert (x[..., ::3] == INF).all() and (x[..., 1::3] == -INF).all() and torch.isfinite(x[..., 2::3]).all()
