"""Values that are not finite, in decode steps and in gradients: what they reach and
what they leave as it is."""
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


@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("at", [20, 200, 399])
@pytest.mark.parametrize("heads", [(4, 2), (3, 3), (8, 1)], ids=str)
def test_a_bad_output_gradient_stays_out_of_later_keys(heads, at, bad):
    """dout of row `at` has no part in dk of later rows, nor in dq of other rows, nor in
    dv of rows in later blocks of 128 or of other features: bit for bit what it is with
    any other value there."""
    q, k, v, _, cu = packed([400], *heads, seed=65)
    g = torch.randn_like(q)
    out, lse = la.softmax_prefill_varlen(q, k, v, cu, 400)
    want = la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu, 400)
    g[at, 0, 3] = bad
    dq, dk, dv = la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu, 400)
    assert la.get_device_status() == la.LA_OK
    others = torch.arange(400, device="cuda") != at
    assert torch.equal(dq[others], want[0][others]) and torch.equal(dq[at, 1:], want[0][at, 1:])
    assert torch.equal(dk[at + 1:], want[1][at + 1:])
    assert torch.equal(dk[:, 1:], want[1][:, 1:]) and torch.equal(dv[:, 1:], want[2][:, 1:])
    block = (at // 128 + 1) * 128
    assert torch.equal(dv[block:], want[2][block:])
    features = torch.arange(128, device="cuda") != 3
    assert torch.equal(dv[..., features], want[2][..., features])
    # and what it reaches, it reaches
    assert not torch.isfinite(dq[at, 0]).any() and not torch.isfinite(dk[:at + 1, 0]).any()
    assert not torch.isfinite(dv[:at + 1, 0, 3]).any()


@pytest.mark.parametrize("bad", [INF, NAN])
@pytest.mark.parametrize("at", [20, 200, 399])
@pytest.mark.parametrize("heads", [(4, 2), (3, 3), (8, 1)], ids=str)
def test_a_bad_query_or_key_reaches_one_feature_of_its_block(heads, at, bad):
    """q of row `at` may reach its feature of dk of later rows, k its feature of dq of
    earlier ones, in the same 128 rows; nothing else of the rows that do not see it."""
    q, k, v, _, cu = packed([400], *heads, seed=67)
    g = torch.randn_like(q)

    def grads(q, k):
        out, lse = la.softmax_prefill_varlen(q, k, v, cu, 400)
        return la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu, 400)
    want = grads(q, k)
    features = torch.arange(128, device="cuda") != 3
    q2, k2 = q.clone(), k.clone()
    q2[at, 0, 3] = bad
    dq, dk, dv = grads(q2, k)
    others = torch.arange(400, device="cuda") != at
    block = (at // 128 + 1) * 128
    assert torch.equal(dq[others], want[0][others]) and torch.equal(dv[at + 1:], want[2][at + 1:])
    assert torch.equal(dk[block:], want[1][block:])
    assert torch.equal(dk[at + 1:][..., features], want[1][at + 1:][..., features])
    k2[at, 0, 3] = bad
    dq, _, _ = grads(q, k2)
    assert torch.equal(dq[:at // 128 * 128], want[0][:at // 128 * 128])
    assert torch.equal(dq[:at][..., features], want[0][:at][..., features])
    assert torch.equal(dq[:, heads[0] // heads[1]:], want[0][:, heads[0] // heads[1]:])
    assert la.get_device_status() == la.LA_OK
