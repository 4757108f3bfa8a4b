"""la_softmax_prefill_varlen against plain attention in 64 bits: group sizes,
ragged lengths around the 128-row tiles, masks, isolation and refusals."""
import pytest
import torch

import linear_attention_blocked_b200 as la
from softmax_util import attention64, check, packed

pytestmark = pytest.mark.gpu
S = 128 ** -0.5


def run_and_check(lens, H, Hkv, seed, scale=None, spread=1.5):
    q, k, v, cu, cu_dev = packed(lens, H, Hkv, seed, scale=spread)
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    la.softmax_prefill_varlen(q, k, v, cu_dev, max(lens, default=0), scale=scale, out=out, lse=lse)
    assert la.get_device_status() == la.LA_OK
    for a, b in zip(cu[:-1], cu[1:]):
        if a == b:
            continue
        ref = attention64(q[a:b], k[a:b], v[a:b], 0, S if scale is None else scale)
        check(out[a:b], lse[a:b], ref, b - a, f"{lens} H={H} Hkv={Hkv} tokens {a}-{b}")
    return q, k, v, cu_dev, out, lse


@pytest.mark.parametrize("heads", [(8, 1), (8, 8), (6, 2), (5, 1), (2, 1), (64, 8)], ids=str)
@pytest.mark.parametrize("lens", [[1], [2, 1], [127], [128], [129], [255, 0, 257], [300, 1, 0, 640, 17]], ids=str)
def test_matches_plain_attention(lens, heads):
    run_and_check(lens, *heads, seed=len(lens) * 1000 + heads[0])


def test_long_rows_and_many_items():
    run_and_check([4097, 1, 2500], 16, 2, seed=5)


def test_scale_and_growing_maximum():
    """Scores that climb along the keys: the running maximum is replaced, and
    O rescaled, in most tiles; and a scale of its own."""
    q, k, v, cu, cu_dev = packed([1100], 4, 2, seed=7)
    ramp = torch.linspace(0.2, 6.0, 1100, device="cuda")[:, None, None]
    k = (torch.ones_like(k) * ramp).bfloat16()
    q = q.abs()
    for scale in (S, 0.02, 1.0):
        out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, 1100, scale=scale)
        assert la.get_device_status() == la.LA_OK
        check(out, lse, attention64(q, k, v, 0, scale), 1100, f"scale {scale}")


def test_sequences_do_not_see_each_other():
    """NaN and infinities in one sequence leave its neighbours' rows bit for
    bit as they are, whatever tile they share."""
    lens = [70, 130, 200]
    q, k, v, cu, cu_dev = packed(lens, 4, 2, seed=11)
    want, want_lse = la.softmax_prefill_varlen(q, k, v, cu_dev, 200)
    for bad in (float("nan"), float("inf"), -float("inf")):
        for seq in (0, 1, 2):
            q2, k2, v2 = q.clone(), k.clone(), v.clone()
            for x in (q2, k2, v2):
                x[cu[seq]:cu[seq + 1]] = bad
            out, lse = la.softmax_prefill_varlen(q2, k2, v2, cu_dev, 200)
            for other in range(3):
                if other != seq:
                    a, b = cu[other], cu[other + 1]
                    assert torch.equal(out[a:b], want[a:b]) and torch.equal(lse[a:b], want_lse[a:b])
    assert la.get_device_status() == la.LA_OK


def test_same_call_twice_is_bit_identical_and_without_lse():
    q, k, v, cu, cu_dev = packed([700, 333], 8, 2, seed=13)
    out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, 700)
    again, none = la.softmax_prefill_varlen(q, k, v, cu_dev, 700, want_lse=False)
    assert none is None and torch.equal(out, again)


def test_side_stream_and_captured_graph():
    q, k, v, cu, cu_dev = packed([500, 40], 8, 2, seed=17)
    want, _ = la.softmax_prefill_varlen(q, k, v, cu_dev, 500)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = la.softmax_prefill_varlen(q, k, v, cu_dev, 500, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.softmax_prefill_varlen(q, k, v, cu_dev, 500, out=out)
    q.copy_(torch.randn_like(q))
    want, _ = la.softmax_prefill_varlen(q, k, v, cu_dev, 500)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_bad_tables_are_refused_on_the_device():
    q, k, v, cu, cu_dev = packed([100, 60], 4, 2, seed=19)
    for table in ([0, 100, 159], [1, 100, 160], [0, 161, 160], [0, 120, 160], [0, -5, 160]):
        out = torch.full_like(q, 3.0)
        la.softmax_prefill_varlen(q, k, v, torch.tensor(table, dtype=torch.int32, device="cuda"), 100, out=out)
        assert la.get_device_status() == la.LA_ERR_INVALID_ARGUMENT
        assert (out == 3.0).all()
    assert la.get_device_status() == la.LA_OK


def test_rejected_calls():
    q, k, v, cu, cu_dev = packed([64], 4, 2, seed=23)
    with pytest.raises(ValueError):
        la.softmax_prefill_varlen(q[:, :3].contiguous(), k, v, cu_dev, 64)   # 3 heads over 2
    with pytest.raises(TypeError):
        la.softmax_prefill_varlen(q.float(), k, v, cu_dev, 64)
    with pytest.raises(ValueError):
        la.softmax_prefill_varlen(q.transpose(0, 1), k, v, cu_dev, 64)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(la.LAError):
            la.softmax_prefill_varlen(q, k, v, cu_dev, 64, scale=scale)
    with pytest.raises(la.LAError):
        la.softmax_prefill_varlen(q, k, v, cu_dev, 64, out=q)


def test_both_orders_of_the_work():
    """Items by length (few tokens) and by head (many), with empty sequences and
    lengths that tie, give the same rows."""
    lens = [130, 0, 700, 129, 700, 1, 0, 1025]
    for H, Hkv in ((64, 64), (64, 8), (9, 3)):
        run_and_check(lens, H, Hkv, seed=31)
    # 2200 tokens of 64 key/value heads and more go head by head
    q, k, v, cu, cu_dev = packed([2000, 3, 300], 64, 64, 33)
    out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, 2000)
    assert la.get_device_status() == la.LA_OK
    for a, b in zip(cu[:-1], cu[1:]):
        check(out[a:b, :2], lse[a:b, :2], attention64(q[a:b, :2], k[a:b, :2], v[a:b, :2], 0, S), b - a)
        check(out[a:b, -1:], lse[a:b, -1:], attention64(q[a:b, -1:], k[a:b, -1:], v[a:b, -1:], 0, S), b - a)


@pytest.mark.parametrize("heads", [(1, 1), (8, 1), (3, 3), (5, 1), (4, 2)], ids=str)
@pytest.mark.parametrize("lens", [[1600], [3000], [5001], [1700, 1, 0, 900, 128]], ids=str)
def test_few_heads_and_long_rows(lens, heads):
    """Few items of many key tiles: equal runs of tiles, cut items joined."""
    run_and_check(lens, *heads, seed=len(lens) * 10 + heads[0])


def test_runs_of_tiles_repeat_and_refuse():
    q, k, v, cu, cu_dev = packed([4000, 300], 4, 1, seed=41)
    out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, 4000)
    again, lse2 = la.softmax_prefill_varlen(q, k, v, cu_dev, 4000)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    held = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.softmax_prefill_varlen(q, k, v, cu_dev, 4000, out=held, want_lse=False)
    graph.replay()
    graph.replay()
    assert torch.equal(held, out)
    for table in ([0, 4000, 4299], [0, 4301, 4300], [0, -1, 4300]):
        held.fill_(3.0)
        la.softmax_prefill_varlen(q, k, v, torch.tensor(table, dtype=torch.int32, device="cuda"), 4300, out=held)
        assert la.get_device_status() == la.LA_ERR_INVALID_ARGUMENT
        assert (held == 3.0).all()
    # NaN in one sequence stays there, whichever runs its tiles fall into
    q[4000:], k[4000:], v[4000:] = float("nan"), float("nan"), float("nan")
    got, _ = la.softmax_prefill_varlen(q, k, v, cu_dev, 4000)
    assert torch.equal(got[:4000], out[:4000])
