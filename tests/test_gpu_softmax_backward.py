"""Gradients of la_softmax_prefill_varlen against the formulas and against
differences in 64 bits, with the bounds of softmax_util.gradients64."""
import pytest
import torch

import linear_attention_blocked_b200 as la
from softmax_util import attention64, gradients64, packed

pytestmark = pytest.mark.gpu
S = 128 ** -0.5


def grads(q, k, v, g, cu_dev, longest, scale=None, **kw):
    out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, longest, scale=scale)
    got = la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu_dev, longest, scale=scale, **kw)
    assert la.get_device_status() == la.LA_OK
    return got


def run_and_check(lens, H, Hkv, seed, scale=None):
    q, k, v, cu, cu_dev = packed(lens, H, Hkv, seed)
    g = torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(seed + 1), device="cuda",
                    dtype=torch.bfloat16)
    got = grads(q, k, v, g, cu_dev, max(lens), scale)
    for a, b in zip(cu[:-1], cu[1:]):
        if a == b:
            continue
        ref = gradients64(q[a:b], k[a:b], v[a:b], g[a:b], S if scale is None else scale)
        for x, name in zip(got, "qkv"):
            want, bound = ref[name]
            assert torch.isfinite(x[a:b]).all(), f"d{name} of tokens {a}-{b}"
            over = ((x[a:b].double() - want).abs() / bound).max().item()
            assert over <= 1, f"d{name} of tokens {a}-{b}, H={H} Hkv={Hkv}: {over:.2f} of its bound"


@pytest.mark.parametrize("heads", [(8, 1), (4, 4), (6, 2), (16, 2), (5, 5)], ids=str)
@pytest.mark.parametrize("lens", [[1], [2, 1], [127], [128], [129], [255, 0, 257], [300, 1, 0, 640, 17]], ids=str)
def test_gradients_match_the_formulas(lens, heads):
    run_and_check(lens, *heads, seed=len(lens) * 100 + heads[0])


def test_gradients_of_longer_rows_and_scale():
    run_and_check([2100, 1, 900], 8, 2, seed=7)
    run_and_check([500], 4, 4, seed=8, scale=0.3)


def test_gradients_match_differences():
    """dL along random directions against (L(x + h d) - L(x - h d)) / 2h with L
    in 64 bits: the difference's own error is of order h^2."""
    q, k, v, cu, cu_dev = packed([150], 4, 2, 11)
    gen = torch.Generator(device="cuda").manual_seed(12)
    g = torch.randn(q.shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    got = grads(q, k, v, g, cu_dev, 150)
    ref = gradients64(q, k, v, g, S)
    x = [t.double() for t in (q, k, v)]

    def loss(y):
        return (attention64(*y, 0, S)[0] * g.double()).sum().item()
    for i, name in enumerate("qkv"):
        d = torch.randn(x[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-4
        diff = (loss([t + h * d if j == i else t for j, t in enumerate(x)]) -
                loss([t - h * d if j == i else t for j, t in enumerate(x)])) / (2 * h)
        along = (got[i].double() * d).sum().item()
        # the kernel's error along d, and the difference's (third derivatives of a
        # softmax are of order 1: h^2 |d|^3 over the sizes here stays below 1e-2)
        tol = (ref[name][1] * d.abs()).sum().item() + 1e-2
        assert abs(along - diff) <= tol, (name, along, diff, tol)


def test_one_token_has_no_gradient_to_its_scores():
    q, k, v, cu, cu_dev = packed([1, 1, 1], 4, 2, 13)
    g = torch.randn_like(q)
    dq, dk, dv = grads(q, k, v, g, cu_dev, 1)
    want = g.double().reshape(3, 2, 2, 128).sum(2)
    # P = 1, dP = delta up to the fp32 sums of 128 products
    bound = 256 * 2.0 ** -24 * (g.double().abs().reshape(3, 2, 2, 128) * v.double().abs()[:, :, None]).sum(-1).amax()
    assert dq.double().abs().max() <= bound * S * k.double().abs().max() * 1.01
    assert dk.double().abs().max() <= 2 * bound * S * q.double().abs().max() * 1.01
    assert ((dv.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all()


def test_sequences_do_not_see_each_other():
    lens = [70, 130, 200]
    q, k, v, cu, cu_dev = packed(lens, 4, 2, 17)
    g = torch.randn_like(q)
    want = grads(q, k, v, g, cu_dev, 200)
    for seq in (0, 1, 2):
        args = [t.clone() for t in (q, k, v, g)]
        for t in args:
            t[cu[seq]:cu[seq + 1]] = float("nan")
        got = grads(*args, cu_dev, 200)
        for other in range(3):
            if other != seq:
                a, b = cu[other], cu[other + 1]
                for x, y in zip(got, want):
                    assert torch.equal(x[a:b], y[a:b])


def test_same_call_twice_is_bit_identical_and_captured():
    q, k, v, cu, cu_dev = packed([700, 333, 1], 16, 2, 19)
    g = torch.randn_like(q)
    out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, 700)
    want = la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu_dev, 700)
    again = la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu_dev, 700)
    outs = [torch.zeros_like(x) for x in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu_dev, 700, dq=outs[0], dk=outs[1], dv=outs[2])
    graph.replay()
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu_dev, 700, stream=side)
    torch.cuda.synchronize()
    for x, y, z, w in zip(want, again, outs, other):
        assert torch.equal(x, y) and torch.equal(x, z) and torch.equal(x, w)
    assert la.get_device_status() == la.LA_OK


def test_bad_tables_and_calls_are_refused():
    q, k, v, cu, cu_dev = packed([100, 60], 8, 2, 23)
    g = torch.randn_like(q)
    out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, 100)
    for table in ([0, 100, 159], [0, 161, 160], [0, 120, 160]):
        got = [torch.full_like(x, 3.0) for x in (q, k, v)]
        la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, torch.tensor(table, dtype=torch.int32, device="cuda"),
                                           100, dq=got[0], dk=got[1], dv=got[2])
        assert la.get_device_status() == la.LA_ERR_INVALID_ARGUMENT
        assert all((x == 3.0).all() for x in got)
    with pytest.raises(la.LAError):
        la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu_dev, 100, dq=g)
    with pytest.raises(TypeError):
        la.softmax_prefill_backward_varlen(q, k, v, out.float(), lse, g, cu_dev, 100)


def test_gradients_of_a_shared_head_in_parts():
    """One key/value head for many query heads: its key blocks' sums are formed
    in parts by several CTAs."""
    run_and_check([300, 1, 129], 24, 1, seed=29)
    run_and_check([1300], 64, 1, seed=31)


@pytest.mark.parametrize("scale", [1.5, 8.0])
@pytest.mark.parametrize("heads", [(8, 8), (8, 2), (3, 1)], ids=str)
def test_short_sequences_take_no_error_from_the_rounded_output(heads, scale):
    """Rows of few keys, or of one heavy key, whose gradients are small against the
    terms that they are differences of: bounds without the rounding of `out`."""
    lens = [2] * 20 + [1, 3, 0, 5, 128, 2, 127, 64, 31]
    q, k, v, cu, cu_dev = packed(lens, *heads, seed=heads[0], scale=scale)
    g = torch.randn_like(q)
    out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, max(lens))
    got = la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu_dev, max(lens))
    assert la.get_device_status() == la.LA_OK
    for a, b in zip(cu[:-1], cu[1:]):
        if a == b:
            continue
        want = gradients64(q[a:b], k[a:b], v[a:b], g[a:b], 128 ** -0.5, own_delta=True)
        for x, (name, (y, bound)) in zip(got, want.items()):
            over = ((x[a:b].double() - y).abs() / bound).max().item()
            assert over <= 1, f"d{name} of {b - a} tokens off by {over:.2f} of its bound"
