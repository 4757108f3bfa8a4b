"""Softmax attention calls where warps, kernels or threads meet: rows that do not
fill a warp, kernels that start behind one that still runs, waits that run out,
calls that block."""
import pytest
import torch

import linear_attention_blocked_b200 as la
from softmax_util import gradients64, packed

pytestmark = pytest.mark.gpu
S = 128 ** -0.5


@pytest.mark.parametrize("lens,heads", [([1], (1, 1)), ([1], (3, 1)), ([3], (5, 5)), ([127], (1, 1)), ([129], (3, 3)),
                                        ([2, 0, 3], (1, 1)), ([301] * 133, (1, 1))], ids=str)
def test_odd_numbers_of_rows(lens, heads):
    """Tokens times heads odd: the last warp that sums dout . out has one row for its
    two halves, in the last case after several rounds of its loop."""
    q, k, v, cu, cu_dev = packed(lens, *heads, seed=41)
    assert q.shape[0] * q.shape[1] % 2
    g = torch.randn_like(q)
    out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, max(lens))
    got = la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu_dev, max(lens))
    assert la.get_device_status() == la.LA_OK
    for i in {0, len(lens) // 2, len(lens) - 1}:
        a, b = cu[i], cu[i + 1]
        if a == b:
            continue
        for x, (name, (want, bound)) in zip(got, gradients64(q[a:b], k[a:b], v[a:b], g[a:b], S).items()):
            over = ((x[a:b].double() - want).abs() / bound).max().item()
            assert over <= 1, f"d{name} of tokens {a}-{b} off by {over:.2f} of its bound"
