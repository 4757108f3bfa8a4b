"""The softmax calls give the same results, errors and side effects whether the
compiled module or Python code marshals them."""
import pytest
import torch

import linear_attention_blocked_b200 as la
from linear_attention_blocked_b200 import softmax
from softmax_util import Cache, packed

pytestmark = pytest.mark.gpu


def everything():
    """All five calls, with outputs made and passed: a list of tensors."""
    got = []
    q, k, v, cu, cu_dev = packed([150, 1, 30], 8, 2, 3)
    g = torch.ones_like(q)
    out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, 150)
    got += [out, lse, *la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu_dev, 150)]
    mine = [torch.zeros_like(x) for x in (q, k, v)]
    la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu_dev, 150, dq=mine[0], dk=mine[1], dv=mine[2])
    o2, none = la.softmax_prefill_varlen(q, k, v, cu_dev, 150, scale=0.3, out=torch.zeros_like(q), want_lse=False)
    assert none is None
    got += mine + [o2]
    c = Cache([20, 0, 100], [150, 1, 30], 2, 16, 4)
    got += la.softmax_prefill_paged(q, k, v, cu_dev, 150, c.k, c.v, c.table, c.lens)
    c.lens += torch.tensor([150, 1, 30], dtype=torch.int32, device="cuda") - 2
    assert c.lens.tolist() == [168, -1, 128]     # the second row has no request: its outputs are not written
    for dtype in (torch.bfloat16, torch.float32):
        out, lse = la.softmax_decode_paged(q[:3], k[:3], v[:3], c.k, c.v, c.table, c.lens, out_dtype=dtype)
        got += [out[[0, 2]], lse[[0, 2]]]
    fp32, l2 = torch.zeros(3, 8, 128, device="cuda"), torch.zeros(3, 8, device="cuda")
    la.softmax_decode_paged(q[:3], k[:3], v[:3], c.k, c.v, c.table, c.lens, out=fp32, lse=l2)
    la.cache_copy_pages(c.k, c.v, c.table[0, :1].clone(), c.table[0, 3:4].clone())
    got += [fp32, l2, c.k, c.v]
    assert la.get_device_status() == la.LA_OK
    return got


def wrong_calls():
    q, k, v, cu, cu_dev = packed([40], 4, 2, 5)
    c = Cache([20], [40], 2, 16, 6)
    out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, 40)
    p, b = la.softmax_prefill_varlen, la.softmax_prefill_backward_varlen
    d, copy = la.softmax_decode_paged, la.cache_copy_pages
    one = (q[:1], k[:1], v[:1], c.k, c.v, c.table, c.lens)
    return [
        lambda: p(q.float(), k, v, cu_dev, 40), lambda: p(q.cpu(), k, v, cu_dev, 40),
        lambda: p(q.transpose(0, 1), k, v, cu_dev, 40), lambda: p(q[:, :3].contiguous(), k, v, cu_dev, 40),
        lambda: p(q, k[:39], v, cu_dev, 40), lambda: p(q, k, v, cu_dev.long(), 40),
        lambda: p(q, k, v, cu_dev[:0], 40), lambda: p(q, k, v, cu_dev, 40, scale=-1.0),
        lambda: p(q, k, v, cu_dev, 40, out=q), lambda: p(q, k, v, cu_dev, 40, out=out[:39]),
        lambda: p(q, k, v, cu_dev, 40, lse=lse.double()), lambda: p(q[..., :64].contiguous(), k, v, cu_dev, 40),
        lambda: p(q, k, v, cu_dev, 40, out=out.float()), lambda: p(q, k, v, cu_dev, 1 << 40),
        lambda: b(q, k, v, out, lse, q[:39], cu_dev, 40), lambda: b(q, k, v, out, lse, q.clone(), cu_dev, 40, dk=q),
        lambda: d(*one, out_dtype=torch.float16), lambda: d(*one[:5], c.table[:0], c.lens),
        lambda: d(*one[:6], c.lens.long()), lambda: d(*one[:3], c.k[:, :1], c.v[:, :1], c.table, c.lens),
        lambda: d(*one[:3], c.k[:, :, :8].contiguous(), c.v[:, :, :8].contiguous(), c.table, c.lens),
        lambda: copy(c.k, c.v[:1], c.lens, c.lens), lambda: copy(c.k, c.v, c.lens, c.table[0]),
        lambda: copy(c.k, c.k, c.lens, c.lens), lambda: copy(c.k[0], c.v[0], c.lens, c.lens),
    ]


def test_compiled_and_python_marshalling_agree(monkeypatch):
    assert softmax._module() is not None, "the marshalling module is not built"
    fast = everything()
    errors = []
    for i, call in enumerate(wrong_calls()):
        with pytest.raises(Exception) as e:
            call()
            print("not refused:", i)
        errors.append(type(e.value))
    monkeypatch.setattr(softmax, "_marshal", None)
    for x, y in zip(fast, everything(), strict=True):
        assert x.dtype == y.dtype and torch.equal(x.nan_to_num(), y.nan_to_num())
    for call, want in zip(wrong_calls(), errors):
        with pytest.raises(want):
            call()
    assert la.get_device_status() == la.LA_OK


def test_calls_leave_nothing_behind():
    """References and memory: a thousand calls end with as much as ten."""
    q, k, v, cu, cu_dev = packed([40], 4, 2, 5)
    out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, 40)

    def calls(n):
        for _ in range(n):
            la.softmax_prefill_varlen(q, k, v, cu_dev, 40)
            la.softmax_prefill_backward_varlen(q, k, v, out, lse, q, cu_dev, 40)
        torch.cuda.synchronize()
        return torch.cuda.memory_allocated()
    assert calls(10) == calls(1000)


def test_lengths_below_zero_raise_the_same(monkeypatch):
    """max_seqlen = -1 and beyond 32 bits: a ValueError, however the call is marshalled."""
    q, k, v, cu, cu_dev = packed([40], 4, 2, 5)
    c = Cache([20], [40], 2, 16, 6)
    out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, 40)
    for _ in range(2):
        for n in (-1, -(1 << 31), 1 << 31, -(1 << 40)):
            with pytest.raises(ValueError):
                la.softmax_prefill_varlen(q, k, v, cu_dev, n)
            with pytest.raises(ValueError):
                la.softmax_prefill_backward_varlen(q, k, v, out, lse, q.clone(), cu_dev, n)
            with pytest.raises(ValueError):
                la.softmax_prefill_paged(q, k, v, cu_dev, n, c.k, c.v, c.table, c.lens)
        monkeypatch.setattr(softmax, "_marshal", None)
    assert la.get_device_status() == la.LA_OK
