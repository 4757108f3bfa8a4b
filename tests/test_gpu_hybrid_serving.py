"""The operators together, as a server of the hybrid model uses them: batches of
prompt chunks and decode tokens (plan_batch) go through a Lightning layer on a
state pool (mixed_step) and a softmax layer on a paged cache (page numbers from
PagePool), with requests that fork, end, and a pool that is compacted.  Every
request's outputs are then those of its whole sequence at once."""
import numpy as np
import pytest
import torch

import la_inputs
import linear_attention_blocked_b200 as la
from parity_util import check_out, to_np
from softmax_util import attention64, check

pytestmark = pytest.mark.gpu
H, HKV, D, PAGE, N_PAGES, SLOTS = 8, 2, 128, 16, 120, 8


class Request:
    def __init__(self, slot, pages, seed, n=400):
        self.slot, self.pages = slot, pages
        self.lin = la_inputs.qkv((n, H, D), seed=seed, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.soft = [torch.randn(n, h, D, generator=g, device="cuda", dtype=torch.bfloat16) for h in (H, HKV, HKV)]
        self.done = 0
        self.out_lin, self.out_soft, self.lse = [], [], []

    def fork(self, slot, pages, seed):
        """Same tokens so far, others from here on."""
        child = Request(slot, pages, seed)
        for mine, theirs in zip(self.lin + tuple(self.soft), child.lin + tuple(child.soft)):
            theirs[:self.done] = mine[:self.done]
        child.done = self.done
        child.out_lin, child.out_soft, child.lse = list(self.out_lin), list(self.out_soft), list(self.lse)
        return child


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def step(requests, news, states, kc, vc, pool):
    """One batch: news[i] new tokens of requests[i]."""
    for r, n in zip(requests, news):
        pool.reserve(r.pages, n)
    src, dst = pool.take_copies()
    la.cache_copy_pages(kc, vc, dev(src), dev(dst))
    plan = la.plan_batch(news, [r.slot for r in requests])
    rows = [torch.empty(plan.total_rows, h, D, dtype=torch.bfloat16, device="cuda") for h in (H, H, H, H, HKV, HKV)]
    for i, (r, n) in enumerate(zip(requests, news)):
        a = int(plan.row_offset[i])
        if n:
            for to, x in zip(rows, r.lin + tuple(r.soft)):
                to[a:a + n] = x[r.done:r.done + n]
    ql, kl, vl, q, k, v = rows
    lin = la.mixed_step(ql, kl, vl, dev(plan.cu_seqlens), dev(plan.prefill_slots), plan.max_seqlen,
                        dev(plan.decode_slots), states, out_dtype=torch.float32)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    t = plan.prefill_tokens
    ids = [requests[i].pages for i in plan.prefill_ids]
    if ids:
        la.softmax_prefill_paged(q[:t], k[:t], v[:t], dev(plan.cu_seqlens), plan.max_seqlen, kc, vc, dev(pool.table(ids)),
                                 dev(pool.lengths(ids)), out=out[:t], lse=lse[:t])
    ids = [requests[i].pages for i in plan.decode_ids]
    if ids:
        la.softmax_decode_paged(q[t:], k[t:], v[t:], kc, vc, dev(pool.table(ids)), dev(pool.lengths(ids)),
                                out=out[t:], lse=lse[t:])
    for i, (r, n) in enumerate(zip(requests, news)):
        a = int(plan.row_offset[i])
        if n:
            r.out_lin.append(lin[a:a + n])
            r.out_soft.append(out[a:a + n])
            r.lse.append(lse[a:a + n])
            r.done += n
            pool.advance(r.pages, n)


def test_hybrid_batches_equal_whole_sequences():
    pool = la.PagePool(N_PAGES, PAGE)
    nan = float("nan")
    kc, vc = (torch.full((N_PAGES, HKV, PAGE, D), nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    states = torch.zeros(SLOTS, H, D, D, device="cuda")
    a, b, c = (Request(i, pool.add(), 50 + 10 * i) for i in range(3))
    step([a, b, c], [70, 1, 33], states, kc, vc, pool)          # prompts, one of a single token
    step([a, b, c], [130, 1, 1], states, kc, vc, pool)          # a long prompt's next chunk beside decode tokens
    step([a, b, c], [1, 1, 0], states, kc, vc, pool)
    d = a.fork(3, pool.fork(a.pages), 90)                       # a forks inside a page
    states[d.slot] = states[a.slot]
    step([a, d, b], [1, 1, 1], states, kc, vc, pool)
    step([d, a], [40, 1], states, kc, vc, pool)
    pool.free(b.pages)
    src, dst = pool.compact()
    assert len(src)
    la.cache_copy_pages(kc, vc, dev(src), dev(dst))
    e = Request(4, pool.add(), 95)
    for _ in range(3):
        step([c, d, e, a], [1, 17, 20, 1], states, kc, vc, pool)
    assert la.get_device_status() == la.LA_OK
    for r in (a, c, d, e, b):
        n = r.done
        want, _ = la.prefill(*(x[None, :n].contiguous() for x in r.lin), out_dtype=torch.float32)
        check_out(to_np(torch.cat(r.out_lin)), to_np(want[0]), bf16_out=False)
        q, k, v = (x[:n] for x in r.soft)
        check(torch.cat(r.out_soft), torch.cat(r.lse), attention64(q, k, v, 0, D ** -0.5), n)
    assert la.get_device_status() == la.LA_OK


def test_training_step_through_both_layers():
    """Forward and backward of a softmax layer behind a Lightning layer on one
    packed batch, against autograd of both in 64 bits."""
    lens = [150, 1, 90]
    T = sum(lens)
    cu = la_inputs.cu_seqlens_from_lengths(lens)
    q, k, v = la_inputs.qkv((T, H, D), seed=7, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    q2 = torch.randn(T, H, D, generator=g, device="cuda", dtype=torch.bfloat16)
    k2 = torch.randn(T, HKV, D, generator=g, device="cuda", dtype=torch.bfloat16)
    dout = torch.randn(T, H, D, generator=g, device="cuda", dtype=torch.bfloat16)
    mid, _ = la.prefill_varlen(q, k, v, dev(cu), max(lens))       # the softmax layer's values: a group's mean
    v2 = mid.float().reshape(T, HKV, H // HKV, D).mean(2).bfloat16()
    out, lse = la.softmax_prefill_varlen(q2, k2, v2, dev(cu), max(lens))
    dq2, dk2, dv2 = la.softmax_prefill_backward_varlen(q2, k2, v2, out, lse, dout, dev(cu), max(lens))
    dmid = (dv2.float() / (H // HKV)).repeat_interleave(H // HKV, 1).bfloat16()
    dq, dk, dv, _ = la.prefill_backward_varlen(q, k, v, dmid, dev(cu), max(lens))
    assert la.get_device_status() == la.LA_OK
    leaves = [x.double().requires_grad_() for x in (q, k, v, q2, k2)]
    total = 0.0
    for a, b in zip(cu[:-1], cu[1:]):
        x = [t[a:b].transpose(0, 1) for t in leaves]
        low = torch.ones(b - a, b - a, dtype=torch.bool, device="cuda").tril()
        m = (x[0] @ x[1].mT * low) @ x[2]
        w = m.reshape(HKV, H // HKV, b - a, D).mean(1).repeat_interleave(H // HKV, 0)
        s = (x[3] @ x[4].repeat_interleave(H // HKV, 0).mT * D ** -0.5).masked_fill(~low, float("-inf"))
        total = total + (torch.softmax(s, -1) @ w * dout[a:b].double().transpose(0, 1)).sum()
    for got, leaf in zip((dq, dk, dv, dq2, dk2), torch.autograd.grad(total, leaves)):
        # bf16 on the way: mid, v2, out, dv2, dmid and the gradient itself, and inside the
        # layers P, dS and the state: at most twelve roundings of 2^-8 in a row
        err = torch.linalg.vector_norm(got.double() - leaf) / torch.linalg.vector_norm(leaf)
        assert err <= 12 * 2.0 ** -8, err
