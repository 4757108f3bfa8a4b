"""Softmax attention calls where warps, kernels or threads meet: rows that do not
fill a warp, kernels that start behind one that still runs, waits that run out,
calls that block."""
import threading
import time

import pytest
import torch

import linear_attention_blocked_b200 as la
from softmax_util import Cache, attention64, check, gradients64, packed

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


def long_call(past=400000):
    """A call of some 5 ms on 100 of the SMs: one new token of 200 heads behind 400000
    cached ones that they share.  The SMs left over take the next kernel's CTAs at once."""
    page = 128
    pages = past // page + 1
    gen = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.randn(pages, 1, page, 128, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q, k, v, _, cu = packed([1], 200, 1, 4)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([past], dtype=torch.int32, device="cuda")
    return lambda: la.softmax_prefill_paged(q, k, v, cu, 1, kc, vc, table, lens)


@pytest.mark.parametrize("kind", ["prompt", "runs", "chunk", "gradients"])
def test_limits_do_not_count_the_kernel_in_front(kind):
    """A kernel that starts while the one in front of it still runs waits for that one's
    end before its own time limits begin."""
    long = long_call()
    lens = [3000] if kind == "runs" else [60]
    q, k, v, _, cu = packed(lens, 2, 1, 5)
    c = Cache([100], [60], 1, 16, 6)
    g = torch.randn_like(q)
    o, l = la.softmax_prefill_varlen(q, k, v, cu, lens[0])

    def call():
        if kind == "chunk":
            return la.softmax_prefill_paged(q, k, v, cu, 60, c.k, c.v, c.table, c.lens)
        if kind == "gradients":
            return la.softmax_prefill_backward_varlen(q, k, v, o, l, g, cu, 60)
        return la.softmax_prefill_varlen(q, k, v, cu, lens[0])
    want = call()
    long()
    torch.cuda.synchronize()
    assert la.get_device_status() == la.LA_OK
    begin, middle, end = (torch.cuda.Event(enable_timing=True) for _ in range(3))
    begin.record()
    long()
    middle.record()
    torch.cuda.synchronize()
    assert begin.elapsed_time(middle) > 2.0, "the call in front is too short to show anything"
    try:
        long()
        la.set_wait_limit_ns(1_000_000)
        got = call()
    finally:
        la.set_wait_limit_ns(0)
    assert la.get_device_status() == la.LA_OK
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("kind", ["prompt", "gradients", "chunk", "decode", "copy"])
def test_other_threads_run_while_a_call_waits(kind):
    """A call that blocks, here behind a full launch queue, does not hold up the
    process's other Python threads."""
    q, k, v, _, cu = packed([40], 4, 2, 7)
    c = Cache([100], [40], 2, 16, 8)
    g = torch.randn_like(q)
    out, lse = la.softmax_prefill_varlen(q, k, v, cu, 40)
    dq, dk, dv = (torch.empty_like(x) for x in (q, k, v))
    one = [torch.empty_like(out[:1]), torch.empty_like(lse[:1])]
    src, dst = (torch.tensor([i], dtype=torch.int32, device="cuda") for i in (0, 1))
    call = {
        "prompt": lambda: la.softmax_prefill_varlen(q, k, v, cu, 40, out=out, lse=lse),
        "gradients": lambda: la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu, 40, dq=dq, dk=dk, dv=dv),
        "chunk": lambda: la.softmax_prefill_paged(q, k, v, cu, 40, c.k, c.v, c.table, c.lens, out=out, lse=lse),
        "decode": lambda: la.softmax_decode_paged(q[:1], k[:1], v[:1], c.k, c.v, c.table, c.lens, out=one[0], lse=one[1]),
        "copy": lambda: la.cache_copy_pages(c.k, c.v, src, dst),
    }[kind]
    call()
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.002)
    other = threading.Thread(target=tick)
    other.start()
    try:
        torch.cuda._sleep(1_500_000_000)  # some 0.8 s: the launches behind it fill the queue
        longest = began = 0.0
        for _ in range(3000):
            t0 = time.perf_counter()
            call()
            t1 = time.perf_counter()
            if t1 - t0 > longest:
                longest, began = t1 - t0, t0
            if longest > 0.1:
                break
    finally:
        stop.set()
        other.join()
    torch.cuda.synchronize()
    assert la.get_device_status() == la.LA_OK
    assert longest > 0.1, "no call blocked"
    inside = [t for t in ticks if began < t < began + longest]
    # a tick takes 2 ms and what the machine's scheduler adds: a fifth of them is plenty
    assert len(inside) >= longest / 0.002 / 5, f"{len(inside)} ticks in {longest:.3f} s"


@pytest.mark.parametrize("heads,lens", [((4, 4), [200]), ((8, 1), [40, 90]), ((16, 2), [700, 33]), ((64, 8), [1])], ids=str)
def test_gradients_in_one_workspace_follow_their_inputs(heads, lens):
    """Calls one behind the other in one workspace, with fewer key blocks than SMs, so
    that dq starts on SMs that dk and dv never used: every call's gradients are those of
    its own inputs, lse and tables."""
    sets, total = [], sum(lens)
    for seed in range(3):
        order = lens[seed % len(lens):] + lens[:seed % len(lens)]
        q, k, v, _, cu = packed(order, *heads, seed)
        g = torch.randn_like(q)
        out, lse = la.softmax_prefill_varlen(q, k, v, cu, max(lens))
        want = la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu, max(lens))
        sets.append(((q, k, v, out, lse, g, cu, max(lens)), want))
    torch.cuda.synchronize()
    size = la.lib().la_softmax_prefill_backward_varlen_workspace_size(len(lens), total, *heads, 128)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    got = [[torch.empty_like(x) for x in sets[0][1]] for _ in range(60)]
    for _ in range(5):
        for i, (dq, dk, dv) in enumerate(got):
            la.softmax_prefill_backward_varlen(*sets[i * i % 3][0], dq=dq, dk=dk, dv=dv, workspace=ws)
        torch.cuda.synchronize()
        for i, xs in enumerate(got):
            for x, y in zip(xs, sets[i * i % 3][1]):
                assert torch.equal(x, y), i
    assert la.get_device_status() == la.LA_OK


@pytest.mark.parametrize("kind", ["prompt", "gradients"])
def test_waits_that_run_out(kind):
    """A limit far below the time of an item, for whose end warps wait: the kernels give
    up, say so, and leave everything behind them as it should be."""
    lens, heads = [300, 1, 129], (6, 2)
    q, k, v, cu, cu_dev = packed(lens, *heads, seed=71)
    g = torch.randn_like(q)
    if kind == "prompt":
        long = long_call(800000)
    else:
        x = [torch.randn(400000, 1, 128, device="cuda", dtype=torch.bfloat16) for _ in range(5)]
        lse = torch.zeros(400000, 1, device="cuda")
        cu_long = torch.tensor([0, 400000], dtype=torch.int32, device="cuda")

        def long():
            return la.softmax_prefill_backward_varlen(*x[:4], lse, x[4], cu_long, 400000)
    try:
        la.set_wait_limit_ns(100_000)
        long()
        torch.cuda.synchronize()
    finally:
        la.set_wait_limit_ns(0)
    assert la.get_device_status() == la.LA_ERR_TIMEOUT
    out, lse = la.softmax_prefill_varlen(q, k, v, cu_dev, max(lens))
    got = la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu_dev, max(lens))
    assert la.get_device_status() == la.LA_OK
    for a, b in zip(cu[:-1], cu[1:]):
        check(out[a:b], lse[a:b], attention64(q[a:b], k[a:b], v[a:b], 0, S), b - a)
        for y, (want, bound) in zip(got, gradients64(q[a:b], k[a:b], v[a:b], g[a:b], S).values()):
            assert ((y[a:b].double() - want).abs() <= bound).all()
    if kind == "prompt":
        first, again = long(), long()
        assert la.get_device_status() == la.LA_OK
        assert all(torch.isfinite(y).all() and torch.equal(y, z) for y, z in zip(first, again))


def test_calls_from_several_threads():
    """Threads with a stream each call at once, as the released interpreter lock allows:
    the same results as one thread's."""
    def work(seed):
        lens = [40, 300, 7 + seed]
        q, k, v, _, cu = packed(lens, 16, 2, seed)
        c = Cache([500, 30, 900], [300, 300, 300], 2, 32, seed)
        g = torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda",
                        dtype=torch.bfloat16)
        got = []
        for _ in range(30):
            out, lse = la.softmax_prefill_varlen(q, k, v, cu, 300)
            got = [out, lse, *la.softmax_prefill_backward_varlen(q, k, v, out, lse, g, cu, 300),
                   *la.softmax_prefill_paged(q, k, v, cu, 300, c.k, c.v, c.table, c.lens),
                   *la.softmax_decode_paged(q[:3], k[:3], v[:3], c.k, c.v, c.table, c.lens)]
        torch.cuda.current_stream().synchronize()
        return got
    want = [work(seed) for seed in range(4)]
    torch.cuda.synchronize()
    got = [None] * 4

    def threaded(seed):
        with torch.cuda.stream(torch.cuda.Stream()):
            got[seed] = work(seed)
    threads = [threading.Thread(target=threaded, args=(seed,)) for seed in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert la.get_device_status() == la.LA_OK
    for x, y in zip(got, want):
        assert x is not None and all(torch.equal(a, b) for a, b in zip(x, y))
