"""Workloads of the softmax-attention operators: the 1-in-8 layers of a hybrid model.

Five operators, chosen by a case's ``op``:

  prefill  causal attention over packed prompts with grouped key/value heads
  train    the same with its gradients (one forward and one backward pass)
  chunk    new tokens of several requests are written into the pages of their
           key/value caches and attend to everything cached
  decode   one new token per request, likewise
  copy     pages copied inside the pool, as forks and compactions do

Head dimension 128, bf16 tensors, fp32 log-sum-exp.  A cache is a pair of
tensors [n_pages, Hkv, page_size, 128]; row b of the page table lists the
pages of request b.
"""
import math
import random

import torch

own = False
D = 128
SCALE = D ** -0.5
SCORE_ELEMS = 1 << 29  # scores that the plain forms hold at a time


# -- cases ------------------------------------------------------------------

def listed():
    return [
        # one short question to the model: launch latency
        {"name": "prefill short", "op": "prefill", "H": 64, "Hkv": 8, "n": 1, "lo": 129, "hi": 129, "ls": 0},
        # prompts of a serving batch, packed without padding
        {"name": "prefill packed", "op": "prefill", "H": 64, "Hkv": 8, "n": 12, "lo": 1, "hi": 4096, "ls": 1},
        # one document of 32K tokens
        {"name": "prefill long", "op": "prefill", "H": 32, "Hkv": 4, "n": 1, "lo": 32768, "hi": 32768, "ls": 0},
        # fine-tuning on short samples, a key/value head per query head
        {"name": "train short", "op": "train", "H": 8, "Hkv": 8, "n": 9, "lo": 1, "hi": 500, "ls": 2},
        # pre-training on samples packed end to end
        {"name": "train packed", "op": "train", "H": 32, "Hkv": 4, "n": 4, "lo": 1024, "hi": 8192, "ls": 3},
        # follow-up turns of a few conversations
        {"name": "chunk small", "op": "chunk", "H": 64, "Hkv": 8, "n": 3, "lo": 2, "hi": 60, "past": 700, "page": 16, "ls": 4},
        # chunks of long prompts, taken between decode steps
        {"name": "chunk large", "op": "chunk", "H": 64, "Hkv": 8, "n": 4, "lo": 1500, "hi": 2048, "past": 16000, "page": 64, "ls": 5},
        # one user, a short conversation: latency
        {"name": "decode single", "op": "decode", "H": 64, "Hkv": 8, "n": 1, "past": 700, "even": True, "page": 16, "ls": 6},
        # a full serving batch of different lengths
        {"name": "decode batch", "op": "decode", "H": 64, "Hkv": 8, "n": 256, "past": 8192, "even": False, "page": 64, "ls": 7},
        # one request with a very long context
        {"name": "decode long", "op": "decode", "H": 64, "Hkv": 8, "n": 1, "past": 524287, "even": True, "page": 128, "ls": 8},
        # a conversation forked a few ways: its ragged last page
        {"name": "copy fork", "op": "copy", "Hkv": 8, "n": 5, "pages": 512, "page": 16, "ls": 9},
        # a pool compacted after many requests ended
        {"name": "copy compact", "op": "copy", "Hkv": 8, "n": 3001, "pages": 8192, "page": 64, "ls": 10},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "train", "chunk", "decode", "decode", "copy"])
    H, Hkv = rng.choice([(64, 8), (32, 4), (16, 2), (8, 8), (12, 4), (20, 4), (24, 1), (16, 16), (40, 8), (1, 1)])
    page = rng.choice([16, 32, 64, 128])
    ls = rng.randrange(1 << 20)
    if op in ("prefill", "train"):
        n = _log(rng, 1, 24)
        hi = _log(rng, 2, min(16384, 40000 // n) if op == "prefill" else min(6000, 16000 // n))
        return {"op": op, "H": H, "Hkv": Hkv, "n": n, "lo": rng.choice([1, max(1, hi // 2), hi]), "hi": hi, "ls": ls}
    if op == "chunk":
        n = _log(rng, 1, 16)
        hi = _log(rng, 1, 4000 // n)
        return {"op": op, "H": H, "Hkv": Hkv, "n": n, "lo": rng.choice([1, hi]), "hi": hi,
                "past": _log(rng, 1, 60000 // n), "page": page, "ls": ls}
    if op == "decode":
        n = _log(rng, 1, 300)
        return {"op": op, "H": H, "Hkv": Hkv, "n": n, "past": _log(rng, 2, min(300000, 800000 // n)),
                "even": rng.random() < 0.3, "page": page, "ls": ls}
    return {"op": op, "Hkv": Hkv, "n": _log(rng, 1, 3000), "pages": 8000, "page": page, "ls": ls}


def _lens(case):
    """New tokens and cached tokens of each sequence."""
    r = random.Random(case["ls"])
    n = case["n"]
    if case["op"] == "decode":
        return [1] * n, [case["past"] if case["even"] else r.randrange(case["past"] + 1) for _ in range(n)]
    new = [r.randint(case["lo"], case["hi"]) for _ in range(n)]
    return new, [r.randrange(case["past"] + 1) if "past" in case else 0 for _ in range(n)]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed * 1009 + case["ls"])
    normal = lambda *shape: torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)  # noqa: E731
    s = {"case": case}
    if case["op"] == "copy":
        shape = (case["pages"], case["Hkv"], case["page"], D)
        s["kc"], s["vc"] = normal(*shape), normal(*shape)
        ids = torch.randperm(case["pages"], generator=g, device=dev).to(torch.int32)
        n = case["n"]
        if 2 * n > case["pages"]:
            raise ValueError("more pages to copy than half the pool")
        s["src"], s["dst"] = ids[:n].contiguous(), ids[n:2 * n].contiguous()
        return s
    new, past = _lens(case)
    T, H, Hkv = sum(new), case["H"], case["Hkv"]
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    s.update(new=new, past=past, cu_list=cu, cu=torch.tensor(cu, dtype=torch.int32, device=dev), max_new=max(new))
    s["q"] = normal(T, H, D) * 1.5  # scores of a few units
    s["k"], s["v"] = normal(T, Hkv, D), normal(T, Hkv, D)
    if case["op"] == "train":
        s["dout"] = normal(T, H, D)
    if case["op"] in ("chunk", "decode"):
        page = case["page"]
        need = [-(-(a + b) // page) for a, b in zip(new, past)]
        total = sum(need)
        ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        table = torch.zeros(len(new), max(need), dtype=torch.int32, device=dev)
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = ids[at:at + m]
            at += m
        s["table"] = table
        s["lens"] = torch.tensor(past, dtype=torch.int32, device=dev)  # cached before the pass
        s["kc"], s["vc"] = normal(total, Hkv, page, D), normal(total, Hkv, page, D)
    return s


def work(case):
    if case["op"] == "copy":
        return {"bytes": 2 * 2 * case["n"] * case["Hkv"] * case["page"] * D * 2, "flops": 0}
    new, past = _lens(case)
    T, H, Hkv = sum(new), case["H"], case["Hkv"]
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    qo, kv, lse = T * H * D * 2, T * Hkv * D * 2, T * H * 4
    if case["op"] == "prefill":
        return {"bytes": 2 * qo + 2 * kv + lse, "flops": 4 * D * H * pairs}
    if case["op"] == "train":  # forward, then gradients: five products of the scores' size; dout is read, dq written
        return {"bytes": 4 * qo + 4 * kv + lse, "flops": 14 * D * H * pairs}
    cached = 2 * sum(past) * Hkv * D * 2
    return {"bytes": 2 * qo + 4 * kv + lse + cached, "flops": 4 * D * H * pairs}


# -- one pass ---------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        import linear_attention_blocked_b200 as la
        if op == "copy":
            la.cache_copy_pages(s["kc"], s["vc"], s["src"], s["dst"])
            return {"k_cache": s["kc"], "v_cache": s["vc"]}
        if op == "prefill":
            out, lse = la.softmax_prefill_varlen(s["q"], s["k"], s["v"], s["cu"], s["max_new"])
            return {"out": out, "lse": lse}
        if op == "train":
            out, lse = la.softmax_prefill_varlen(s["q"], s["k"], s["v"], s["cu"], s["max_new"])
            dq, dk, dv = la.softmax_prefill_backward_varlen(s["q"], s["k"], s["v"], out, lse, s["dout"], s["cu"],
                                                            s["max_new"])
            return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
        if op == "chunk":
            out, lse = la.softmax_prefill_paged(s["q"], s["k"], s["v"], s["cu"], s["max_new"], s["kc"], s["vc"],
                                                s["table"], s["lens"])
        else:
            out, lse = la.softmax_decode_paged(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"])
        return {"out": out, "lse": lse, "k_cache": s["kc"], "v_cache": s["vc"]}
    if op == "copy":
        src, dst = s["src"].long(), s["dst"].long()
        s["kc"][dst] = s["kc"][src]
        s["vc"][dst] = s["vc"][src]
        return {"k_cache": s["kc"], "v_cache": s["vc"]}
    if op in ("prefill", "train"):
        return _plain_packed(s, op == "train")
    if op == "chunk":
        _plain_append(s)
        out, lse = _plain_chunk(s)
    else:
        _plain_append(s)
        out, lse = _plain_decode(s)
    return {"out": out, "lse": lse, "k_cache": s["kc"], "v_cache": s["vc"]}


def _head_steps(H, G, rows, cols):
    """Query heads in steps whose scores fit, and the key/value head of each."""
    step = max(1, min(H, SCORE_ELEMS // max(1, rows * cols)))
    for h0 in range(0, H, step):
        h1 = min(H, h0 + step)
        yield h0, h1, torch.arange(h0, h1, device="cuda") // G


def _plain_scores(q, k, past):
    """Masked scores [h, n, m] of queries [n, h, D] behind `past` keys."""
    n, m = q.shape[0], k.shape[0]
    x = torch.matmul(q.permute(1, 0, 2), k.permute(1, 2, 0)) * SCALE
    rows = torch.arange(n, device=x.device)[:, None] + past
    return x.masked_fill_(torch.arange(m, device=x.device)[None, :] > rows, float("-inf"))


def _plain_packed(s, train):
    q, k, v = s["q"], s["k"], s["v"]
    T, H, _ = q.shape
    G = H // k.shape[1]
    out = torch.empty_like(q)
    lse = torch.empty(T, H, dtype=torch.float32, device=q.device)
    if train:
        dq = torch.empty_like(q)
        dk32, dv32 = torch.zeros_like(k, dtype=torch.float32), torch.zeros_like(v, dtype=torch.float32)
    for a, b in zip(s["cu_list"][:-1], s["cu_list"][1:]):
        for h0, h1, kvh in _head_steps(H, G, b - a, b - a):
            qf, kf, vf = q[a:b, h0:h1].float(), k[a:b, kvh].float(), v[a:b, kvh].float()
            x = _plain_scores(qf, kf, 0)
            top = x.amax(-1, keepdim=True)
            p = torch.exp_(x.sub_(top))
            total = p.sum(-1, keepdim=True)
            p = p.div_(total)
            out[a:b, h0:h1] = torch.matmul(p, vf.permute(1, 0, 2)).permute(1, 0, 2)
            lse[a:b, h0:h1] = (top + torch.log(total))[..., 0].T
            if train:
                gf = s["dout"][a:b, h0:h1].float()
                dp = torch.matmul(gf.permute(1, 0, 2), vf.permute(1, 2, 0))
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * SCALE
                dq[a:b, h0:h1] = torch.matmul(ds, kf.permute(1, 0, 2)).permute(1, 0, 2)
                dk32[a:b].index_add_(1, kvh, torch.matmul(ds.mT, qf.permute(1, 0, 2)).permute(1, 0, 2))
                dv32[a:b].index_add_(1, kvh, torch.matmul(p.mT, gf.permute(1, 0, 2)).permute(1, 0, 2))
    if train:
        return {"out": out, "lse": lse, "dq": dq, "dk": dk32.to(k.dtype), "dv": dv32.to(v.dtype)}
    return {"out": out, "lse": lse}


def _plain_append(s):
    """Token t of sequence b goes to position lens[b] + t of its cache."""
    page = s["case"]["page"]
    T, n = s["q"].shape[0], len(s["new"])
    tok = torch.arange(T, device="cuda")
    b = torch.searchsorted(s["cu"][1:].contiguous(), tok, right=True).clamp_(max=n - 1)
    pos = s["lens"].long()[b] + tok - s["cu"].long()[b]
    pid = s["table"][b, pos // page].long()
    s["kc"][pid, :, pos % page] = s["k"]
    s["vc"][pid, :, pos % page] = s["v"]


def _pages_of(cache, table, b, length):
    """The first `length` cached rows of request b: [length, Hkv, D]."""
    page = cache.shape[2]
    x = cache[table[b, :-(-length // page)].long()]
    return x.permute(0, 2, 1, 3).reshape(-1, cache.shape[1], D)[:length]


def _plain_chunk(s):
    q = s["q"]
    T, H, _ = q.shape
    G = H // s["k"].shape[1]
    out = torch.empty_like(q)
    lse = torch.empty(T, H, dtype=torch.float32, device=q.device)
    for b, (a, e) in enumerate(zip(s["cu_list"][:-1], s["cu_list"][1:])):
        m = s["past"][b] + e - a
        k, v = _pages_of(s["kc"], s["table"], b, m), _pages_of(s["vc"], s["table"], b, m)
        for h0, h1, kvh in _head_steps(H, G, e - a, m):
            x = _plain_scores(q[a:e, h0:h1].float(), k[:, kvh].float(), s["past"][b])
            top = x.amax(-1, keepdim=True)
            p = torch.exp_(x.sub_(top))
            total = p.sum(-1, keepdim=True)
            out[a:e, h0:h1] = (torch.matmul(p, v[:, kvh].float().permute(1, 0, 2)) / total).permute(1, 0, 2)
            lse[a:e, h0:h1] = (top + torch.log(total))[..., 0].T
    return out, lse


def _plain_decode(s):
    q, table, page = s["q"], s["table"], s["case"]["page"]
    B, H, _ = q.shape
    Hkv = s["k"].shape[1]
    L = table.shape[1] * page
    out = torch.empty_like(q)
    lse = torch.empty(B, H, dtype=torch.float32, device=q.device)
    step = max(1, min(B, (1 << 31) // (L * Hkv * D)))
    for b0 in range(0, B, step):
        b1 = min(B, b0 + step)
        k = s["kc"][table[b0:b1].long()].permute(0, 2, 1, 3, 4).reshape(b1 - b0, Hkv, L, D).float()
        x = torch.matmul(q[b0:b1].float().reshape(b1 - b0, Hkv, H // Hkv, D), k.mT) * SCALE
        del k
        x.masked_fill_(torch.arange(L, device=q.device) > s["lens"][b0:b1, None, None, None], float("-inf"))
        top = x.amax(-1, keepdim=True)
        p = torch.exp_(x.sub_(top))
        total = p.sum(-1, keepdim=True)
        v = s["vc"][table[b0:b1].long()].permute(0, 2, 1, 3, 4).reshape(b1 - b0, Hkv, L, D).float()
        out[b0:b1] = (torch.matmul(p, v) / total).reshape(b1 - b0, H, D)
        lse[b0:b1] = (top + torch.log(total)).reshape(b1 - b0, H)
        del v
    return out, lse


# -- the definition in 64 bits ----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "copy":
        return None  # nothing is computed: values move as they are
    G = case["H"] // case["Hkv"]
    train = case["op"] == "train"
    T, H = s["q"].shape[:2]
    f64 = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.empty(T, H, D, **f64), torch.empty(T, H, **f64)
    if train:
        dq, dk, dv = (torch.zeros(T, h, D, **f64) for h in (H, case["Hkv"], case["Hkv"]))
    for b, n in enumerate(s["new"]):
        t0, past = s["cu_list"][b], s["past"][b]
        for h in range(case["Hkv"]):
            k, v = s["k"][t0:t0 + n, h].double(), s["v"][t0:t0 + n, h].double()
            if past:  # cached rows come before the new ones
                at = torch.arange(past, device="cuda")
                pid = s["table"][b].long()[at // case["page"]]
                k = torch.cat([s["kc"][pid, h, at % case["page"]].double(), k])
                v = torch.cat([s["vc"][pid, h, at % case["page"]].double(), v])
            key = torch.arange(past + n, device="cuda")
            for hq in range(h * G, (h + 1) * G):
                q = s["q"][t0:t0 + n, hq].double()
                if train:
                    go = s["dout"][t0:t0 + n, hq].double()
                for r0 in range(0, n, 4096):  # rows of queries, each with the keys up to its own
                    r1 = min(n, r0 + 4096)
                    m = past + r1
                    z = (q[r0:r1] @ k[:m].T) / math.sqrt(D)
                    seen = key[None, :m] <= (past + torch.arange(r0, r1, device="cuda"))[:, None]
                    z = torch.where(seen, z, torch.full((), -math.inf, **f64))
                    ls = torch.logsumexp(z, 1)
                    w = torch.exp(z - ls[:, None])
                    o = w @ v[:m]
                    out[t0 + r0:t0 + r1, hq], lse[t0 + r0:t0 + r1, hq] = o, ls
                    if train:
                        g = go[r0:r1]
                        dz = w * (g @ v[:m].T - (g * o).sum(1, keepdim=True)) / math.sqrt(D)
                        dq[t0 + r0:t0 + r1, hq] = dz @ k[:m]
                        dk[t0:t0 + m, h] += dz.T @ q[r0:r1]
                        dv[t0:t0 + m, h] += w.T @ g
    if train:
        return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if "kc" in s:
        return {"out": out, "lse": lse, "k_cache": None, "v_cache": None}
    return {"out": out, "lse": lse}
