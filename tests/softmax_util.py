"""Plain 64-bit softmax attention for the GPU tests, and the bounds that the
kernels' roundings allow.

Half a step of bf16 is eps/2 = 2^-8 of a value.  The prefill kernel rounds the
weights once to bf16 and the output once to bf16, everything else is fp32, so

    |out - exact| <= 2^-8 |exact| + 2^-8 A + f,   A = sum_s p_ts |v_s|

(the second term: each p_ts is off by at most 2^-8 p_ts), where f collects the
fp32 work.  A score is an fp32 sum of 128 exact products: off by at most
128 * 2^-24 sum |q_i k_i| =: e (scaled).  It enters p as a factor e^{+-2e}
(numerator and lse), the exponential instruction adds 2^-22, the 2^-24 of
c x - c m adds |c x| 2^-23, and the sums over n keys add n 2^-24 each at worst,
so f <= A (4 e + 2^-21 + |s| 2^-22 + n 2^-23) with |s| the largest score.
"""
import torch

D = 128
BF16 = torch.finfo(torch.bfloat16).eps / 2


def attention64(q, k, v, past, scale):
    """q [n, H, D] behind `past` of the keys k, v [past + n, Hkv, D], all on
    the GPU.  Returns (out, lse, A, smax, e): A as above per element, smax
    the largest |score| and e the bound of a score's fp32 error, per row."""
    n, H, _ = q.shape
    m, Hkv, _ = k.shape
    G = H // Hkv
    rows = torch.arange(n, device=q.device)[:, None] + past
    seen = torch.arange(m, device=q.device)[None, :] <= rows
    out, A = (torch.empty(n, H, D, dtype=torch.float64, device=q.device) for _ in range(2))
    lse, smax, e = (torch.empty(n, H, dtype=torch.float64, device=q.device) for _ in range(3))
    for h in range(H):
        q64, k64, v64 = q[:, h].double(), k[:, h // G].double(), v[:, h // G].double()
        x = (q64 @ k64.T) * scale
        mag = (q64.abs() @ k64.abs().T) * scale
        x = x.masked_fill(~seen, float("-inf"))
        lse[:, h] = torch.logsumexp(x, 1)
        p = torch.exp(x - lse[:, h, None])
        out[:, h], A[:, h] = p @ v64, p @ v64.abs()
        smax[:, h] = x.masked_fill(~seen, 0).abs().amax(1)
        e[:, h] = mag.masked_fill(~seen, 0).amax(1) * 128 * 2.0 ** -24
    return out, lse, A, smax, e


def check(out, lse, ref, keys, what="", p_step=BF16, out_step=BF16):
    """out [n, H, D], lse [n, H] or None against attention64's `ref`; `keys`:
    the longest row.  p_step, out_step: half steps of the weights and outputs."""
    r_out, r_lse, A, smax, e = ref
    f = 4 * e + 2.0 ** -21 + smax * 2.0 ** -22 + keys * 2.0 ** -23
    assert torch.isfinite(out).all(), what
    tol = out_step * r_out.abs() + A * (p_step + f[..., None]) * (1 + out_step) + 1e-30
    over = ((out.double() - r_out).abs() / tol).max().item() if out.numel() else 0.0
    assert over <= 1, f"{what}: out off by {over:.2f} of its bound"
    if lse is not None:
        # the sum's relative error (as f), the log's and the product's roundings
        tol = f + (smax + r_lse.abs() + 1) * 2.0 ** -21
        over = ((lse.double() - r_lse).abs() / tol).max().item() if lse.numel() else 0.0
        assert over <= 1, f"{what}: lse off by {over:.2f} of its bound"


def packed(lens, H, Hkv, seed, device="cuda", scale=1.5):
    g = torch.Generator(device=device).manual_seed(seed)
    T = sum(lens)
    q = torch.randn(T, H, D, generator=g, device=device, dtype=torch.bfloat16) * scale
    k, v = (torch.randn(T, Hkv, D, generator=g, device=device, dtype=torch.bfloat16) for _ in range(2))
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return q, k, v, cu, torch.tensor(cu, dtype=torch.int32, device=device)


class Cache:
    """A paged cache of requests with `past` cached tokens and room for `new`
    more: pages in random order, NaN in every row that holds no token."""

    def __init__(self, past, new, Hkv, page, seed, spare=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        need = [-(-(a + b) // page) for a, b in zip(past, new)]
        self.n_pages = sum(need) + spare
        ids = torch.randperm(self.n_pages, generator=g, device="cuda").to(torch.int32)
        # entries behind a request's pages are out of range: they must not be read
        self.table = torch.full((len(past), max(need + [1])), 1 << 30, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        shape = (self.n_pages, Hkv, page, D)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.page = page
        self.past = [torch.randn(2, n, Hkv, D, generator=g, device="cuda", dtype=torch.bfloat16) for n in past]
        for b, n in enumerate(past):
            self.write(b, 0, self.past[b][0], self.past[b][1])
        self.lens = torch.tensor(past, dtype=torch.int32, device="cuda")

    def rows(self, b, n):
        pos = torch.arange(n, device="cuda")
        return self.table[b, pos // self.page].long(), pos % self.page

    def write(self, b, at, k, v):
        pos = torch.arange(at, at + k.shape[0], device="cuda")
        pid = self.table[b, pos // self.page].long()
        self.k[pid, :, pos % self.page] = k
        self.v[pid, :, pos % self.page] = v

    def read(self, b, n):
        pid, off = self.rows(b, n)
        return self.k[pid, :, off], self.v[pid, :, off]


def gradients64(q, k, v, g, scale, own_delta=False):
    """Gradients of one sequence (no past) for dL/dout = g, and bounds of what
    the kernels' roundings may add to them: {"q": (dq, bound), ...}.

    P is rounded to bf16 once for dv, dS once for dq and dk, and each gradient
    once: half a step of 2^-8 each.  delta = g . out is formed from the bf16
    out, which `check` allows to be off by 2^-8 (|out| + A) + f A.  fp32: P is
    off by a factor of 1 +- r, r = 4 e + 2^-21 + smax 2^-22 as in `check`;
    g . v and delta are sums of 128 terms; sums over n terms add n 2^-23.

    own_delta (sequences of at most 128 tokens): delta is the fp32 sum of P (g . v),
    off by the errors of its P and g . v and of a sum over n terms."""
    n, H, _ = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    out, lse, A, smax, e = attention64(q, k, v, 0, scale)
    seen = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
    dq, bq = (torch.zeros(n, H, D, dtype=torch.float64, device=q.device) for _ in range(2))
    dk, bk, dv, bv = (torch.zeros(n, Hkv, D, dtype=torch.float64, device=q.device) for _ in range(4))
    u = 2.0 ** -24
    for h in range(H):
        q64, k64, v64, g64 = (x.double() for x in (q[:, h], k[:, h // G], v[:, h // G], g[:, h]))
        p = torch.exp((q64 @ k64.T * scale).masked_fill(~seen, float("-inf")) - lse[:, h, None])
        r = (4 * e[:, h] + 2.0 ** -21 + smax[:, h] * 2.0 ** -22 + n * 2.0 ** -23)[:, None]
        o = out[:, h]
        delta = (g64 * o).sum(1, keepdim=True)
        dp = g64 @ v64.T
        ds = p * (dp - delta)
        o_off = BF16 * o.abs() + A[:, h] * (BF16 + r) * (1 + BF16)
        off = (g64.abs() * o_off).sum(1, keepdim=True) + 129 * u * (g64.abs() @ v64.abs().T +
                                                                     (g64 * o).abs().sum(1, keepdim=True))
        if own_delta:
            dp_off = 129 * u * (g64.abs() @ v64.abs().T)
            off = dp_off + (p * (dp.abs() * (r + n * 2 * u) + dp_off)).sum(1, keepdim=True)
        ds_off = ds.abs() * (BF16 + 2 * r) + p * off * (1 + BF16) * (1 + r)
        p_off = p * (BF16 + 2 * r)
        dq[:, h] = ds @ k64 * scale
        bq[:, h] = (ds_off + n * u * 2 * ds.abs()) @ k64.abs() * scale
        dk[:, h // G] += ds.T @ q64 * scale
        bk[:, h // G] += (ds_off + n * G * u * 2 * ds.abs()).T @ q64.abs() * scale
        dv[:, h // G] += p.T @ g64
        bv[:, h // G] += (p_off + n * G * u * 2 * p).T @ g64.abs()
    return {name: (x, BF16 * x.abs() + b * (1 + BF16) + 1e-30)
            for name, x, b in (("q", dq, bq), ("k", dk, bk), ("v", dv, bv))}
