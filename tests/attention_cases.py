"""Ragged batches over a paged cache for the attention operators' tests, and the operators in 64 bits on the host.

The error bounds follow from the arithmetic, not from what the kernels give:

* rotation: the fraction of a turn is held to 2^-24 turns (two fp32 roundings of a number below 1), so the angle to
  2 pi 2^-24 = 3.8e-7; sine and cosine add 2 ulp (2.4e-7), the products and the sum three roundings (1.8e-7): 1e-6 of
  the pair's length, rounded up to 1.2e-6, and one rounding to the result's type.
* attention: a score is a sum of d products with at most d roundings of 2^-24 of the sum of their absolute values S,
  plus two for the scale, and exp adds 2^-21; a weight is so off by the factor delta = S (d + 4) 2^-24 + 2^-21 at most,
  the running sums by 2^-20 more.  With u the type's largest relative rounding (2^-8 bf16, 2^-11 fp16) an output is off by at most u |out| + (u + 4 delta + 2^-20) A where A is the mean of |v| under the weights (the
  rounding of weights, the weights' error in numerator and denominator); lse by delta + 2^-20 + |lse| 2^-22.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 0.0, torch.float64: 0.0}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -24, torch.float32: 0.0, torch.float64: 0.0}   # fp16's subnormals


class Batch:
    """windows and lens per request; k, v of every cached token in the pages, garbage (NaN) in every other slot."""

    def __init__(self, windows, lens, hq, hkv, d, page, dtype, seed=0, heads_first=False, garbage=float("nan"),
                 pad_tokens=0, extra_pages=2, q_scale=1.5):
        g = torch.Generator().manual_seed(seed)
        self.windows, self.lens = list(windows), list(lens)
        self.hq, self.hkv, self.d, self.page, self.dtype = hq, hkv, d, page, dtype
        n = len(windows)
        self.n = n
        per = [-(-x // page) for x in lens]
        self.n_pages = sum(per) + extra_pages
        cols = max(per + [1]) + 1
        order = torch.randperm(self.n_pages, generator=g)
        self.table = torch.zeros((n, cols), dtype=torch.int32)
        at = 0
        for r in range(n):
            self.table[r, :per[r]] = order[at:at + per[r]].to(torch.int32)
            at += per[r]
        dims = (self.n_pages, hkv, page, d) if heads_first else (self.n_pages, page, hkv, d)
        self.k_pages = torch.full(dims, garbage, dtype=dtype)
        self.v_pages = torch.full(dims, garbage, dtype=dtype)
        if heads_first:
            self.k_pages, self.v_pages = self.k_pages.transpose(1, 2), self.v_pages.transpose(1, 2)
        for r in range(n):
            for x, scale in ((self.k_pages, 1.0), (self.v_pages, 1.0)):
                vals = (torch.randn((lens[r], hkv, d), generator=g) * scale).to(dtype)
                for p in range(0, lens[r], page):
                    m = min(page, lens[r] - p)
                    x[self.table[r, p // page].item(), :m] = vals[p:p + m]
        self.qo = [0]
        for w in windows:
            self.qo.append(self.qo[-1] + w)
        self.tokens = self.qo[-1] + pad_tokens
        self.q = (torch.randn((self.tokens, hq, d), generator=g) * q_scale).to(dtype)

    def cached(self, r, which):
        """[len, hkv, d] of request r."""
        x = self.k_pages if which == "k" else self.v_pages
        pages = self.table[r, : -(-self.lens[r] // self.page)].long()
        return x[pages].reshape(-1, self.hkv, self.d)[: self.lens[r]]

    def gpu(self, heads_first=False, device="cuda"):
        """(q, k_pages, v_pages, table, qo_indptr, kv_len) on the device, with the storage order of the pages kept."""
        def pages(x):
            return x.transpose(1, 2).contiguous().to(device).transpose(1, 2) if heads_first else x.contiguous().to(device)
        return (self.q.to(device), pages(self.k_pages), pages(self.v_pages), self.table.to(device),
                torch.tensor(self.qo, dtype=torch.int32, device=device),
                torch.tensor(self.lens, dtype=torch.int32, device=device))


def attend64(b: Batch, scale=None, window=0, full=False):
    """(out, lse, bound_out, bound_lse) in fp64 on the host; rows of no window are left at 0."""
    scale = b.d ** -0.5 if scale is None else scale
    out = torch.zeros((b.tokens, b.hq, b.d), dtype=torch.float64)
    lse = torch.full((b.tokens, b.hq), -math.inf, dtype=torch.float64)
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    u = U[b.dtype]
    grp = b.hq // b.hkv
    for r in range(b.n):
        n, w, t0 = b.lens[r], b.windows[r], b.qo[r]
        k, v = b.cached(r, "k").double(), b.cached(r, "v").double()
        for i in range(w):
            p = n - w + i
            lo = max(0, p - window + 1) if window else 0
            hi = n if full else max(0, min(n, p + 1))
            if hi <= lo:
                continue
            for g in range(b.hkv):
                kk, vv = k[lo:hi, g], v[lo:hi, g]
                q = b.q[t0 + i, g * grp:(g + 1) * grp].double()
                s = scale * (q @ kk.T)
                size = abs(scale) * (q.abs() @ kk.abs().T)
                m = s.amax(-1, keepdim=True)
                e = torch.exp(s - m)
                z = e.sum(-1, keepdim=True)
                o = (e @ vv) / z
                a = (e @ vv.abs()) / z
                delta = size.amax(-1, keepdim=True) * (b.d + 4) * 2.0 ** -24 + 2.0 ** -21
                h = slice(g * grp, (g + 1) * grp)
                out[t0 + i, h], lse[t0 + i, h] = o, (m + z.log()).squeeze(-1)
                tol[t0 + i, h] = u * o.abs() + (u + 4 * delta + 2.0 ** -20) * a + TINY[b.dtype]
                tol_l[t0 + i, h] = (delta.squeeze(-1) + 2.0 ** -20) + lse[t0 + i, h].abs() * 2.0 ** -22
    return out, lse, tol, tol_l


def rotate64(x, positions, freq, interleaved=False, inverse=False, mscale=1.0):
    """(y, bound) in fp64 of x [tokens, heads, d] (any dtype, host)."""
    rot = 2 * freq.shape[0]
    turns = positions.double()[:, None] * freq.double().sum(1)
    t = 2 * math.pi * (turns - turns.floor()) * (-1.0 if inverse else 1.0)
    c, s = (torch.cos(t) * mscale)[:, None], (torch.sin(t) * mscale)[:, None]
    y = x.double().clone()
    i0 = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    i1 = i0 + 1 if interleaved else i0 + rot // 2
    a, b = x.double()[..., i0], x.double()[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    tol = torch.zeros_like(y)
    length = (a * a + b * b).sqrt() * abs(mscale) * 1.2e-6
    tol[..., i0] = tol[..., i1] = length
    tol[..., :rot] += y[..., :rot].abs() * U[x.dtype] * (1 + 2.0 ** -10) + TINY[x.dtype]
    return y, tol
