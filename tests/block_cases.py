"""Cases and 64-bit references of the attention half of a decoder block:
residual RMSNorm, rotary positions with the cache append, paged attention.

Error bounds count the roundings that the operators' statements allow: half a
step of the output's type, half a step of the 16-bit softmax weights, and
fp32 arithmetic (2^-24 per operation) for everything between.
"""
from __future__ import annotations

import math

import numpy as np
import torch

U32 = 2.0 ** -24
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


class Batch:
    """A ragged batch over a paged cache, on the CPU.  Pages are handed out in
    no order; every cache row that holds no token is NaN; table entries past a
    sequence's last page name a page that is not there."""

    def __init__(self, new, lens, Hq, Hkv, D, page, dtype, seed=0, spare_rows=0, spare_pages=2):
        g = torch.Generator().manual_seed(seed)
        self.new, self.lens_list = list(new), list(lens)
        self.Hq, self.Hkv, self.D, self.page, self.dtype = Hq, Hkv, D, page, dtype
        self.B = len(new)
        self.used = [-(-L // page) for L in lens]
        self.P = sum(self.used) + spare_pages
        self.N = max(1, sum(new) + spare_rows)
        order = torch.randperm(self.P, generator=g).tolist()
        self.table = torch.full((self.B, max(1, max(self.used))), 1 << 30, dtype=torch.int32)
        at = 0
        for b, u in enumerate(self.used):
            self.table[b, :u] = torch.tensor(order[at:at + u], dtype=torch.int32)
            at += u
        self.offs = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.k = torch.full((self.P, Hkv, page, D), float("nan"), dtype=dtype)
        self.v = torch.full((self.P, Hkv, page, D), float("nan"), dtype=dtype)
        for b, L in enumerate(lens):
            for j in range(0, L, page):
                n = min(page, L - j)
                pg = int(self.table[b, j // page])
                self.k[pg, :, :n] = torch.randn(Hkv, n, D, generator=g).to(dtype)
                self.v[pg, :, :n] = torch.randn(Hkv, n, D, generator=g).to(dtype)
        self.q = torch.randn(self.N, Hq, D, generator=g).to(dtype)

    def cached(self, b, pages):
        """[Hkv, L, D] of sequence b in fp64."""
        ids = self.table[b, :self.used[b]].long()
        return pages[ids].transpose(0, 1).flatten(1, 2)[:, :self.lens_list[b]].double()

    @property
    def most(self):
        return max(1, max(self.new))

    def dev(self, device):
        return {n: getattr(self, n).to(device) for n in ("q", "k", "v", "table", "offs", "lens")}


def attention_ref(case: Batch, scale, window=0, softcap=0.0):
    """out, lse and their error bounds, [N, Hq, D] and [N, Hq] fp64; rows of no
    sequence are NaN in all four."""
    nan = float("nan")
    out = torch.full((case.N, case.Hq, case.D), nan, dtype=torch.float64)
    tol = torch.full_like(out, nan)
    lse = torch.full((case.N, case.Hq), nan, dtype=torch.float64)
    lse_tol = torch.full_like(lse, nan)
    G, u = case.Hq // case.Hkv, half_step(case.dtype)
    tiny = 2.0 ** -25 if case.dtype is torch.float16 else 0.0  # half a step of fp16 below 2^-14
    row0 = 0
    for b, (n, L) in enumerate(zip(case.new, case.lens_list)):
        if n == 0:
            continue
        q = case.q[row0:row0 + n].double().view(n, case.Hkv, G, case.D).permute(1, 2, 0, 3)
        rows = slice(row0, row0 + n)
        row0 += n
        if L == 0:
            out[rows], tol[rows], lse[rows], lse_tol[rows] = 0, 0, -math.inf, 0
            continue
        k, v = case.cached(b, case.k), case.cached(b, case.v)
        z = torch.einsum("hgnd,hkd->hgnk", q, k) * scale
        # the products are exact in fp32; their sum and what follows are not
        dz = torch.einsum("hgnd,hkd->hgnk", q.abs(), k.abs()) * abs(scale) * (case.D + 8) * U32
        if softcap > 0:
            z = softcap * torch.tanh(z / softcap)
            dz = dz + softcap * 2.0 ** -20  # tanh within a few fp32 steps of 1
        t = torch.arange(L - n, L)[:, None]
        j = torch.arange(L)[None]
        seen = j <= t
        if window > 0:
            seen &= j > t - window
        z = z.masked_fill(~seen, -math.inf)
        dz = torch.where(seen, dz, 0.0)
        e = torch.logsumexp(z, -1)
        none = ~seen.any(-1)
        p = torch.where(none[:, None], 0.0, torch.exp(z - torch.where(none, 0.0, e)[..., None]))
        o = torch.einsum("hgnk,hkd->hgnd", p, v)
        # weights: relative error of the scores (both sides of the fraction),
        # of exp2 (2^-21) and of fp32 sums over L terms, and the 16-bit rounding
        rel = 2 * dz.amax(-1) + 2.0 ** -20 + (L + 64) * U32
        absv = torch.einsum("hgnk,hkd->hgnd", p, v.abs())
        top = torch.where(none, 0.0, z.amax(-1))
        small = tiny * torch.exp(top - torch.where(none, 0.0, e))[..., None] * v.abs().sum(1)[:, None, None]
        err = (rel[..., None] + u) * absv + small
        err = err + u * (o.abs() + err) + torch.finfo(case.dtype).smallest_normal * u
        put = lambda x: x.permute(2, 0, 1, *range(3, x.dim())).reshape(n, case.Hq, *x.shape[3:])  # noqa: E731
        out[rows], tol[rows] = put(o), put(err)
        lse[rows] = put(e)
        lse_tol[rows] = put(torch.where(none, 0.0, dz.amax(-1) + 2.0 ** -20 + (L + 64) * U32 + 4 * U32 * e.abs()))
    return out, lse, tol, lse_tol


def inv_freq(rot, theta=1e6):
    return theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def rope_ref(qkv, pos, freq, axis, Hq, Hkv, D, qw, kw, eps, interleaved):
    """Rotated q [N, Hq, D], rotated k and v [N, Hkv, D] in fp64, and the error bounds of q and k."""
    N = qkv.shape[0]
    x = qkv.double().view(N, Hq + 2 * Hkv, D)
    q, k, v = x[:, :Hq].clone(), x[:, Hq:Hq + Hkv].clone(), x[:, Hq + Hkv:]
    dev = []
    rot = 2 * freq.numel()
    ax = axis.long() if axis is not None else torch.zeros(rot // 2, dtype=torch.long)
    ang = pos.long()[ax].t().double() * freq  # [N, rot/2]
    cos, sin = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    # an fp64 angle's own error, on both sides
    da = (pos.long()[ax].t().abs().double() * freq * 2.0 ** -51)[:, None] + 6 * U32
    res = []
    for y, w in ((q, qw), (k, kw)):
        rel = 0.0
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
            rel = (D // 2 + 6) * U32
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
        ra, rb = a * cos - b * sin, b * cos + a * sin
        out = y.clone()
        size = y.abs().clone()
        if interleaved:
            out[..., 0:rot:2], out[..., 1:rot:2] = ra, rb
        else:
            out[..., :rot // 2], out[..., rot // 2:rot] = ra, rb
        m = (a.abs() + b.abs()) * (1 + 0 * da)
        e = m * (da + 3 * U32 + rel)
        err = size * rel
        if interleaved:
            err[..., 0:rot:2], err[..., 1:rot:2] = e, e
        else:
            err[..., :rot // 2], err[..., rot // 2:rot] = e, e
        u = half_step(qkv.dtype)
        res.append((out, err * (1 + u) + u * out.abs() + torch.finfo(qkv.dtype).smallest_normal * u))
    (qo, qe), (ko, ke) = res
    return qo, ko, v, qe, ke


def norm_ref(x, residual, gamma, eps):
    """s and y in fp64."""
    s = x.double() + (residual.double() if residual is not None else 0)
    y = s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps) * gamma.double()
    return s, y
