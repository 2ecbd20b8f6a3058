"""Cases and 64-bit references of what the paged cache has beside its 16-bit
chains: 8-bit codes, trees of drafted tokens, sinks beside a window.

Error bounds count the roundings that the operators' statements allow, as in
block_cases; over codes also one fp32 product for each scale, and, as the weights may
be fp16 there whatever the type, half of that type's smallest step beside the largest
value of the cache.
"""
from __future__ import annotations

import math

import torch

from tests.block_cases import U32, Batch, half_step


def quantised(x):
    """Codes and scales of the last dimension, by the quantiser's fp32 steps (values of any type, on the CPU)."""
    x = x.float()
    most = torch.where(x.isnan().any(-1, keepdim=True), math.nan, x.abs().amax(-1, keepdim=True))
    f = torch.tensor(127.0) / most
    some = f <= torch.finfo(torch.float32).max
    codes = torch.nan_to_num(torch.round(x * torch.where(some, f, 0.0)), nan=0.0).to(torch.int8)
    return codes, torch.where(some | most.isnan(), most / 127, 0.0).squeeze(-1)


class Batch8(Batch):
    """A Batch whose cache holds codes: rows of no token have NaN scales and any codes."""

    def __init__(self, *args, **kwargs):
        super().__init__(*args, **kwargs)
        g = torch.Generator().manual_seed(kwargs.get("seed", 0) + 99)
        for n in "kv":
            x = getattr(self, n)
            none = x.isnan().any(-1)
            codes, scales = quantised(x.nan_to_num())
            codes[none] = torch.randint(-128, 128, (int(none.sum()), self.D), generator=g, dtype=torch.int8)
            scales[none] = math.nan
            setattr(self, n, codes)
            setattr(self, n + "s", scales)

    def cached(self, b, pages):
        scales = self.ks if pages is self.k else self.vs
        ids = self.table[b, :self.used[b]].long()
        take = lambda p: p[ids].transpose(0, 1).flatten(1, 2)[:, :self.lens_list[b]].double()  # noqa: E731
        return take(pages) * take(scales).unsqueeze(-1)

    def dev(self, device):
        return super().dev(device) | {"ks": self.ks.to(device), "vs": self.vs.to(device)}


def random_trees(new, seed=0, width=5, empty=0.0, own=True):
    """Masks (python integers) of the new rows of every sequence: ancestors and the row itself;
    a share `empty` of the rows sees no new token, without `own` none sees itself."""
    g = torch.Generator().manual_seed(seed)
    rows = []
    for n in new:
        mine = []
        for i in range(n):
            p = int(torch.randint(max(0, i - width), i, (1,), generator=g)) if i else -1
            mine.append((mine[p] if p >= 0 else 0) | 1 << i)
        for i in range(n):
            if float(torch.rand(1, generator=g)) < empty:
                mine[i] = 0
            elif not own:
                mine[i] &= ~(1 << i)
        rows += mine
    return rows


def tree_tensor(rows, N, words, fill=0):
    """int32 [N, words] of the masks; rows past them and what the words do not hold: `fill`, cut off."""
    t = torch.full((N, words), fill, dtype=torch.int32)
    full = (1 << 32 * words) - 1
    for r, bits in enumerate(rows):
        raw = (bits & full).to_bytes(4 * words, "little")
        t[r] = torch.frombuffer(bytearray(raw), dtype=torch.int32)
    return t


def visible(n, L, window, sinks, masks, words):
    """[n, L]: what the new rows of one sequence see."""
    base = L - n
    j = torch.arange(L)[None]
    own = torch.arange(base, L)[:, None]
    if masks is None:
        at, seen, new = own, j <= own, None
    else:
        new = torch.zeros(n, max(L, 1), dtype=torch.bool)[:, :L]
        at = torch.empty(n, 1, dtype=torch.long)
        for r, bits in enumerate(masks):
            bits &= (1 << min(n, 32 * words)) - 1
            at[r] = base + max(bin(bits).count("1"), 1) - 1
            for i in range(min(n, 32 * words)):
                if bits >> i & 1 and base + i >= 0:
                    new[r, base + i] = True
        seen = (j < base).expand(n, -1)
    if window > 0:
        seen = seen & ((j > at - window) | (j < sinks))
    if new is not None:
        seen = seen | new
    return seen & (own >= 0)


def cache_ref(case, scale, window=0, softcap=0.0, sinks=0, trees=None, words=0):
    """out, lse and their error bounds, [N, Hq, D] and [N, Hq] fp64; rows of no sequence are NaN in
    all four.  `trees`: the rows' masks, or None."""
    nan, codes = float("nan"), isinstance(case, Batch8)
    out = torch.full((case.N, case.Hq, case.D), nan, dtype=torch.float64)
    tol = torch.full_like(out, nan)
    lse = torch.full((case.N, case.Hq), nan, dtype=torch.float64)
    lse_tol = torch.full_like(lse, nan)
    t = case.q.dtype
    G, u = case.Hq // case.Hkv, half_step(t)
    # half a step of fp16 below 2^-14; over codes bf16 queries' weights are fp16 as well (up to 16 rows a head)
    tiny = 2.0 ** -25 if codes or t is torch.float16 else 0.0
    row0 = 0
    for b, (n, L) in enumerate(zip(case.new, case.lens_list)):
        if n == 0:
            continue
        rows = slice(row0, row0 + n)
        q = case.q[rows].double().view(n, case.Hkv, G, case.D).permute(1, 2, 0, 3)
        masks = trees[rows] if trees is not None else None
        row0 += n
        if L == 0:
            out[rows], tol[rows], lse[rows], lse_tol[rows] = 0, 0, -math.inf, 0
            continue
        k, v = case.cached(b, case.k), case.cached(b, case.v)
        z = torch.einsum("hgnd,hkd->hgnk", q, k) * scale
        # the products are exact in fp32; their sum and what follows (a code's scale among it) are not
        dz = torch.einsum("hgnd,hkd->hgnk", q.abs(), k.abs()) * abs(scale) * (case.D + 8 + 2 * codes) * U32
        if softcap > 0:
            z = softcap * torch.tanh(z / softcap)
            dz = dz + softcap * 2.0 ** -20
        seen = visible(n, L, window, sinks, masks, words)
        z = z.masked_fill(~seen, -math.inf)
        dz = torch.where(seen, dz, 0.0)
        e = torch.logsumexp(z, -1)
        none = ~seen.any(-1)
        p = torch.where(none[:, None], 0.0, torch.exp(z - torch.where(none, 0.0, e)[..., None]))
        o = torch.einsum("hgnk,hkd->hgnd", p, v)
        rel = 2 * dz.amax(-1) + 2.0 ** -20 + (L + 64 + 2 * codes) * U32
        absv = torch.einsum("hgnk,hkd->hgnd", p, v.abs())
        top = torch.where(none, 0.0, z.amax(-1))
        # weights below the type's normal range: half a step of each beside a value; over codes a
        # step is of the largest scale's next power of two, and the value a code of up to 128
        values = v.abs().sum(1)
        if codes:
            ids = case.table[b, :case.used[b]].long()
            vs = case.vs[ids].transpose(0, 1).flatten(1, 2)[:, :L].double()
            values = (128.0 * L * 2 * vs.amax(1))[:, None].expand(-1, case.D)
        small = tiny * torch.exp(top - torch.where(none, 0.0, e))[..., None] * values[:, None, None]
        err = (rel[..., None] + u) * absv + small
        err = err + u * (o.abs() + err) + torch.finfo(t).smallest_normal * u
        put = lambda x: x.permute(2, 0, 1, *range(3, x.dim())).reshape(n, case.Hq, *x.shape[3:])  # noqa: E731
        out[rows], tol[rows] = put(torch.where(none[:, None], 0.0, o)), put(err)
        lse[rows] = put(e)
        lse_tol[rows] = put(torch.where(none, 0.0, dz.amax(-1) + 2.0 ** -20 + (L + 64) * U32 + 4 * U32 * e.abs()))
    return out, lse, tol, lse_tol
