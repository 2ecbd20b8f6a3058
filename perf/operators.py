"""The operators around the routed-expert layer in a decoder block, as they are timed.

Three operators: ``norm`` (residual addition, RMSNorm, output in 16 or 32 bits
or in Q8_K blocks), ``rope`` (per-head Q/K norm, rotary positions with one or
several axes, append to a paged cache) and ``attn`` (attention of each
sequence's newest tokens over the paged cache: one token, a few, a chunk).

``run`` computes them in elementary torch operations (``own`` false) or through
the library's entry points (``own`` true) on what ``prepare`` made.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
WS_BYTES = 48 << 20  # at least moe_attention_workspace_bytes() of every shape


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _attn(name, B, new, ctx, Hq, Hkv, D, page, dtype, window=0, softcap=0.0, lse=False, spread=1):
    """``new`` and ``ctx``: (least, most) new tokens and total cached tokens of a sequence."""
    return {"name": name, "op": "attn", "B": B, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "dtype": dtype,
            "window": window, "softcap": softcap, "lse": lse, "spread": spread}


def _rope(name, B, new, ctx, Hq, Hkv, D, page, dtype, rot, axes, qk_norm, interleaved, spread=1):
    return {"name": name, "op": "rope", "B": B, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "dtype": dtype, "rot": rot,
            "axes": axes, "qk_norm": qk_norm, "interleaved": interleaved, "spread": spread}


def _norm(name, T, H, x, out):
    """``x``: the type of the branch output that is added; ``out``: "q8k" (fp32 rows
    and Q8_K blocks, the router's and the experts' input) or the type of the normed rows."""
    return {"name": name, "op": "norm", "T": T, "H": H, "x": x, "out": out}


def listed():
    return [
        # a chat's first answers: one new token over a short cache, where latency is all
        _attn("attn one token short", 1, (1, 1), (93, 93), 32, 4, 128, 16, "bf16"),
        # a serving batch in decode, sequences of very different lengths
        _attn("attn decode ragged", 48, (1, 1), (150, 12000), 32, 4, 128, 32, "fp16", lse=True),
        # one token at the end of a long document
        _attn("attn decode long", 1, (1, 1), (131071, 131071), 32, 4, 128, 64, "bf16"),
        # checking six drafted tokens of each of 16 sequences
        _attn("attn draft check", 16, (6, 6), (900, 8100), 64, 4, 128, 16, "bf16"),
        # a prompt of 4096 tokens into an empty cache
        _attn("attn prompt", 1, (4096, 4096), (4096, 4096), 32, 4, 128, 64, "bf16"),
        # chunks of three prompts far into their caches, small heads, capped scores, a sliding window
        _attn("attn chunks window", 3, (310, 1100), (6000, 20000), 16, 2, 64, 16, "fp16", window=4096,
              softcap=30.0, lse=True),
        # the pre-FFN norm of one token, in the form that the integer experts read
        _norm("norm one token q8k", 1, 2048, "fp32", "q8k"),
        # the same for a decode batch of odd size after a 16-bit output projection
        _norm("norm batch q8k", 333, 4096, "bf16", "q8k"),
        # the pre-attention norm of a prompt, 16-bit rows for the projections
        _norm("norm prompt bf16", 4096, 4096, "fp32", "bf16"),
        # one new token: per-head norm, rotation, append
        _rope("rope one token", 1, (1, 1), (700, 700), 32, 4, 128, 16, "bf16", 128, 1, True, False),
        # a decode batch with partial interleaved rotation and no per-head norm
        _rope("rope decode batch", 64, (1, 1), (10, 900), 16, 2, 64, 32, "fp16", 32, 1, False, True),
        # prompts with images: time, height and width positions
        _rope("rope prompt axes", 2, (2000, 2100), (2100, 2500), 64, 4, 128, 64, "bf16", 128, 3, True,
              False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    cap = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["attn", "attn", "norm", "rope"])
        dtype = rng.choice(["bf16", "fp16"])
        Hq, Hkv = rng.choice([(32, 4), (64, 4), (16, 2), (8, 8), (28, 4), (12, 2), (40, 8)])
        D = rng.choice([64, 128, 128])
        page = rng.choice([16, 32, 64, 128])
        spread = rng.randrange(1 << 20)
        if op == "norm":
            c = _norm("", _log(rng, 1, 8192), 256 * rng.choice([3, 8, 11, 16, 20, 32]),
                      rng.choice(["fp32", "bf16", "fp16"]), rng.choice(["q8k", "q8k", "bf16", "fp16", "fp32"]))
        elif op == "rope":
            B = _log(rng, 1, 64)
            new = _log(rng, 1, 1 if rng.random() < 0.4 else max(1, 8192 // B))
            ctx = new + _log(rng, 1, 1000)
            rot = rng.choice([D, D, D // 2])
            c = _rope("", B, (max(1, new // 2), new), (max(1, ctx // 3), ctx), Hq, Hkv, D, page, dtype, rot,
                      rng.choice([1, 1, 3]), rng.random() < 0.5, rng.random() < 0.3, spread)
        else:
            kind = rng.choice(["decode", "decode", "few", "chunk"])
            if kind == "decode":
                B, new, ctx = _log(rng, 1, 128), 1, _log(rng, 16, 100000)
            elif kind == "few":
                B, new, ctx = _log(rng, 1, 32), rng.randint(2, 12), _log(rng, 64, 16000)
            else:
                B, new = rng.randint(1, 4), _log(rng, 32, 4096)
                ctx = new + _log(rng, 1, 24000)
            # the plain form's padded scores and gathered caches have to fit several times over
            if B * new * ctx * Hq * 4 > 2.2e9 or B * ctx * Hkv * D * 4 > 2.2e9:
                continue
            c = _attn("", B, (max(1, new // 2), new), (max(1, ctx // 8) if kind == "decode" else max(new, ctx // 2), ctx),
                      Hq, Hkv, D, page, dtype, window=rng.choice([0, 0, 0, _log(rng, 16, 8192)]),
                      softcap=rng.choice([0.0, 0.0, 20.0, 50.0]), lse=rng.random() < 0.5, spread=spread)
        if _cost(c) <= cap:
            c.pop("name")
            return c


def _lens(c):
    """New tokens and total cached tokens of every sequence (the case alone decides them)."""
    r = random.Random(c["spread"])
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])]
    ctx = [max(n, _log(r, c["ctx_lo"], c["ctx_hi"])) for n in new]
    if c["B"] == 1:
        new, ctx = [c["new_hi"]], [max(c["new_hi"], c["ctx_hi"])]
    return new, ctx


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        out = n * 4 + n + n // 64 + n // 8 if c["out"] == "q8k" else n * SIZE[c["out"]]
        return {"bytes": n * SIZE[c["x"]] + n * 4 + n * 4 + out + c["H"] * 4, "flops": 6 * n}
    new, ctx = _lens(c)
    N, D, Hq, Hkv = sum(new), c["D"], c["Hq"], c["Hkv"]
    if c["op"] == "rope":
        row = (Hq + 2 * Hkv) * D
        return {"bytes": N * row * 2 * 2 + N * 4 * c["axes"], "flops": 8 * N * row}
    pairs = keys = 0
    for n, L in zip(new, ctx):
        w = c["window"]
        first = max(0, L - n + 1 - w) if w else 0  # the oldest key any of the new tokens sees
        keys += L - first
        if w:
            pairs += sum(min(L - n + i + 1, w) for i in range(n))
        else:
            pairs += n * (L - n) + n * (n + 1) // 2
    return {"bytes": 2 * keys * Hkv * D * 2 + 2 * N * Hq * D * 2 + (4 * N * Hq if c["lse"] else 0),
            "flops": 4 * pairs * Hq * D}


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _cache(c, g, ctx):
    """A paged cache that holds ``ctx`` tokens of each sequence, its pages in no order."""
    used = [-(-L // c["page"]) for L in ctx]
    total = sum(used) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(len(ctx), max(used), dtype=torch.int32, device=DEV)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    shape = (total, c["Hkv"], c["page"], c["D"])
    t = TYPES[c["dtype"]]
    return (torch.randn(shape, generator=g, device=DEV, dtype=t), torch.randn(shape, generator=g, device=DEV, dtype=t),
            table)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=DEV, dtype=dtype)

    s = {"case": c}
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        s |= {"x": normal(T, H, dtype=TYPES[c["x"]]), "residual": 3 * normal(T, H),
              "gamma": 1 + 0.2 * normal(H), "sum": torch.empty(T, H, device=DEV)}
        if c["out"] == "q8k":
            s |= {"y": torch.empty(T, H, device=DEV), "q": torch.empty(T, H, device=DEV, dtype=torch.int8),
                  "d": torch.empty(T, H // 256, device=DEV),
                  "sums": torch.empty(T, H // 32, device=DEV, dtype=torch.int32),
                  "values": torch.empty(T, H // 256, 256, device=DEV, dtype=torch.float16)}
        else:
            s["y"] = torch.empty(T, H, device=DEV, dtype=TYPES[c["out"]])
        return s
    new, ctx = _lens(c)
    N, D, Hq, Hkv = sum(new), c["D"], c["Hq"], c["Hkv"]
    t = TYPES[c["dtype"]]
    s["k"], s["v"], s["table"] = _cache(c, g, ctx)
    s["offs"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
    s["lens"] = torch.tensor(ctx, device=DEV, dtype=torch.int32)
    s["most"] = max(new)
    s["ws"] = torch.zeros(WS_BYTES, dtype=torch.uint8, device=DEV)
    if c["op"] == "attn":
        s |= {"q": normal(N, Hq, D, dtype=t), "scale": 1 / math.sqrt(D),
              "out": torch.empty(N, Hq, D, dtype=t, device=DEV),
              "lse": torch.empty(N, Hq, device=DEV) if c["lse"] else None}
        return s
    place = torch.cat([torch.arange(L - n, L, device=DEV) for n, L in zip(new, ctx)])
    # text runs along every axis; image patches share a time and differ in height and width
    pos = place[None].repeat(c["axes"], 1)
    if c["axes"] > 1:
        pos[1:] += torch.randint(0, 64, (c["axes"] - 1, N), generator=g, device=DEV)
    s |= {"qkv": normal(N, (Hq + 2 * Hkv) * D, dtype=t), "pos": pos.to(torch.int32).contiguous(),
          "inv_freq": 1e6 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"]),
          "axis": (torch.arange(c["rot"] // 2, device=DEV) * c["axes"] // (c["rot"] // 2)).to(torch.int32)
          if c["axes"] > 1 else None,
          "qw": 1 + 0.2 * normal(D) if c["qk_norm"] else None,
          "kw": 1 + 0.2 * normal(D) if c["qk_norm"] else None,
          "q_out": torch.empty(N, Hq, D, dtype=t, device=DEV)}
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "rope": _own_rope, "attn": _own_attn}[op](state)
    return {"norm": _plain_norm, "rope": _plain_rope, "attn": _plain_attn}[op](state)


def _own_norm(s):
    from quantized_routed_expert_02_gb300 import moeq4k as m
    if s["case"]["out"] == "q8k":
        m.moe_add_rmsnorm(s["x"], s["residual"], s["gamma"], EPS, sum_out=s["sum"], y=s["y"],
                          q8k=(s["q"], s["d"], s["sums"]))
        torch.mul(s["q"].view(s["values"].shape), s["d"].unsqueeze(-1), out=s["values"])
        return {"sum": s["sum"], "y": s["y"], "values": s["values"]}
    m.moe_add_rmsnorm(s["x"], s["residual"], s["gamma"], EPS, sum_out=s["sum"], y=s["y"])
    return {"sum": s["sum"], "y": s["y"]}


def _plain_norm(s):
    c = s["case"]
    h = s["residual"] + s["x"].float()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["gamma"]
    if c["out"] != "q8k":
        return {"sum": h, "y": y.to(TYPES[c["out"]])}
    b = y.view(c["T"], -1, 256)
    most = b.abs().amax(2, keepdim=True)
    codes = torch.round(b * torch.where(most > 0, 127 / most, 0))
    return {"sum": h, "y": y, "values": (codes * (most / 127)).to(torch.float16)}


def _own_rope(s):
    from quantized_routed_expert_02_gb300 import moeq4k as m
    m.moe_rope_append(s["qkv"], s["pos"], s["inv_freq"], s["q_out"], s["k"], s["v"], s["table"], s["offs"],
                      s["lens"], s["ws"], axis=s["axis"], q_norm_w=s["qw"], k_norm_w=s["kw"], eps=EPS,
                      interleaved=s["case"]["interleaved"])
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _plain_rope(s):
    c = s["case"]
    N, D, Hq, Hkv, rot = s["qkv"].shape[0], c["D"], c["Hq"], c["Hkv"], c["rot"]
    rows = s["qkv"].float().view(N, Hq + 2 * Hkv, D)
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    if c["qk_norm"]:
        q = q / torch.sqrt((q * q).mean(2, keepdim=True) + EPS) * s["qw"]
        k = k / torch.sqrt((k * k).mean(2, keepdim=True) + EPS) * s["kw"]
    p = s["pos"][s["axis"].long()].t() if s["axis"] is not None else s["pos"][0][:, None]
    angle = p.double() * s["inv_freq"]  # far positions need 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x):
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        u, w = a * cos - b * sin, b * cos + a * sin
        r = torch.stack((u, w), -1).flatten(-2) if c["interleaved"] else torch.cat((u, w), -1)
        return torch.cat((r, x[..., rot:]), -1)

    t = TYPES[c["dtype"]]
    n = (s["offs"][1:] - s["offs"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(c["B"], device=DEV), n, output_size=N)
    at = torch.arange(N, device=DEV) - s["offs"].long()[seq] + (s["lens"].long() - n)[seq]
    page, row = s["table"].long()[seq, at // c["page"]], at % c["page"]
    s["k"][page, :, row] = turned(k).to(t)
    s["v"][page, :, row] = v.to(t)
    return {"q": turned(q).to(t), "k": s["k"], "v": s["v"]}


def _own_attn(s):
    from quantized_routed_expert_02_gb300 import moeq4k as m
    c = s["case"]
    m.moe_attention_paged(s["q"], s["k"], s["v"], s["table"], s["offs"], s["lens"], s["most"], s["scale"],
                          s["out"], s["ws"], lse=s["lse"], window=c["window"], softcap=c["softcap"])
    return {"out": s["out"], "lse": s["lse"]} if c["lse"] else {"out": s["out"]}


def _plain_attn(s):
    c = s["case"]
    B, D, Hq, Hkv, most = c["B"], c["D"], c["Hq"], c["Hkv"], s["most"]
    N, G = s["q"].shape[0], Hq // Hkv
    cached = lambda pages: pages[s["table"].long()].transpose(1, 2).flatten(2, 3).float()  # noqa: E731
    n, L = (s["offs"][1:] - s["offs"][:-1]).long(), s["lens"].long()
    i = torch.arange(most, device=DEV)
    token = (s["offs"][:-1].long()[:, None] + i).clamp(max=N - 1)  # [B, most], padded
    q = s["q"].float()[token].view(B, most, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * most, D)
    score = (q @ cached(s["k"]).transpose(2, 3)).mul_(s["scale"])
    if c["softcap"]:
        score.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    at = (L - n)[:, None, None] + i[:, None]  # [B, most, 1]
    key = torch.arange(score.shape[3], device=DEV)
    seen = (key <= at) & (key < L[:, None, None])
    if c["window"]:
        seen &= key > at - c["window"]
    score.view(B, Hkv, G, most, -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(3, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    out = (p @ cached(s["v"])) / total
    lse = (top + total.log()).view(B, Hkv, G, most)
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), n, output_size=N)
    row = torch.arange(N, device=DEV) - s["offs"].long()[seq]
    out = out.view(B, Hkv, G, most, D)[seq, :, :, row].reshape(N, Hq, D).to(TYPES[c["dtype"]])
    return {"out": out, "lse": lse[seq, :, :, row].reshape(N, Hq)} if c["lse"] else {"out": out}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "norm":
        h = s["residual"].double().add_(s["x"])
        y = h * s["gamma"].double() * h.pow(2).mean(-1, keepdim=True).add(EPS).rsqrt()
        if c["out"] != "q8k":
            return {"sum": h, "y": y}
        blocks = y.unflatten(1, (-1, 256))
        step = blocks.abs().amax(-1, keepdim=True) / 127
        return {"sum": h, "y": y, "values": torch.nan_to_num((blocks / step).round() * step)}
    new, ctx = _lens(c)
    D, Hq, Hkv, page = c["D"], c["Hq"], c["Hkv"], c["page"]
    starts = [sum(new[:b]) for b in range(len(new))]
    if c["op"] == "rope":
        x = s["qkv"].double().unflatten(1, (-1, D))
        half = c["rot"] // 2
        for part, w in ((x[:, :Hq], s["qw"]), (x[:, Hq:Hq + Hkv], s["kw"])):
            if w is not None:
                part *= part.square().mean(-1, keepdim=True).add(EPS).rsqrt() * w.double()
        first = torch.arange(half, device=DEV) * (2 if c["interleaved"] else 1)
        second = first + (1 if c["interleaved"] else half)
        which = s["axis"].tolist() if s["axis"] is not None else [0] * half
        angle = torch.stack([s["pos"][which[j]].double() * s["inv_freq"][j] for j in range(half)], 1)
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        both = torch.complex(x[:, :Hq + Hkv, first], x[:, :Hq + Hkv, second]) * turn
        x[:, :Hq + Hkv, first] = both.real
        x[:, :Hq + Hkv, second] = both.imag
        k, v = s["k"].double(), s["v"].double()
        for b, (n, L) in enumerate(zip(new, ctx)):
            where = torch.arange(L - n, L, device=DEV)
            slots = s["table"][b].long()[torch.div(where, page, rounding_mode="floor")]
            mine = x[starts[b]:starts[b] + n]
            k[slots, :, where % page] = mine[:, Hq:Hq + Hkv]
            v[slots, :, where % page] = mine[:, Hq + Hkv:]
        return {"q": x[:, :Hq], "k": k, "v": v}
    out = torch.zeros(sum(new), Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(sum(new), Hq, dtype=torch.float64, device=DEV)
    for b, (n, L) in enumerate(zip(new, ctx)):
        pages = s["table"][b, :-(-L // page)].long()
        for h in range(Hkv):
            k = s["k"][pages, h].reshape(-1, D)[:L].double()
            v = s["v"][pages, h].reshape(-1, D)[:L].double()
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            q = s["q"][starts[b]:starts[b] + n, heads].double()
            a = torch.einsum("nhd,kd->nhk", q, k) * s["scale"]
            if c["softcap"]:
                a = torch.tanh(a / c["softcap"]) * c["softcap"]
            behind = torch.arange(L - n, L, device=DEV)[:, None] - torch.arange(L, device=DEV)
            hidden = behind < 0
            if c["window"]:
                hidden |= behind >= c["window"]
            a = a.masked_fill(hidden[:, None], -math.inf)
            e = torch.logsumexp(a, -1)
            lse[starts[b]:starts[b] + n, heads] = e
            out[starts[b]:starts[b] + n, heads] = torch.einsum("nhk,kd->nhd", torch.exp(a - e[..., None]), v)
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}
