"""The cache's further operators, as they are timed: 8-bit codes, drafted trees, attention sinks.

Four operators: ``append8`` (per-head Q/K norm, rotary positions, keys and values
quantised into a paged cache of 8-bit codes), ``attn`` (attention over the paged
cache: over 8-bit codes, of the nodes of a tree of drafted tokens, with a sliding
window beside first tokens that stay visible, and what they make together) and
``keep`` (the accepted path of a drafted tree moves to its place in the cache).

``run`` computes them in elementary torch operations (``own`` false) or through
the library's entry points (``own`` true) on what ``prepare`` made.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
WS_BYTES = 48 << 20  # at least moe_attention_workspace_bytes() of every shape


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _attn(name, B, new, ctx, Hq, Hkv, D, page, dtype, q8=False, tree=False, window=0, sinks=0, softcap=0.0,
          lse=False, spread=1):
    """``new`` and ``ctx``: (least, most) new tokens and total cached tokens of a sequence."""
    return {"name": name, "op": "attn", "B": B, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "dtype": dtype, "q8": q8,
            "tree": tree, "window": window, "sinks": sinks, "softcap": softcap, "lse": lse, "spread": spread}


def _append(name, B, new, ctx, Hq, Hkv, D, page, dtype, rot, axes, qk_norm, interleaved, spread=1):
    return {"name": name, "op": "append8", "B": B, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "dtype": dtype, "rot": rot,
            "axes": axes, "qk_norm": qk_norm, "interleaved": interleaved, "spread": spread}


def _keep(name, B, new, ctx, most, Hkv, D, page, dtype, spread=1):
    """``most``: the longest accepted path of a sequence."""
    return {"name": name, "op": "keep", "B": B, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "keep_hi": most, "Hkv": Hkv, "D": D, "page": page, "dtype": dtype, "spread": spread}


def listed():
    return [
        # one new token of a chat into the 8-bit cache, where latency is all
        _append("append8 one token", 1, (1, 1), (40, 40), 32, 4, 128, 16, "bf16", 128, 1, True, False),
        # two prompts with images (time, height and width positions) into the 8-bit cache
        _append("append8 prompt axes", 2, (2000, 2100), (2100, 2500), 64, 4, 128, 64, "fp16", 128, 3, True, False),
        # a chat's first answers from the 8-bit cache
        _attn("attn8 one token short", 1, (1, 1), (93, 93), 32, 4, 128, 16, "bf16", q8=True),
        # a serving batch in decode, sequences of very different lengths, 8-bit cache
        _attn("attn8 decode ragged", 48, (1, 1), (150, 12000), 32, 4, 128, 32, "fp16", q8=True, lse=True),
        # a chunk of a long document's prompt far into its 8-bit cache
        _attn("attn8 chunk", 1, (2048, 2048), (16384, 16384), 32, 4, 128, 64, "bf16", q8=True),
        # a small tree of drafts of one chat, a head of its own for every query head
        _attn("tree one sequence", 1, (12, 12), (700, 700), 8, 8, 128, 16, "bf16", tree=True),
        # trees of some 60 drafts of each of 16 sequences
        _attn("tree batch", 16, (48, 64), (900, 8100), 64, 4, 128, 16, "fp16", tree=True, lse=True),
        # larger trees over the 8-bit cache with a window, sinks and capped scores, small heads
        _attn("tree8 window", 6, (70, 110), (6000, 20000), 16, 2, 64, 32, "bf16", q8=True, tree=True, window=4096,
              sinks=4, softcap=30.0),
        # a decode batch of endless chats: a window, and the first tokens
        _attn("sinks decode", 32, (1, 1), (3000, 30000), 32, 4, 128, 32, "bf16", window=2048, sinks=4, lse=True),
        # a prompt of such a model
        _attn("sinks prompt", 1, (4096, 4096), (4096, 4096), 32, 4, 128, 64, "fp16", window=1000, sinks=64),
        # one chat's accepted drafts
        _keep("keep one sequence", 1, (24, 24), (700, 700), 5, 4, 128, 16, "bf16"),
        # the accepted drafts of a serving batch, deep trees
        _keep("keep batch", 64, (60, 250), (300, 3000), 24, 8, 128, 64, "fp16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    cap = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["attn", "attn", "attn", "append8", "keep"])
        dtype = rng.choice(["bf16", "fp16"])
        Hq, Hkv = rng.choice([(32, 4), (64, 4), (16, 2), (8, 8), (28, 4), (12, 2), (40, 8)])
        D = rng.choice([64, 128, 128])
        page = rng.choice([16, 32, 64, 128])
        spread = rng.randrange(1 << 20)
        if op == "append8":
            B = _log(rng, 1, 64)
            new = _log(rng, 1, 1 if rng.random() < 0.4 else max(1, 8192 // B))
            ctx = new + _log(rng, 1, 1000)
            c = _append("", B, (max(1, new // 2), new), (max(1, ctx // 3), ctx), Hq, Hkv, D, page, dtype,
                        rng.choice([D, D, D // 2]), rng.choice([1, 1, 3]), rng.random() < 0.5, rng.random() < 0.3,
                        spread)
        elif op == "keep":
            B, new = _log(rng, 1, 64), _log(rng, 3, 256)
            most = rng.randint(1, max(1, min(32, new // 4)))
            ctx = new + _log(rng, 1, 3000)
            c = _keep("", B, (max(1, new // 2), new), (max(new, ctx // 2), ctx), most, Hkv, D, page, dtype, spread)
        else:
            kind = rng.choice(["q8", "q8", "tree", "tree8", "sinks", "sinks8"])
            window, sinks = 0, 0
            if kind.startswith("sinks"):
                window, sinks = _log(rng, 16, 8192), _log(rng, 1, 200)
            elif rng.random() < 0.25:
                window = _log(rng, 16, 8192)
                sinks = rng.choice([0, _log(rng, 1, 200)])
            if kind.startswith("tree"):
                B, new = _log(rng, 1, 32), _log(rng, 2, 256)
                ctx = new + _log(rng, 1, 16000)
            else:
                part = rng.choice(["decode", "decode", "few", "chunk"])
                if part == "decode":
                    B, new, ctx = _log(rng, 1, 128), 1, _log(rng, 16, 100000)
                elif part == "few":
                    B, new, ctx = _log(rng, 1, 32), rng.randint(2, 12), _log(rng, 64, 16000)
                else:
                    B, new = rng.randint(1, 4), _log(rng, 32, 4096)
                    ctx = new + _log(rng, 1, 24000)
            # the plain form's padded scores and gathered caches have to fit several times over
            if B * new * ctx * Hq * 4 > 2.2e9 or B * ctx * Hkv * D * 4 > 2.2e9:
                continue
            few = new == 1 and not kind.startswith("tree")
            c = _attn("", B, (max(1, new // 2), new), (max(1, ctx // 8) if few else max(new, ctx // 2), ctx), Hq, Hkv,
                      D, page, dtype, q8=kind in ("q8", "tree8", "sinks8"), tree=kind.startswith("tree"),
                      window=window, sinks=sinks, softcap=rng.choice([0.0, 0.0, 20.0, 50.0]), lse=rng.random() < 0.5,
                      spread=spread)
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


def _trees(c, new):
    """The ancestors of every drafted token, itself among them, as the bits of an integer; a
    token's parent is one of the twelve before it, so that trees are some ten deep and bushy."""
    r = random.Random(c["spread"] + 1)
    rows = []
    for n in new:
        mine = [1]
        for i in range(1, n):
            mine.append(mine[r.randrange(max(0, i - 12), i)] | 1 << i)
        rows += mine
    return rows


def _paths(c, new):
    """The accepted path of every sequence: places among its new tokens, rising.  The trees are
    laid out by depth: what moves comes from behind the path's own length."""
    r = random.Random(c["spread"] + 2)
    paths = []
    for n in new:
        k = r.randint(max(1, c["keep_hi"] // 2), c["keep_hi"])
        k = max(1, min(k, (n + 1) // 2))
        paths.append([0] + sorted(r.sample(range(k, n), k - 1)))
    return paths


def work(case):
    c = case
    new, ctx = _lens(c)
    N, D, Hkv = sum(new), c["D"], c["Hkv"]
    if c["op"] == "keep":
        moved = sum(sum(i != j for j, i in enumerate(p)) for p in _paths(c, new))
        return {"bytes": moved * Hkv * D * 2 * 2 * 2 + sum(4 * len(p) for p in _paths(c, new)) + 16 * c["B"], "flops": 0}
    Hq = c["Hq"]
    if c["op"] == "append8":
        row = (Hq + 2 * Hkv) * D
        return {"bytes": N * (row * 2 + Hq * D * 2 + 2 * Hkv * (D + 4) + 4 * c["axes"]), "flops": N * (8 * row + 4 * Hkv * D)}
    w, sinks = c["window"], c["sinks"]
    near = lambda at: at + 1 if not w else min(at + 1, w) + min(sinks, max(0, at + 1 - w))  # noqa: E731
    pairs = keys = 0
    trees = iter(_trees(c, new)) if c["tree"] else None
    for n, L in zip(new, ctx):
        base = L - n
        first = max(0, base + 1 - w) if w else 0  # the oldest key, but the sinks, any of the new tokens sees
        keys += L - first + min(sinks, first)
        for i in range(n):
            if trees is None:
                pairs += near(base + i)
                continue
            own_path = bin(next(trees)).count("1")
            lo = max(0, base + own_path - w) if w else 0  # of the cached tokens, behind its place in the text
            pairs += max(0, base - lo) + min(sinks, lo, base) + own_path
    size = D + 4 if c["q8"] else 2 * D
    more = 4 * N * -(-max(new) // 32) if c["tree"] else 0
    return {"bytes": 2 * keys * Hkv * size + 2 * N * Hq * D * 2 + (4 * N * Hq if c["lse"] else 0) + more,
            "flops": 4 * pairs * Hq * D}


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _cache(c, g, ctx, q8):
    """A paged cache that holds ``ctx`` tokens of each sequence, its pages in no order: keys and
    values [2, pages, Hkv, page, D] of the case's type, or 8-bit codes and their scales."""
    used = [-(-L // c["page"]) for L in ctx]
    total = sum(used) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(len(ctx), max(used), dtype=torch.int32, device=DEV)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    shape = (2, total, c["Hkv"], c["page"], c["D"])
    if not q8:
        return torch.randn(shape, generator=g, device=DEV, dtype=TYPES[c["dtype"]]), None, table
    # a token's head as it is quantised: the largest magnitude gives code 127 or -127
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float16)
    most = x.abs().amax(-1, keepdim=True).float()
    codes = (x * (127 / most)).round_().to(torch.int8)
    return codes, (most / 127).squeeze(-1).contiguous(), table


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=DEV, dtype=dtype)

    new, ctx = _lens(c)
    N, D, Hkv, t = sum(new), c["D"], c["Hkv"], TYPES[c["dtype"]]
    q8 = c["op"] == "append8" or c.get("q8", False)
    kv, scales, table = _cache(c, g, ctx, q8)
    s = {"case": c, "kv": kv, "scales": scales, "table": table, "most": max(new),
         "offs": torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32),
         "lens": torch.tensor(ctx, device=DEV, dtype=torch.int32),
         "ws": torch.zeros(WS_BYTES, dtype=torch.uint8, device=DEV)}
    if c["op"] == "keep":
        paths = _paths(c, new)
        keep = torch.zeros(c["B"], c["keep_hi"], dtype=torch.int32)
        for b, p in enumerate(paths):
            keep[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        return s | {"keep": keep.to(DEV), "kept": torch.tensor([len(p) for p in paths], dtype=torch.int32, device=DEV)}
    Hq = c["Hq"]
    if c["op"] == "attn":
        if c["tree"]:
            words = -(-max(new) // 32)
            raw = b"".join(r.to_bytes(4 * words, "little") for r in _trees(c, new))
            s["tree"] = torch.frombuffer(bytearray(raw), dtype=torch.int32).view(N, words).to(DEV)
        return s | {"q": normal(N, Hq, D, dtype=t), "scale": 1 / math.sqrt(D),
                    "out": torch.empty(N, Hq, D, dtype=t, device=DEV),
                    "lse": torch.empty(N, Hq, device=DEV) if c["lse"] else None}
    place = torch.cat([torch.arange(L - n, L, device=DEV) for n, L in zip(new, ctx)])
    # text runs along every axis; image patches share a time and differ in height and width
    pos = place[None].repeat(c["axes"], 1)
    if c["axes"] > 1:
        pos[1:] += torch.randint(0, 64, (c["axes"] - 1, N), generator=g, device=DEV)
    return s | {"qkv": normal(N, (Hq + 2 * Hkv) * D, dtype=t), "pos": pos.to(torch.int32).contiguous(),
                "inv_freq": 1e6 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"]),
                "axis": (torch.arange(c["rot"] // 2, device=DEV) * c["axes"] // (c["rot"] // 2)).to(torch.int32)
                if c["axes"] > 1 else None,
                "qw": 1 + 0.2 * normal(D) if c["qk_norm"] else None,
                "kw": 1 + 0.2 * normal(D) if c["qk_norm"] else None,
                "q_out": torch.empty(N, Hq, D, dtype=t, device=DEV),
                "values": torch.empty(kv.shape, dtype=torch.float16, device=DEV)}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"append8": _own_append, "attn": _own_attn, "keep": _own_keep}[op](state)
    return {"append8": _plain_append, "attn": _plain_attn, "keep": _plain_keep}[op](state)


def _own_append(s):
    from quantized_routed_expert_02_gb300 import moeq4k as m
    k, v = s["kv"]
    ks, vs = s["scales"]
    m.moe_rope_append_q8(s["qkv"], s["pos"], s["inv_freq"], s["q_out"], k, v, ks, vs, s["table"], s["offs"],
                         s["lens"], s["ws"], axis=s["axis"], q_norm_w=s["qw"], k_norm_w=s["kw"], eps=EPS,
                         interleaved=s["case"]["interleaved"])
    torch.mul(s["kv"], s["scales"].unsqueeze(-1), out=s["values"])
    return {"q": s["q_out"], "kv": s["values"]}


def _places(s):
    """The sequence of every row, its page and its row of the page."""
    page, N = s["case"]["page"], s["qkv"].shape[0]
    n = (s["offs"][1:] - s["offs"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(len(n), device=DEV), n, output_size=N)
    at = torch.arange(N, device=DEV) - s["offs"].long()[seq] + (s["lens"].long() - n)[seq]
    return s["table"].long()[seq, at // page], at % page


def _plain_append(s):
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

    page, row = _places(s)
    both = torch.stack((turned(k), v))  # [2, N, Hkv, D]
    most = both.abs().amax(-1, keepdim=True)
    codes = torch.round(both * torch.where(most > 0, 127 / most, 0))
    s["kv"][:, page, :, row] = codes.to(torch.int8).transpose(0, 1)
    s["scales"][:, page, :, row] = (most / 127).squeeze(-1).transpose(0, 1)
    torch.mul(s["kv"], s["scales"].unsqueeze(-1), out=s["values"])
    return {"q": turned(q).to(TYPES[c["dtype"]]), "kv": s["values"]}


def _own_attn(s):
    from quantized_routed_expert_02_gb300 import moeq4k as m
    c = s["case"]
    k, v = s["kv"]
    ks, vs = s["scales"] if c["q8"] else (None, None)
    m.moe_attention_cache(s["q"], k, v, s["table"], s["offs"], s["lens"], s["most"], s["scale"], s["out"], s["ws"],
                          k_scales=ks, v_scales=vs, tree=s.get("tree"), sinks=c["sinks"], lse=s["lse"],
                          window=c["window"], softcap=c["softcap"])
    return {"out": s["out"], "lse": s["lse"]} if c["lse"] else {"out": s["out"]}


def _plain_attn(s):
    c = s["case"]
    B, D, Hq, Hkv, most = c["B"], c["D"], c["Hq"], c["Hkv"], s["most"]
    N, G = s["q"].shape[0], Hq // Hkv
    pages = s["table"].long()

    def cached(i):
        x = s["kv"][i][pages].float()
        if c["q8"]:
            x = x * s["scales"][i][pages].unsqueeze(-1)
        return x.transpose(1, 2).flatten(2, 3)

    n, L = (s["offs"][1:] - s["offs"][:-1]).long(), s["lens"].long()
    i = torch.arange(most, device=DEV)
    token = (s["offs"][:-1].long()[:, None] + i).clamp(max=N - 1)  # [B, most], padded
    q = s["q"].float()[token].view(B, most, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * most, D)
    score = (q @ cached(0).transpose(2, 3)).mul_(s["scale"])
    if c["softcap"]:
        score.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    base = (L - n)[:, None, None]
    key = torch.arange(score.shape[3], device=DEV)
    if c["tree"]:
        bit = key - base  # [B, 1, keys]: a key's place among the new tokens
        word = (bit >> 5).clamp(0, s["tree"].shape[1] - 1).expand(B, most, -1)
        path = (s["tree"][token].gather(2, word) >> (bit & 31)) & 1
        path = (path != 0) & (bit >= 0) & (bit < n[:, None, None])
        at = base + path.sum(2, keepdim=True) - 1
        seen = key < base
    else:
        at = base + i[:, None]  # [B, most, 1]
        seen = (key <= at) & (key < L[:, None, None])
    if c["window"]:
        seen = seen & ((key > at - c["window"]) | (key < c["sinks"]))
    if c["tree"]:
        seen = seen | path
    score.view(B, Hkv, G, most, -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(3, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    out = (p @ cached(1)) / total
    lse = (top + total.log()).view(B, Hkv, G, most)
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), n, output_size=N)
    row = torch.arange(N, device=DEV) - s["offs"].long()[seq]
    out = out.view(B, Hkv, G, most, D)[seq, :, :, row].reshape(N, Hq, D).to(TYPES[c["dtype"]])
    return {"out": out, "lse": lse[seq, :, :, row].reshape(N, Hq)} if c["lse"] else {"out": out}


def _own_keep(s):
    from quantized_routed_expert_02_gb300 import moeq4k as m
    k, v = s["kv"]
    m.moe_cache_keep(k, v, s["table"], s["offs"], s["lens"], s["keep"], s["kept"], s["ws"])
    return {"kv": s["kv"]}


def _plain_keep(s):
    c = s["case"]
    page = c["page"]
    base = (s["lens"] - (s["offs"][1:] - s["offs"][:-1])).long()[:, None]
    j = torch.arange(s["keep"].shape[1], device=DEV)[None]
    # an entry past a path's end moves the path's first row onto itself
    live = j < s["kept"][:, None]
    src, dst = base + torch.where(live, s["keep"], 0), base + torch.where(live, j, 0)
    seq = torch.arange(c["B"], device=DEV)[:, None]
    table = s["table"].long()
    rows = s["kv"][:, table[seq, src // page], :, src % page]
    s["kv"][:, table[seq, dst // page], :, dst % page] = rows
    return {"kv": s["kv"]}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    new, ctx = _lens(c)
    D, Hkv, page = c["D"], c["Hkv"], c["page"]
    starts = [sum(new[:b]) for b in range(len(new))]
    slot = lambda b, j: (s["table"][b].long()[torch.div(j, page, rounding_mode="floor")], j % page)  # noqa: E731
    if c["op"] == "keep":
        kv = s["kv"].double()
        for b, (n, L, path) in enumerate(zip(new, ctx, _paths(c, new))):
            for d, i in enumerate(path):
                (p0, r0), (p1, r1) = (slot(b, torch.tensor(L - n + x, device=DEV)) for x in (i, d))
                kv[:, p1, :, r1] = kv[:, p0, :, r0].clone()
        return {"kv": kv}
    Hq = c["Hq"]
    if c["op"] == "append8":
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
        step = x.abs().amax(-1, keepdim=True) / 127
        rounded = torch.nan_to_num((x / step).round() * step)
        kv = s["kv"].double() * s["scales"].double().unsqueeze(-1)
        for b, (n, L) in enumerate(zip(new, ctx)):
            pages, rows = slot(b, torch.arange(L - n, L, device=DEV))
            mine = rounded[starts[b]:starts[b] + n]
            kv[0, pages, :, rows] = mine[:, Hq:Hq + Hkv]
            kv[1, pages, :, rows] = mine[:, Hq + Hkv:]
        return {"q": x[:, :Hq], "kv": kv}
    out = torch.zeros(sum(new), Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(sum(new), Hq, dtype=torch.float64, device=DEV)
    trees = _trees(c, new) if c["tree"] else None
    for b, (n, L) in enumerate(zip(new, ctx)):
        pages = s["table"][b, :-(-L // page)].long()
        keys = torch.arange(L, device=DEV)
        if trees is None:
            at = torch.arange(L - n, L, device=DEV)
            hidden = keys > at[:, None]
        else:
            mine = trees[starts[b]:starts[b] + n]
            at = torch.tensor([L - n - 1 + bin(r).count("1") for r in mine], device=DEV)
            hidden = torch.zeros(n, L, dtype=torch.bool)
            hidden[:, L - n:] = torch.tensor([[not r >> i & 1 for i in range(n)] for r in mine])
            hidden = hidden.to(DEV)
        if c["window"]:
            far = (at[:, None] - keys >= c["window"]) & (keys >= c["sinks"])
            if trees is not None:
                far[:, L - n:] = False
            hidden |= far
        for h in range(Hkv):
            k, v = (s["kv"][i, pages, h].reshape(-1, D)[:L].double() for i in range(2))
            if c["q8"]:
                ks, vs = (s["scales"][i, pages, h].reshape(-1)[:L].double() for i in range(2))
                k, v = k * ks[:, None], v * vs[:, None]
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            q = s["q"][starts[b]:starts[b] + n, heads].double()
            a = torch.einsum("nhd,kd->nhk", q, k) * s["scale"]
            if c["softcap"]:
                a = torch.tanh(a / c["softcap"]) * c["softcap"]
            a = a.masked_fill(hidden[:, None], -math.inf)
            e = torch.logsumexp(a, -1)
            lse[starts[b]:starts[b] + n, heads] = e
            out[starts[b]:starts[b] + n, heads] = torch.einsum("nhk,kd->nhd", torch.exp(a - e[..., None]), v)
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}
