"""What the paged cache has beside its 16-bit chains, through the C ABI against
64-bit references: the append in 8-bit codes, attention over them, of trees of
drafted tokens and with sinks, and the accepted path's move."""
import math

import pytest

from tests.block_cases import Batch, inv_freq, rope_ref
from tests.cache_cases import Batch8, cache_ref, quantised, random_trees, tree_tensor
from tests.test_gpu_attention_half import EPS, run_rope, within
from tests.test_gpu_parity import DEV, m  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF16, F16 = torch.bfloat16, torch.float16


def same(a, b):
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


# --------------------------------------------------------------------------
# moe_rope_append_q8
# --------------------------------------------------------------------------
def run_rope8(m, case, pos, rot, axis=None, qk_norm=False, interleaved=False, seed=1, qkv=None):
    """As run_rope, into the codes of a Batch8; the same rows and weights for the same seed."""
    g = torch.Generator().manual_seed(seed)
    N, Hq, Hkv, D, dtype = case.N, case.Hq, case.Hkv, case.D, case.dtype
    rows = torch.randn(N, (Hq + 2 * Hkv) * D, generator=g).to(dtype)
    qkv = rows if qkv is None else qkv
    qw = 1 + 0.3 * torch.randn(D, generator=g) if qk_norm else None
    kw = 1 + 0.3 * torch.randn(D, generator=g) if qk_norm else None
    f = inv_freq(rot)
    d = case.dev(DEV)
    q_out = torch.full((N, Hq, D), float("nan"), dtype=dtype, device=DEV)
    ws = m.alloc_attention_workspace(Hq, Hkv, D, device=DEV)
    up = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    m.moe_rope_append_q8(qkv.to(DEV), pos.to(DEV), f.to(DEV), q_out, d["k"], d["v"], d["ks"], d["vs"], d["table"],
                         d["offs"], d["lens"], ws, axis=up(axis), q_norm_w=up(qw), k_norm_w=up(kw), eps=EPS,
                         interleaved=interleaved)
    code, detail = m.moe_read_device_status(ws)
    _, k, v, _, ke = rope_ref(qkv, pos, f, axis, Hq, Hkv, D, qw, kw, EPS, interleaved)
    # rope_ref's bound of k rounds to the 16-bit type; before that rounding what is left of it
    ke = ke - torch.finfo(dtype).eps / 2 * k.abs() * (1 - 2.0 ** -20)
    return dict(q_out=q_out.cpu(), code=code, detail=detail, k_ref=k, v_ref=v, ke=ke, qkv=qkv,
                **{n: d[n].cpu() for n in ("k", "v", "ks", "vs")})


def check_rope8(case, r):
    """V's codes and scales bit for bit; K's values within half a step and what fp32 adds."""
    assert r["code"] == 0
    written = torch.zeros(case.k.shape[:3], dtype=torch.bool)
    row = 0
    vc, vd = quantised(r["v_ref"])
    for b, (n, L) in enumerate(zip(case.new, case.lens_list)):
        for i in range(n):
            j = L - n + i
            if j < 0:
                continue
            pg, at = int(case.table[b, j // case.page]), j % case.page
            assert torch.equal(r["v"][pg, :, at], vc[row + i]) and torch.equal(r["vs"][pg, :, at], vd[row + i])
            want, err = r["k_ref"][row + i], r["ke"][row + i]
            d, most = r["ks"][pg, :, at].double(), want.abs().amax(-1)
            assert bool(((d - most / 127).abs() <= err.amax(-1) / 127 + 2.0 ** -24 * d).all())
            got = r["k"][pg, :, at].double()
            assert bool((got.abs() <= 127).all())
            # half a step of the code, the product's rounding and the factor's (2 steps at 127), the values' own
            tol = d[:, None] * (0.5 + 127 * 3 * 2.0 ** -24) + err + err.amax(-1, keepdim=True)
            within(got * d[:, None], want, tol, f"k {b},{i}")
            written[pg, :, at] = True
        row += n
    for new, old in ((r["k"], case.k), (r["v"], case.v), (r["ks"], case.ks), (r["vs"], case.vs)):
        a, o = new[~written], old[~written]
        assert same(a.float(), o.float())
    return written


ROPE = [
    # new, lens, Hq, Hkv, D, page, rot
    ([1], [1], 4, 1, 128, 16, 128),
    ([1], [700], 32, 4, 128, 16, 128),
    ([5, 0, 1, 17], [5, 9, 33, 40], 28, 4, 128, 32, 64),
    ([3, 2], [64, 65], 8, 8, 64, 64, 64),
    ([40, 1], [40, 256], 12, 2, 64, 128, 16),
    ([7], [300], 3, 1, 64, 256, 48),
    ([5, 3], [2, 30], 5, 5, 128, 16, 32),
    ([2000], [2100], 16, 2, 64, 16, 32),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("qk_norm", [False, True])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D,page,rot", ROPE)
def test_append(m, new, lens, Hq, Hkv, D, page, rot, qk_norm, interleaved, dtype):
    args = (new, lens, Hq, Hkv, D, page, dtype)
    pos = torch.cat([torch.arange(L - n, L) for n, L in zip(new, lens)] + [torch.zeros(2, dtype=torch.long)])
    pos = pos[None].to(torch.int32)
    case = Batch8(*args, seed=3, spare_rows=2)
    r = run_rope8(m, case, pos, rot, qk_norm=qk_norm, interleaved=interleaved)
    check_rope8(case, r)
    # the queries are moe_rope_append's, bit for bit
    q = run_rope(m, Batch(*args, seed=3, spare_rows=2), pos, rot, qk_norm=qk_norm, interleaved=interleaved)["q_out"]
    assert same(r["q_out"], q)


def test_append_axes(m):
    case = Batch8([9, 4], [9, 30], 8, 2, 128, 16, BF16, seed=4)
    pos = torch.randint(0, 1 << 20, (3, case.N), generator=torch.Generator().manual_seed(2)).to(torch.int32)
    pos[0, 0], pos[1, 0], pos[2, 1] = 2 ** 31 - 1, -(2 ** 31), -5
    check_rope8(case, run_rope8(m, case, pos, 128, axis=(torch.arange(64) % 3).to(torch.int32), qk_norm=True))


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 32)])
def test_append_special_values(m, D, rot, dtype):
    """Zeros, a single value, the type's largest and smallest, infinities and NaN: by the quantiser's
    rules in V, and in K at position 0, where the rotation changes nothing; one head's do not reach another's."""
    Hq, Hkv = 4, 2
    f = torch.finfo(dtype)
    rows = torch.randn(9, Hq + 2 * Hkv, D, generator=torch.Generator().manual_seed(7)).to(dtype)
    special = torch.zeros(9, D, dtype=dtype)
    special[1, 5] = -1.5
    special[2] = f.max
    special[3] = -f.max
    special[4, ::2] = f.tiny
    special[5] = f.tiny * f.eps  # the smallest subnormal
    special[6] = rows[6, 0]
    special[6, D - 1] = math.inf
    special[7] = rows[7, 0]
    special[7, 0] = -math.inf
    special[8] = rows[8, 0]
    special[8, D // 2] = math.nan
    rows[:, Hq] = special
    rows[:, Hq + Hkv] = special
    case = Batch8([9], [20], Hq, Hkv, D, 16, dtype, seed=1)
    # a vanishing angle: x - 0 * y and y + 0 * x keep every finite value, and an infinity's partner becomes NaN
    r = run_rope8(m, case, torch.zeros(1, 9, dtype=torch.int32), rot, qkv=rows.reshape(9, -1))
    assert r["code"] == 0
    codes, scales = quantised(rows[:, Hq:].double())
    for i in range(9):
        pg, at = int(case.table[0, (11 + i) // 16]), (11 + i) % 16
        assert torch.equal(r["v"][pg, :, at], codes[i, Hkv:]) and same(r["vs"][pg, :, at], scales[i, Hkv:]), i
        assert torch.equal(r["k"][pg, 1, at], codes[i, 1]) and torch.equal(r["ks"][pg, 1, at], scales[i, 1]), i
        if i < 6:
            assert torch.equal(r["k"][pg, 0, at], codes[i, 0]) and torch.equal(r["ks"][pg, 0, at], scales[i, 0]), i
        else:
            assert not bool(r["k"][pg, 0, at].any()) and not math.isfinite(float(r["ks"][pg, 0, at])), i


def test_append_bad_descriptions(m):
    """Out-of-range pages, lengths and offsets are recorded; nothing is written through them, and the
    other sequence's rows are."""
    def spoiled(change):
        case = Batch8([2, 3], [20, 33], 4, 2, 64, 16, F16)
        change(case)
        return case, run_rope8(m, case, torch.zeros(1, case.N, dtype=torch.int32), 64)
    for bad in (-1, 1 << 30):
        for b, j in ((1, 1), (1, 2)):  # the second sequence's rows lie in its pages 1 and 2
            case, r = spoiled(lambda c: c.table.__setitem__((b, j), bad))
            assert m.status_str(r["code"]) == "MOE_ERR_CACHE_RANGE" and r["detail"] == bad
            pg = int(case.table[0, 1])
            assert not same(r["ks"][pg, :, 2], case.ks[pg, :, 2])  # row 18 of the first
    for L in (-1, 16 * 3 + 1, 2 ** 31 - 1):
        case, r = spoiled(lambda c: c.lens.__setitem__(1, L))
        assert m.status_str(r["code"]) == "MOE_ERR_CACHE_RANGE" and r["detail"] == L
    for o in ([0, 6, 5], [0, -1, 5], [0, 2, 99], [7, 8, 9]):
        case, r = spoiled(lambda c: c.offs.copy_(torch.tensor(o)))
        assert m.status_str(r["code"]) == "MOE_ERR_CACHE_RANGE", o


# --------------------------------------------------------------------------
# moe_attention_cache
# --------------------------------------------------------------------------
def run_attn(m, case, window=0, softcap=0.0, sinks=0, tree=None, scale=None, most=None, ws=None, d=None):
    scale = 1 / math.sqrt(case.D) if scale is None else scale
    d = case.dev(DEV) if d is None else d
    out = torch.full((case.N, case.Hq, case.D), float("nan"), dtype=case.dtype, device=DEV)
    lse = torch.full((case.N, case.Hq), float("nan"), device=DEV)
    ws = m.alloc_attention_workspace(case.Hq, case.Hkv, case.D, device=DEV) if ws is None else ws
    m.moe_attention_cache(d["q"], d["k"], d["v"], d["table"], d["offs"], d["lens"], most or case.most, scale, out, ws,
                          k_scales=d.get("ks"), v_scales=d.get("vs"), tree=None if tree is None else tree.to(DEV),
                          sinks=sinks, lse=lse, window=window, softcap=softcap)
    code, detail = m.moe_read_device_status(ws)
    return out, lse, code, detail


def check_attn(m, case, window=0, softcap=0.0, sinks=0, trees=None, words=None, fill=0, scale=None, most=None,
               ws=None):
    words = 0 if trees is None else words or max(1, -(-case.most // 32))
    tree = None if trees is None else tree_tensor(trees, case.N, words, fill)
    out, lse, code, detail = run_attn(m, case, window, softcap, sinks, tree, scale, most, ws)
    assert code == 0, (m.status_str(code), detail)
    o, e, tol, lse_tol = cache_ref(case, 1 / math.sqrt(case.D) if scale is None else scale, window, softcap, sinks,
                                   trees, words)
    used = sum(case.new)
    within(out[:used], o[:used], tol[:used], "out")
    within(lse[:used], e[:used], lse_tol[:used], "lse")
    assert bool(out[used:].isnan().all()) and bool(lse[used:].isnan().all())
    return out, lse


SHAPES = [
    # new, lens, Hq, Hkv, D, page
    ([1], [1], 4, 1, 128, 16),
    ([1], [93], 32, 4, 128, 16),
    ([1], [2049], 16, 2, 64, 64),
    ([1, 1, 1], [1, 17, 1000], 28, 4, 128, 32),
    ([1, 0, 1, 1], [5, 7, 129, 128], 8, 8, 64, 128),
    ([1] * 7, [3, 64, 65, 127, 255, 256, 257], 64, 4, 128, 256),
    ([6, 6, 5], [6, 300, 1111], 64, 4, 128, 16),
    ([2, 3, 1], [2, 50, 700], 12, 2, 64, 16),
    ([12], [40], 8, 8, 128, 32),
    ([33, 1, 0, 90], [40, 200, 3, 90], 16, 2, 128, 32),
    ([128], [128], 8, 1, 128, 128),
    ([129], [500], 8, 1, 64, 64),
    ([300, 260], [300, 1300], 4, 2, 128, 16),
    ([257], [777], 20, 4, 64, 32),
    ([5, 70], [2, 30], 8, 2, 128, 16),          # more new tokens than cached ones
    ([3], [0], 4, 2, 64, 16),                    # an empty cache
    ([11], [400], 128, 1, 128, 16),
    ([64], [64], 1, 1, 64, 16),
]
IDS = [f"B{len(a[0])}n{max(a[0])}L{max(a[1])}h{a[2]}k{a[3]}d{a[4]}p{a[5]}" for a in SHAPES]
MASKS = {"plain": {}, "cap": dict(softcap=15.0), "window1": dict(window=1), "sinks": dict(window=37, sinks=5),
         "sinkscap": dict(window=70, sinks=150, softcap=15.0), "far": dict(window=300, sinks=1)}


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("masks", MASKS)
@pytest.mark.parametrize("new,lens,Hq,Hkv,D,page", SHAPES, ids=IDS)
def test_codes(m, new, lens, Hq, Hkv, D, page, masks, dtype):
    case = Batch8(new, lens, Hq, Hkv, D, page, dtype, seed=len(new) + max(lens), spare_rows=3)
    check_attn(m, case, **MASKS[masks])


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("masks", ["sinks", "sinkscap", "far"])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D,page", SHAPES, ids=IDS)
def test_sinks(m, new, lens, Hq, Hkv, D, page, masks, dtype):
    case = Batch(new, lens, Hq, Hkv, D, page, dtype, seed=len(new) + max(lens), spare_rows=3)
    check_attn(m, case, **MASKS[masks])


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("codes", [False, True], ids=["16bit", "codes"])
@pytest.mark.parametrize("masks", ["plain", "cap", "sinks", "window1"])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D,page", SHAPES, ids=IDS)
def test_tree(m, new, lens, Hq, Hkv, D, page, masks, codes, dtype):
    kind = Batch8 if codes else Batch
    case = kind(new, lens, Hq, Hkv, D, page, dtype, seed=len(new) + max(lens), spare_rows=3)
    trees = random_trees(new, seed=max(lens), empty=0.2, own=masks != "cap")
    check_attn(m, case, trees=trees, fill=-1, **MASKS[masks])


@pytest.mark.parametrize("codes", [False, True], ids=["16bit", "codes"])
@pytest.mark.parametrize("words,n", [(1, 31), (1, 32), (1, 33), (2, 64), (2, 65), (2, 100), (7, 100), (32, 1000), (3, 1)])
def test_tree_words(m, words, n, codes):
    """Words that hold just the new tokens, fewer, more (whose bits are ignored)."""
    kind = Batch8 if codes else Batch
    case = kind([n, 3], [n + 45, 3], 4, 2, 64, 16, BF16, seed=n)
    trees = random_trees(case.new, seed=n, width=40)
    extra = [t | (~0 & ((1 << 1100) - 1)) << k for t, k in zip(trees, [n] * n + [3] * 3)]
    check_attn(m, case, trees=extra, words=words)
    check_attn(m, case, trees=extra, words=words, window=20, sinks=2)


@pytest.mark.parametrize("codes", [False, True], ids=["16bit", "codes"])
@pytest.mark.parametrize("n,L,Hq,Hkv", [(1, 700, 16, 2), (12, 500, 8, 8), (60, 900, 16, 2), (200, 1500, 4, 1)])
def test_tree_that_is_a_chain(m, n, L, Hq, Hkv, codes):
    """A tree of one path sees what a chain sees, windows and sinks among it."""
    kind = Batch8 if codes else Batch
    case = kind([n, n], [L, L + 3], Hq, Hkv, 128, 32, BF16, seed=n)
    chain = [(2 << i) - 1 for i in range(n)] * 2
    for kw in ({}, dict(window=n + 50, sinks=3)):
        # (a window shorter than the path would hide a chain's new tokens, not a tree's)
        a, la = check_attn(m, case, trees=chain, **kw)
        b, lb = check_attn(m, case, **kw)
        assert float((la - lb).abs().max()) < 1e-5


def test_rows_that_see_nothing(m):
    """No older tokens and no bits: 0 and -inf, whatever the cache holds; beside rows that see themselves."""
    for kind in (Batch, Batch8):
        for n in (1, 3, 40):
            case = kind([n], [n], 8, 2, 64, 16, F16, seed=n)
            trees = [0 if i % 2 == 0 else 1 << i for i in range(n)]
            out, lse = check_attn(m, case, trees=trees)
            assert not bool(out[::2].any()) and bool((lse[::2] == -math.inf).all())


def test_nothing_used_is_the_paged_call(m):
    """Without codes, tree and sinks the results are moe_attention_paged's, bit for bit."""
    for new, lens, window, cap in (([1, 1], [900, 90], 0, 0.0), ([60, 3], [300, 3], 50, 20.0)):
        case = Batch(new, lens, 16, 2, 128, 16, BF16, seed=5)
        d = case.dev(DEV)
        a, la, code, _ = run_attn(m, case, window, cap, sinks=0, d=d)
        b, lb = torch.empty_like(a), torch.empty_like(la)
        ws = m.alloc_attention_workspace(16, 2, 128, device=DEV)
        m.moe_attention_paged(d["q"], d["k"], d["v"], d["table"], d["offs"], d["lens"], case.most, 128 ** -0.5, b, ws,
                              lse=lb, window=window, softcap=cap)
        torch.cuda.synchronize()
        assert code == 0 and torch.equal(a, b) and torch.equal(la, lb)
        if not window:  # sinks without a window change nothing
            c, lc, _, _ = run_attn(m, case, window, cap, sinks=7, d=d)
            assert torch.equal(a, c) and torch.equal(la, lc)


@pytest.mark.parametrize("codes", [False, True], ids=["16bit", "codes"])
@pytest.mark.parametrize("new,L,window,sinks,page", [
    (1, 3000, 100, 4, 16), (1, 3000, 700, 128, 128), (1, 5000, 64, 200, 16), (6, 3000, 129, 17, 32),
    (90, 4000, 500, 1, 16), (150, 4000, 1000, 130, 128), (300, 2000, 64, 64, 64)])
def test_pages_out_of_sight(m, new, L, window, sinks, page, codes):
    """The pages between the sinks and the oldest window may be gone: their table entries are out of range
    and not read."""
    kind = Batch8 if codes else Batch
    for trees in (None, [1 << i for i in range(new)]):
        case = kind([new, 1], [L, 50], 16, 2, 128, page, BF16, seed=3)
        first = max(0, L - new - window + 1)
        gone = [p for p in range(case.used[0]) if p * page >= sinks and (p + 1) * page <= first]
        assert gone
        ids = case.table[0].clone()
        for p in gone:
            pg = int(ids[p])
            for t in (case.k, case.v):
                t[pg] = 77 if codes else math.nan
            for t in ((case.ks, case.vs) if codes else ()):
                t[pg] = math.nan
        # the reference reads the whole table: finite there, hidden by the mask
        want = kind([new, 1], [L, 50], 16, 2, 128, page, BF16, seed=3)
        words = max(1, -(-new // 32))
        full = None if trees is None else trees + [1]
        o, e, tol, lse_tol = cache_ref(want, 128 ** -0.5, window, 0.0, sinks, full, words)
        for p in gone:
            case.table[0, p] = -5 if p % 2 else 1 << 30
        tree = None if trees is None else tree_tensor(full, case.N, words)
        out, lse, code, detail = run_attn(m, case, window, 0.0, sinks, tree)
        assert code == 0, (m.status_str(code), detail)
        within(out, o, tol, "out")
        within(lse, e, lse_tol, "lse")


@pytest.mark.parametrize("new", [1, 5, 40])
def test_bad_descriptions(m, new):
    """Bad pages, lengths and offsets of one sequence are recorded, and the other's rows are right."""
    for kind in (Batch, Batch8):
        for spoil in ("page", "length", "offset"):
            case = kind([new, new], [100, 90], 8, 2, 64, 16, F16, seed=6)
            trees = random_trees(case.new, seed=1)
            o, e, tol, lse_tol = cache_ref(case, 0.125, 50, 0.0, 3, trees, 2)
            if spoil == "page":
                case.table[1, 5] = -3
            elif spoil == "length":
                case.lens[1] = 16 * 7 + 1
            else:
                case.offs[2] = case.N + 1
            out, lse, code, _ = run_attn(m, case, 50, 0.0, 3, tree_tensor(trees, case.N, 2), scale=0.125)
            assert m.status_str(code) == "MOE_ERR_CACHE_RANGE"
            within(out[:new], o[:new], tol[:new], "out")
            within(lse[:new], e[:new], lse_tol[:new], "lse")


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("new", [1, 50])
def test_codes_scales_of_many_sizes(m, new, dtype):
    """Values' scales far apart, zero, beyond a 16-bit type's range together with the codes; scales of keys of 0."""
    L = 700
    for span in ((-20, 8), (-100, -90), (0, 9) if dtype is F16 else (90, 100)):
        case = Batch8([new], [L], 8, 2, 128, 16, dtype, seed=11)
        g = torch.Generator().manual_seed(1)
        ids = case.table[0, :case.used[0]].long()
        size = 2.0 ** torch.randint(span[0], span[1], (len(ids), 2, 16), generator=g).float()
        size[torch.rand(size.shape, generator=g) < 0.1] = 0.0
        live = ~case.vs[ids].isnan()
        case.vs[ids] = torch.where(live, size, math.nan)
        zero = torch.rand(size.shape, generator=g) < 0.1
        case.ks[ids] = torch.where(live & zero, 0.0, case.ks[ids])
        case.k[ids] = torch.where((live & zero)[..., None], 0, case.k[ids])
        o, e, tol, lse_tol = cache_ref(case, 128 ** -0.5)
        out, lse, code, _ = run_attn(m, case)
        assert code == 0
        fits = o.abs() <= torch.finfo(dtype).max / 2
        if span[0] >= 0:
            assert bool(fits.float().mean() > 0.2)
        got = torch.where(fits, out.double().cpu(), o)
        within(got, o, tol, "out")
        within(lse, e, lse_tol, "lse")


def test_codes_rising_scores(m):
    """The running maximum and the largest scale so far move at every tile."""
    for new in (1, 40):
        for dtype in (F16, BF16):
            case = Batch8([new], [3000], 8, 2, 128, 32, dtype, seed=8)
            ids = case.table[0, :case.used[0]].long()
            j = (torch.arange(len(ids))[:, None, None] * 32 + torch.arange(32)).expand(-1, 2, -1)
            live = j < 3000
            case.k[ids] = torch.where((j % 2 == 0)[..., None], 127, 126).to(torch.int8).expand(-1, -1, -1, 128)
            case.ks[ids] = torch.where(live, j / 1000 * 0.02, math.nan).float()
            case.vs[ids] = torch.where(live, 2.0 ** (j / 300 - 8), math.nan).float()
            case.q.fill_(1.0)
            check_attn(m, case)
            check_attn(m, case, scale=-0.05)
            check_attn(m, case, scale=-0.05, softcap=25.0)
            check_attn(m, case, softcap=100.0)


@pytest.mark.parametrize("codes", [False, True], ids=["16bit", "codes"])
@pytest.mark.parametrize("most", [1, 4, 100000])
def test_max_new_is_a_hint(m, most, codes):
    kind = Batch8 if codes else Batch
    case = kind([1, 40, 3], [500, 90, 3], 16, 2, 128, 16, BF16)
    check_attn(m, case, most=most, window=60, sinks=9)
    check_attn(m, case, most=most, trees=random_trees(case.new))


@pytest.mark.parametrize("codes", [False, True], ids=["16bit", "codes"])
@pytest.mark.parametrize("B,new,tile", [(1, 1, 128), (19, 1, 128), (40, 1, 64), (1, 70, 128), (9, 40, 128), (30, 90, 128)])
def test_whole_and_parted(m, B, new, tile, codes):
    """Lengths around those from which items are parted; one long sequence among short ones."""
    kind = Batch8 if codes else Batch
    for tiles in (2, 3, 9, 10, 17):
        lens = [tiles * tile + d for d in (-1, 0, 1)] * B
        case = kind([new] * B, lens[:B], 8, 2, 64, 16, BF16, seed=tiles)
        check_attn(m, case, trees=random_trees(case.new, seed=tiles))
    case = kind([new] * B, [new + 5] * (B - 1) + [40 * tile], 8, 2, 64, 16, BF16)
    check_attn(m, case, trees=random_trees(case.new))
    check_attn(m, case, window=2 * tile, sinks=tile + 3)


def test_repeats_bit_for_bit(m):
    """The same call gives the same bits, on a used workspace too."""
    for kind, new, lens in ((Batch8, [1] * 9, [900 + 100 * i for i in range(9)]), (Batch8, [70, 40], [2000, 900]),
                            (Batch, [70, 40], [2000, 900]), (Batch, [1, 2], [5000, 90])):
        case = kind(new, lens, 16, 2, 128, 16, F16, seed=2)
        tree = tree_tensor(random_trees(new), case.N, 3)
        ws = m.alloc_attention_workspace(16, 2, 128, device=DEV)
        d = case.dev(DEV)
        first = run_attn(m, case, 300, 0.0, 20, tree, ws=ws, d=d)
        other = Batch8([30, 1], [700, 4000], 16, 2, 128, 16, F16, seed=1)
        for _ in range(3):
            run_attn(m, other, ws=ws)
            again = run_attn(m, case, 300, 0.0, 20, tree, ws=ws, d=d)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_cache_past_32_bits(m):
    """Codes, scales and pages whose offsets pass 32 bits."""
    page, Hkv, D = 256, 8, 128
    P = (1 << 32) // (page * Hkv * D) + 40  # over 2^32 codes
    for op in ("codes", "append", "keep"):
        case = Batch8([5], [300], 16, Hkv, D, page, BF16, seed=4)
        far = [P - 7, P - 2]
        k, v = (torch.empty(P, Hkv, page, D, dtype=torch.int8, device=DEV) for _ in range(2))
        ks, vs = (torch.full((P, Hkv, page), math.nan, device=DEV) for _ in range(2))
        for i, pg in enumerate(far):
            old = int(case.table[0, i])
            for big, small in ((k, case.k), (v, case.v), (ks, case.ks), (vs, case.vs)):
                big[pg] = small[old].to(DEV)
        table = torch.tensor([far], dtype=torch.int32)
        d = case.dev(DEV) | dict(k=k, v=v, ks=ks, vs=vs, table=table.to(DEV))
        if op == "codes":
            trees = random_trees([5])
            o, e, tol, lse_tol = cache_ref(case, D ** -0.5, trees=trees, words=1)
            for most in (5, 100):
                out, lse, code, _ = run_attn(m, case, tree=tree_tensor(trees, 5, 1), d=d, most=most)
                assert code == 0
                within(out, o, tol, "out")
                within(lse, e, lse_tol, "lse")
            continue
        ws = m.alloc_attention_workspace(16, Hkv, D, device=DEV)
        before = [int(case.table[0, i]) for i in range(2)]
        if op == "append":
            pos = torch.arange(295, 300, dtype=torch.int32)[None]
            r = run_rope8(m, case, pos, 128)
            q = torch.empty(5, 16, D, dtype=BF16, device=DEV)
            m.moe_rope_append_q8(r["qkv"].to(DEV), pos.to(DEV), inv_freq(128).to(DEV), q, k, v, ks, vs, d["table"],
                                 d["offs"], d["lens"], ws, eps=EPS)
            want = {n: r[n] for n in ("k", "v", "ks", "vs")}
        else:
            keep = torch.tensor([[0, 2, 4]], dtype=torch.int32, device=DEV)
            kept = torch.tensor([3], dtype=torch.int32, device=DEV)
            m.moe_cache_keep(k, v, d["table"], d["offs"], d["lens"], keep, kept, ws, k_scales=ks, v_scales=vs)
            want = {n: getattr(case, n).clone() for n in ("k", "v", "ks", "vs")}
            for t in want.values():
                for dst, src in ((296, 297), (297, 299)):
                    t[before[dst // page], :, dst % page] = t[before[src // page], :, src % page].clone()
        assert m.moe_read_device_status(ws)[0] == 0
        for n, big in (("k", k), ("v", v), ("ks", ks), ("vs", vs)):
            for i in range(2):
                assert same(big[far[i]].cpu().float(), want[n][before[i]].float()), (op, n)


# --------------------------------------------------------------------------
# moe_cache_keep
# --------------------------------------------------------------------------
def random_path(n, k, g):
    return sorted(torch.randperm(n, generator=g)[:k].tolist())


def run_keep(m, case, paths, most, kept=None):
    d = case.dev(DEV)
    keep = torch.full((case.B, most), -9, dtype=torch.int32)
    for b, p in enumerate(paths):
        keep[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    kept = torch.tensor([len(p) for p in paths] if kept is None else kept, dtype=torch.int32)
    ws = m.alloc_attention_workspace(case.Hq, case.Hkv, case.D, device=DEV)
    scales = dict(k_scales=d["ks"], v_scales=d["vs"]) if isinstance(case, Batch8) else {}
    m.moe_cache_keep(d["k"], d["v"], d["table"], d["offs"], d["lens"], keep.to(DEV), kept.to(DEV), ws, **scales)
    code, detail = m.moe_read_device_status(ws)
    return {n: d[n].cpu() for n in ("k", "v", "ks", "vs") if n in d}, code, detail


def kept_ref(case, paths):
    r = {n: getattr(case, n).clone() for n in ("k", "v", "ks", "vs") if hasattr(case, n)}
    for b, path in enumerate(paths):
        base = case.lens_list[b] - case.new[b]
        at = lambda j: (int(case.table[b, j // case.page]), j % case.page)  # noqa: E731
        for t in r.values():
            rows = [t[at(base + i)[0], :, at(base + i)[1]].clone() for i in path]
            for d, row in enumerate(rows):
                t[at(base + d)[0], :, at(base + d)[1]] = row
    return r


@pytest.mark.parametrize("codes", [False, True], ids=["16bit", "codes"])
@pytest.mark.parametrize("new,lens,Hkv,D,page,most", [
    ([1], [1], 1, 64, 16, 1), ([7], [40], 4, 128, 16, 7), ([64, 0, 33], [64, 9, 500], 2, 128, 32, 20),
    ([250] * 5, [250, 300, 999, 257, 400], 8, 64, 64, 250), ([1000], [1100], 2, 128, 256, 700)])
def test_keep(m, new, lens, Hkv, D, page, most, codes):
    kind = Batch8 if codes else Batch
    g = torch.Generator().manual_seed(most)
    for share in (0.1, 0.5, 1.0):
        case = kind(new, lens, Hkv, Hkv, D, page, BF16, seed=1)
        paths = [random_path(n, min(most, int(math.ceil(share * n))), g) for n in new]
        got, code, detail = run_keep(m, case, paths, most)
        assert code == 0, (m.status_str(code), detail)
        for n, want in kept_ref(case, paths).items():
            assert same(got[n].float(), want.float()), n


@pytest.mark.parametrize("codes", [False, True], ids=["16bit", "codes"])
def test_keep_refused_sequences_stay(m, codes):
    """An index twice, falling, out of range, too many of them, a bad page: recorded, that sequence as it was,
    the others moved."""
    kind = Batch8 if codes else Batch
    good = [3, 7, 20]
    for bad, kept, page in (([2, 2], None, None), ([5, 4], None, None), ([-1, 3], None, None), ([0, 25], None, None),
                            ([0, 1], [3, 9, 3], None), ([0, 1], [3, -1, 3], None), ([0, 24], None, (1, 4))):
        case = kind([25, 25, 25], [60, 70, 80], 2, 2, 64, 16, F16, seed=2)
        before = case.table.clone()
        if page is not None:
            case.table[page] = -7  # of rows 64 ..: token 24 of the second sequence lies there
        got, code, _ = run_keep(m, case, [good, bad, good], 5, kept)
        assert m.status_str(code) == "MOE_ERR_CACHE_RANGE", (bad, kept)
        case.table.copy_(before)
        for n, want in kept_ref(case, [good, [], good]).items():
            assert same(got[n].float(), want.float()), (n, bad)


# --------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 4)])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
def test_drafting_over_the_cache(m, dtype, window, sinks):
    """A prompt, then drafted trees whose accepted paths are kept: after each step the codes are those of
    the accepted tokens appended as a chain, bit for bit, and the next step's attention is right over them."""
    Hq, Hkv, D, page, B = 8, 2, 64, 16, 2
    g = torch.Generator().manual_seed(3)
    ws = m.alloc_attention_workspace(Hq, Hkv, D, device=DEV)
    width = (Hq + 2 * Hkv) * D
    freq = inv_freq(D).to(DEV)
    most = 12

    def caches():
        c = [torch.zeros(B * most, Hkv, page, D, dtype=torch.int8, device=DEV) for _ in range(2)]
        return c + [torch.full((B * most, Hkv, page), math.nan, device=DEV) for _ in range(2)]

    table = torch.randperm(B * most, generator=g).view(B, most).to(torch.int32)
    drafted, chained = caches(), caches()

    def append(cache, rows, pos, new, lens):
        offs = torch.tensor([0] + new).cumsum(0).to(torch.int32).to(DEV)
        q = torch.empty(sum(new), Hq, D, dtype=dtype, device=DEV)
        ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
        m.moe_rope_append_q8(rows.to(DEV), pos.to(DEV), freq, q, *cache, table.to(DEV), offs, ln, ws, eps=EPS)
        return q, offs, ln

    def attend(cache, q, offs, ln, new, trees):
        case = Batch8.__new__(Batch8)
        case.new, case.lens_list = new, ln.tolist()
        case.Hq, case.Hkv, case.D, case.page, case.dtype, case.B, case.N = Hq, Hkv, D, page, dtype, B, sum(new)
        case.used = [-(-x // page) for x in case.lens_list]
        case.table, case.q, case.lens, case.offs = table, q.cpu(), ln.cpu(), offs.cpu()
        case.k, case.v, case.ks, case.vs = (t.cpu() for t in cache)
        check_attn(m, case, window, 0.0, sinks, trees, ws=ws)

    lens = [30, 17]
    rows = torch.randn(sum(lens), width, generator=g).to(dtype)
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)[None]
    for c in (drafted, chained):
        q, offs, ln = append(c, rows, pos, lens, lens)
    attend(drafted, q, offs, ln, lens, None)
    for step in range(4):
        new = [[20, 9], [1, 33], [5, 5], [40, 1]][step]
        trees = random_trees(new, seed=step)
        rows = torch.randn(sum(new), width, generator=g).to(dtype)
        depth = [bin(t).count("1") - 1 for t in trees]
        place = torch.tensor([lens[b] + depth[sum(new[:b]) + i] for b in range(B) for i in range(new[b])])
        q, offs, ln = append(drafted, rows, place.to(torch.int32)[None], new, [a + n for a, n in zip(lens, new)])
        attend(drafted, q, offs, ln, new, trees)
        paths = []
        for b in range(B):
            leaf = trees[sum(new[:b]) + int(torch.randint(0, new[b], (1,), generator=g))]
            paths.append([i for i in range(new[b]) if leaf >> i & 1])
        keep = torch.zeros(B, 40, dtype=torch.int32)
        for b, p in enumerate(paths):
            keep[b, :len(p)] = torch.tensor(p)
        kept = torch.tensor([len(p) for p in paths], dtype=torch.int32)
        m.moe_cache_keep(drafted[0], drafted[1], table.to(DEV), offs, ln, keep.to(DEV), kept.to(DEV), ws,
                         k_scales=drafted[2], v_scales=drafted[3])
        take = torch.tensor([sum(new[:b]) + i for b in range(B) for i in paths[b]])
        steps = [len(p) for p in paths]
        chain = torch.cat([torch.arange(lens[b], lens[b] + steps[b]) for b in range(B)])
        lens = [a + k for a, k in zip(lens, steps)]
        append(chained, rows[take], chain.to(torch.int32)[None], steps, lens)
        for a, c in zip(drafted, chained):
            for b in range(B):
                ids = table[b].long()
                x, y = (t[ids.to(DEV)].transpose(0, 1).flatten(1, 2)[:, :lens[b]] for t in (a, c))
                assert torch.equal(x, y)
    assert m.moe_read_device_status(ws)[0] == 0


@pytest.mark.parametrize("new", [1, 6, 40])
def test_captured_and_replayed(m, new):
    """A captured step (append, attention over a tree, keep) over lengths, tables and paths that change on the
    device; two graphs take turns on one workspace."""
    Hq, Hkv, D, page, B = 16, 2, 128, 16, 3
    graphs = []
    ws = m.alloc_attention_workspace(Hq, Hkv, D, device=DEV)
    for kind in range(2):
        case = Batch8([new] * B, [200, 90, 150], Hq, Hkv, D, page, BF16, seed=kind)
        d = case.dev(DEV)
        words = -(-new // 32)
        d["tree"] = torch.zeros(case.N, words, dtype=torch.int32, device=DEV)
        d["keep"] = torch.zeros(B, new, dtype=torch.int32, device=DEV)
        d["kept"] = torch.ones(B, dtype=torch.int32, device=DEV)
        d["qkv"] = torch.zeros(case.N, (Hq + 2 * Hkv) * D, dtype=BF16, device=DEV)
        d["pos"] = torch.zeros(1, case.N, dtype=torch.int32, device=DEV)
        d["q2"], d["out"] = (torch.zeros(case.N, Hq, D, dtype=BF16, device=DEV) for _ in range(2))
        d["lse"] = torch.zeros(case.N, Hq, device=DEV)
        d["freq"] = inv_freq(D).to(DEV)  # the graph's as long as it lives

        def step(d=d):
            m.moe_rope_append_q8(d["qkv"], d["pos"], d["freq"], d["q2"], d["k"], d["v"], d["ks"], d["vs"], d["table"],
                                 d["offs"], d["lens"], ws, eps=EPS)
            m.moe_attention_cache(d["q2"], d["k"], d["v"], d["table"], d["offs"], d["lens"], new, D ** -0.5, d["out"],
                                  ws, k_scales=d["ks"], v_scales=d["vs"], tree=d["tree"], lse=d["lse"], window=100,
                                  sinks=5)
            m.moe_cache_keep(d["k"], d["v"], d["table"], d["offs"], d["lens"], d["keep"], d["kept"], ws,
                             k_scales=d["ks"], v_scales=d["vs"])

        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graphs.append((graph, case, d, words))
    g = torch.Generator().manual_seed(9)
    for turn in range(3):
        for graph, case, d, words in graphs:
            fresh = Batch8([new] * B, [200 - 3 * turn, 90 + turn, 150], Hq, Hkv, D, page, BF16, seed=10 + turn)
            trees = random_trees(fresh.new, seed=turn)
            paths = [random_path(new, (new + 1) // 2, g) for _ in range(B)]
            keep = torch.zeros(B, new, dtype=torch.int32)
            keep[:, :(new + 1) // 2] = torch.tensor(paths)
            pos = torch.randint(0, 500, (1, fresh.N), generator=g).to(torch.int32)
            qkv = torch.randn(fresh.N, (Hq + 2 * Hkv) * D, generator=g).to(BF16)
            r = run_rope8(m, fresh, pos, D, qkv=qkv)  # codes after the append, by a call of its own
            for n, t in (("table", fresh.table), ("lens", fresh.lens), ("tree", tree_tensor(trees, fresh.N, words)),
                         ("keep", keep), ("kept", torch.full((B,), (new + 1) // 2)), ("pos", pos), ("qkv", qkv)):
                d[n].copy_(t)
            for n in ("k", "v", "ks", "vs"):
                d[n].copy_(getattr(fresh, n))
            graph.replay()
            torch.cuda.synchronize()
            assert m.moe_read_device_status(ws)[0] == 0
            for n in ("k", "v", "ks", "vs"):
                setattr(fresh, n, r[n])
            fresh.q = d["q2"].cpu()
            o, e, tol, lse_tol = cache_ref(fresh, D ** -0.5, 100, 0.0, 5, trees, words)
            within(d["out"], o, tol, "out")
            within(d["lse"], e, lse_tol, "lse")
            for n, want in kept_ref(fresh, paths).items():
                assert same(d[n].cpu().float(), want.float()), n


def test_other_stream(m):
    """Calls on a side stream, ordered by events, while the current stream is another."""
    case = Batch8([1, 3], [500, 90], 8, 2, 128, 16, F16, seed=1)
    d = case.dev(DEV)
    o, e, tol, lse_tol = cache_ref(case, 128 ** -0.5, 64, 0.0, 4)
    ws = m.alloc_attention_workspace(8, 2, 128, device=DEV)
    out, lse = torch.empty(4, 8, 128, dtype=F16, device=DEV), torch.empty(4, 8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.moe_attention_cache(d["q"], d["k"], d["v"], d["table"], d["offs"], d["lens"], 3, 128 ** -0.5, out, ws,
                          k_scales=d["ks"], v_scales=d["vs"], window=64, sinks=4, lse=lse, stream=side)
    side.synchronize()
    within(out, o, tol, "out")
    within(lse, e, lse_tol, "lse")
