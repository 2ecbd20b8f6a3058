"""Scales of 8-bit codes: of either zero, far apart where a row does not see them or gives them no
weight, tiny, and not finite."""
import math

import pytest

from tests.cache_cases import Batch8, cache_ref, random_trees, tree_tensor, visible
from tests.test_gpu_attention_half import within
from tests.test_gpu_cache import check_attn, run_attn
from tests.test_gpu_parity import DEV, m  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF16, F16 = torch.bfloat16, torch.float16
TYPES = pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])


def at(case, b, j):
    """The page and row of cached token j of sequence b."""
    return int(case.table[b, j // case.page]), j % case.page


@TYPES
@pytest.mark.parametrize("new", [1, 50])
def test_scales_of_minus_zero(m, new, dtype):
    """-0.0 is a scale of 0, for keys and for values, in a sequence's first tile and later."""
    for L in (new + 4, 300):
        case = Batch8([new], [L], 8, 2, 128, 16, dtype, seed=3)
        for j in (0, 2, L - 1, 150):
            if j < L:
                pg, row = at(case, 0, j)
                case.ks[pg, 0, row] = case.vs[pg, :, row] = -0.0
        check_attn(m, case)


def row_ref(case, window=0, softcap=0.0, sinks=0, trees=None, words=0):
    """cache_ref with what a row sees as the only thing that bounds its error: over codes a weight times its
    value's scale is off by half a step of the type it is rounded to and, where that is fp16, by at most 2^-24
    of the largest such product of the row."""
    o, e, _, lse_tol = cache_ref(case, case.D ** -0.5, window, softcap, sinks, trees, words)
    tol = torch.full_like(o, math.nan)
    G, u = case.Hq // case.Hkv, torch.finfo(case.dtype).eps / 2
    fp16 = case.dtype is F16 or case.most * G <= 16
    row0 = 0
    for b, (n, L) in enumerate(zip(case.new, case.lens_list)):
        rows = slice(row0, row0 + n)
        q = case.q[rows].double().view(n, case.Hkv, G, case.D).permute(1, 2, 0, 3)
        ids = case.table[b, :case.used[b]].long()
        take = lambda p: p[ids].transpose(0, 1).flatten(1, 2)[:, :L].double()  # noqa: E731
        k, vc, vs = case.cached(b, case.k), take(case.v), take(case.vs)
        z = torch.einsum("hgnd,hkd->hgnk", q, k) * case.D ** -0.5
        # the products' sum, the scale's and the key scale's product, in fp32
        dz = torch.einsum("hgnd,hkd->hgnk", q.abs(), k.abs()) * case.D ** -0.5 * (case.D + 10) * 2.0 ** -24
        if softcap > 0:
            z, dz = softcap * torch.tanh(z / softcap), dz + softcap * 2.0 ** -20
        seen = visible(n, L, window, sinks, None if trees is None else trees[rows], words)
        p = torch.where(seen, z, -math.inf).softmax(-1)
        # (of keys whose weight matters: the others' relative errors change nothing)
        rel = 2 * torch.where(seen & (p > 2.0 ** -40), dz, 0.0).amax(-1) + 2.0 ** -20 + (L + 66) * 2.0 ** -24
        absv = torch.einsum("hgnk,hkd->hgnd", p, (vc * vs[..., None]).abs())
        most = (p * vs[:, None, None]).amax(-1)
        codes = torch.einsum("nk,hkd->hnd", seen.double(), vc.abs())
        err = (rel[..., None] + u) * absv + (2.0 ** -24 * most[..., None] * codes[:, None] if fp16 else 0.0)
        want = o[rows].view(n, case.Hkv, G, case.D).permute(1, 2, 0, 3)
        err = err + u * (want.abs() + err) + torch.finfo(case.dtype).smallest_normal * u
        tol[rows] = err.permute(2, 0, 1, 3).reshape(n, case.Hq, case.D)
        row0 += n
    return o, e, tol, lse_tol


def run_row_ref(m, case, window=0, softcap=0.0, sinks=0, trees=None):
    words = 0 if trees is None else -(-case.most // 32)
    out, lse, code, detail = run_attn(m, case, window, softcap, sinks,
                                      None if trees is None else tree_tensor(trees, case.N, words))
    assert code == 0, (m.status_str(code), detail)
    o, e, tol, lse_tol = row_ref(case, window, softcap, sinks, trees, words)
    fits = o.abs() <= torch.finfo(case.dtype).max / 2
    within(torch.where(fits, out.double().cpu(), o), o, tol, "out")
    within(lse, e, lse_tol, "lse")


def louder(case, b, tokens, by):
    """The values' scales of some cached tokens, 2^by times what they are."""
    for j in tokens:
        pg, row = at(case, b, j)
        case.vs[pg, :, row] *= 2.0 ** by


LOUD = pytest.mark.parametrize("by", [8, 14, 20, 40])


@LOUD
@TYPES
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [2, 6, 60, 150])
def test_large_scales_of_other_branches(m, new, D, dtype, by):
    """Every other drafted token has values 2^by times the others': the rows that do not see it are as
    exact as without it, and so are those that do (their largest products are their own)."""
    case = Batch8([new, 1], [new + 200, 70], 8, 4, D, 16, dtype, seed=new)
    evens = sum(1 << i for i in range(0, new, 2))
    trees = [evens & ((2 << i) - 1) | 1 << i for i in range(new)] + [1]
    louder(case, 0, range(201, new + 200, 2), by)
    run_row_ref(m, case, trees=trees)
    run_row_ref(m, case, trees=trees, softcap=20.0)
    run_row_ref(m, case, trees=trees, softcap=100.0)


@LOUD
@TYPES
@pytest.mark.parametrize("new", [4, 40, 300])
def test_large_scales_of_later_tokens(m, new, dtype, by):
    """A chunk whose last tokens' values are large: the tokens before them."""
    case = Batch8([new], [new + 30], 8, 4, 128, 32, dtype, seed=1)
    louder(case, 0, range(30 + new - new // 3 - 1, new + 30), by)
    run_row_ref(m, case)


@LOUD
@TYPES
@pytest.mark.parametrize("new", [1, 3, 40, 200])
def test_large_scales_between_the_sinks_and_the_window(m, new, dtype, by):
    """Tokens that a window hides, in the tiles that it cuts too."""
    window, sinks, L = 150, 5, new + 700
    case = Batch8([new], [L], 8, 4, 64, 16, dtype, seed=2)
    louder(case, 0, range(sinks, L - new - window + 1), by)
    run_row_ref(m, case, window=window, sinks=sinks)


@LOUD
@TYPES
@pytest.mark.parametrize("softcap", [0.0, 50.0, 100.0])
@pytest.mark.parametrize("new", [1, 7, 60])
def test_large_scales_without_weight(m, new, softcap, dtype, by):
    """Tokens that every row sees, with large values and scores so low that they have no weight; or whose weight is
    lost to those of later tiles."""
    L = new + 600
    for which in ("low", "overtaken"):
        case = Batch8([new], [L], 8, 4, 128, 16, dtype, seed=4)
        case.q.copy_(0.5 + 0.5 * torch.rand(case.q.shape, generator=torch.Generator().manual_seed(1)))
        loud = range(0, 512, 3) if which == "low" else range(300)
        for j in range(L):
            pg, row = at(case, 0, j)
            away = j in loud
            case.k[pg, :, row] = (-100 if away else 0) + case.k[pg, :, row] // 8  # some 45 below the others
            case.ks[pg, :, row] = 0.05
        louder(case, 0, loud, by)
        run_row_ref(m, case, softcap=softcap)


@TYPES
@pytest.mark.parametrize("new", [1, 60])
def test_large_scales_that_come_and_go(m, new, dtype):
    """A scale for every token, 2^-90 to 2^20, in any order; of each head's, a tenth are 0."""
    g = torch.Generator().manual_seed(5)
    for lo, hi in ((-30, 20), (-90, -60), (-6, 0), (0, 7)):
        case = Batch8([new], [new + 700], 8, 4, 128, 16, dtype, seed=6)
        size = 2.0 ** (lo + (hi - lo) * torch.rand(case.vs.shape, generator=g)) * (torch.rand(case.vs.shape, generator=g) > 0.1)
        if dtype is F16:  # results stay in its range
            size = size.clamp(max=2.0 ** 7)
        case.vs = torch.where(case.vs.isnan(), math.nan, size)
        run_row_ref(m, case)
        run_row_ref(m, case, window=100, sinks=3, trees=random_trees([new]))


SPOILED = pytest.mark.parametrize("which", ["k", "v", "both"])


def spoil(case, b, tokens, value, which):
    """Heads as the append stores them where they hold an infinity or a NaN: that as the scale, codes 0."""
    for j in tokens:
        pg, row = at(case, b, j)
        for n in "kv" if which == "both" else which:
            getattr(case, n)[pg, :, row] = 0
            getattr(case, n + "s")[pg, :, row] = value


def check_spoiled(m, case, b, tokens, value, which, window=0, softcap=0.0, sinks=0, trees=None, scale=None):
    """The rows that see one of the tokens are NaN (and say so in lse), all others as if it were finite."""
    words = 0 if trees is None else -(-case.most // 32)
    scale = case.D ** -0.5 if scale is None else scale
    o, e, tol, lse_tol = cache_ref(case, scale, window, softcap, sinks, trees, words)
    spoil(case, b, tokens, value, which)
    out, lse, code, detail = run_attn(m, case, window, softcap, sinks,
                                      None if trees is None else tree_tensor(trees, case.N, words), scale=scale)
    assert code == 0, (m.status_str(code), detail)
    first, n = sum(case.new[:b]), case.new[b]
    seen = visible(n, case.lens_list[b], window, sinks, None if trees is None else trees[first:first + n], words)
    hit = torch.zeros(case.N, dtype=torch.bool)
    hit[first:first + n] = seen[:, list(tokens)].any(1)
    assert bool(out[hit].isnan().all()) and bool(lse[hit].isnan().all())
    within(out[~hit], o[~hit], tol[~hit], "out")
    within(lse[~hit], e[~hit], lse_tol[~hit], "lse")
    return int(hit.sum())


MODES = pytest.mark.parametrize("softcap,scale", [(0.0, None), (20.0, None), (100.0, None), (0.0, -0.1), (30.0, -0.1)],
                                ids=["plain", "cap", "farcap", "negative", "negativecap"])


@SPOILED
@TYPES
@MODES
@pytest.mark.parametrize("new", [2, 6, 60, 150])
def test_scales_that_are_not_finite_in_other_branches(m, new, softcap, scale, dtype, which):
    """A drafted token whose head holds an infinity or a NaN: its own row and its descendants' are NaN, no others."""
    for value in (math.inf, math.nan):
        case = Batch8([new, 1], [new + 200, 70], 8, 4, 64, 16, dtype, seed=new)
        evens = sum(1 << i for i in range(0, new, 2))
        trees = [evens & ((2 << i) - 1) | 1 << i for i in range(new)] + [1]
        assert check_spoiled(m, case, 0, [200 + new // 4 * 2 + 1], value, which, softcap=softcap, scale=scale, trees=trees) == 1


@SPOILED
@TYPES
@pytest.mark.parametrize("new", [1, 4, 40, 300])
def test_scales_that_are_not_finite_out_of_sight(m, new, dtype, which):
    """Between the sinks and the window, at both ends of that, and in a chunk's last tokens."""
    window, sinks, L = 150, 5, new + 700
    for value in (math.inf, math.nan):
        hidden = [sinks, sinks + 1, 100, L - new - window - 5, L - new - window]
        case = Batch8([new], [L], 8, 4, 128, 16, dtype, seed=2)
        assert check_spoiled(m, case, 0, hidden, value, which, window=window, sinks=sinks) == 0
        case = Batch8([new], [new + 30], 8, 4, 128, 32, dtype, seed=1)
        assert check_spoiled(m, case, 0, [new + 29], value, which) == 1
        case = Batch8([new], [L], 8, 4, 128, 32, dtype, seed=1)
        assert check_spoiled(m, case, 0, [sinks - 1, 333], value, which, window=window, sinks=sinks) == new
        assert check_spoiled(m, Batch8([new], [L], 8, 4, 128, 32, dtype, seed=1), 0, [333], value, which) == new


@TYPES
@pytest.mark.parametrize("new", [1, 40])
def test_a_spoiled_row_from_append_to_attention(m, new, dtype):
    """A projected row that holds a NaN: the append stores it, and the rows that do not see it are as without."""
    from tests.test_gpu_cache import run_rope8
    case = Batch8([new + 2], [new + 202], 8, 2, 128, 16, dtype, seed=5)
    rows = torch.randn(case.N, 12 * 128, generator=torch.Generator().manual_seed(1)).to(dtype)
    rows[new + 1, 8 * 128:] = math.nan
    r = run_rope8(m, case, torch.arange(200, new + 202, dtype=torch.int32)[None], 128, qkv=rows)
    for n in ("k", "v", "ks", "vs"):
        setattr(case, n, r[n])
    case.q = r["q_out"]
    trees = [(1 << i) - 1 | 1 << i for i in range(new + 1)] + [2 << new]
    words = -(-case.most // 32)
    clean = Batch8([new + 2], [new + 202], 8, 2, 128, 16, dtype, seed=5)
    for n in ("k", "v", "ks", "vs", "q"):
        setattr(clean, n, getattr(case, n).clone())
    pg, row = at(clean, 0, new + 201)
    clean.ks[pg, :, row] = clean.vs[pg, :, row] = 0.0
    o, e, tol, lse_tol = cache_ref(clean, 128 ** -0.5, trees=trees, words=words)
    out, lse, code, _ = run_attn(m, case, tree=tree_tensor(trees, case.N, words))
    assert code == 0 and bool(out[new + 1].isnan().all()) and bool(lse[new + 1].isnan().all())
    within(out[:new + 1], o[:new + 1], tol[:new + 1], "out")
    within(lse[:new + 1], e[:new + 1], lse_tol[:new + 1], "lse")


@pytest.mark.parametrize("softcap", [0.0, 20.0, 100.0])
@pytest.mark.parametrize("new", [1, 60])
def test_tiny_key_scales_under_large_queries(m, new, softcap):
    """Keys' scales at and below the smallest normal fp32, whose products with large queries are scores of some size."""
    case = Batch8([new], [new + 300], 8, 4, 64, 16, BF16, seed=7)
    case.q.mul_(2.0 ** 114)  # q . code up to some 2^126
    case.ks.mul_(2.0 ** -123)  # about 2^-129
    check_attn(m, case, scale=0.25, softcap=softcap)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,lens", [([60], [100]), ([300] * 8, [900] * 8), ([900], [2500]), ([4] * 20, [3000] * 20)])
def test_waits_that_run_out_over_scales_far_apart(m, new, lens, D):
    """Whatever a warp reads after a wait has run out, the call ends, and the workspace serves again."""
    case = Batch8(new, lens, 16, 2, D, 16, F16, seed=11)
    g = torch.Generator().manual_seed(3)
    case.vs *= 2.0 ** torch.randint(-40, 3, case.vs.shape, generator=g)
    ws = m.alloc_attention_workspace(16, 2, D, device=DEV)
    try:
        m.moe_debug_set_wait_limit(20_000_000)      # 20 ms
        m.moe_debug_withhold_arrivals(1)
        assert m.status_str(run_attn(m, case, ws=ws)[2]) == "MOE_ERR_TIMEOUT"
    finally:
        m.moe_debug_withhold_arrivals(0)
        m.moe_debug_set_wait_limit(0)
    m.moe_workspace_init(ws)
    check_attn(m, case, ws=ws)
