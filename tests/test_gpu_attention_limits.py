"""The attention half at the edges of what its entry points promise: waits that run out, contents of
rows that are nobody's, caps far from the scores, products past fp32, descriptions of the batch
that are wrong in part."""
import math

import pytest

from tests.block_cases import U32, Batch, attention_ref, half_step, norm_ref
from tests.test_gpu_attention_half import run_attn, run_rope, within
from tests.test_gpu_parity import DEV, m  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("new,lens", [([1], [93]), ([1] * 32, [1500] * 32), ([1], [60000]),
                                      ([3, 1], [60, 40]), ([60], [100]), ([300] * 8, [900] * 8), ([2000], [2500])])
def test_waits_that_run_out(m, new, lens):
    """CTA 0, whose run reaches keys in each of these, waits for an arrival that nobody makes (both
    kernels, items whole, parted and joined inside or by a launch): the call ends by itself, records
    MOE_ERR_TIMEOUT, and the workspace serves again once initialised."""
    case = Batch(new, lens, 8, 2, 128, 16, torch.bfloat16, seed=11)
    ws = m.alloc_attention_workspace(8, 2, 128, device=DEV)
    try:
        m.moe_debug_set_wait_limit(20_000_000)      # 20 ms
        m.moe_debug_withhold_arrivals(1)
        assert m.status_str(run_attn(m, case, ws=ws)[2]) == "MOE_ERR_TIMEOUT"
    finally:
        m.moe_debug_withhold_arrivals(0)
        m.moe_debug_set_wait_limit(0)
    m.moe_workspace_init(ws)
    out, lse, code, detail = run_attn(m, case, ws=ws)
    assert code == 0, (m.status_str(code), detail)
    o, e, tol, lse_tol = attention_ref(case, 1 / math.sqrt(128))
    within(out, o, tol, "out")
    within(lse, e, lse_tol, "lse")


@pytest.mark.parametrize("G,D,cap,sign", [(3, 128, 0.0, 1), (7, 64, 0.0, 1), (12, 128, 0.0, 1), (3, 128, 2.0, 1),
                                          (7, 128, 500.0, 1), (3, 64, 5.0, -1)])
def test_what_ran_before_leaves_no_trace(m, G, D, cap, sign):
    """A group that does not fill the tensor cores' 128 rows: the rows left over hold what the call
    before left in shared memory, and the result is the same bit for bit whatever that was."""
    Hkv = 2
    case = Batch([700, 1200], [2000, 1500], Hkv * G, Hkv, D, 16, torch.bfloat16, seed=G)
    other = Batch([2000, 2000], [2100, 2000], 4 * Hkv, Hkv, D, 16, torch.bfloat16, seed=1)  # fills all 128
    d, e = case.dev(DEV), other.dev(DEV)
    ws = m.alloc_attention_workspace(case.Hq, Hkv, D, device=DEV)
    out, out2 = torch.empty_like(d["q"]), torch.empty_like(e["q"])
    lse = torch.empty(case.N, case.Hq, device=DEV)
    got = []
    for size in (0.0, 30.0, 100.0, 1000.0):
        big = e["q"] * size
        torch.cuda.synchronize()
        m.moe_attention_paged(big, e["k"], e["v"], e["table"], e["offs"], e["lens"], 2000, 0.1, out2, ws)
        m.moe_attention_paged(d["q"], d["k"], d["v"], d["table"], d["offs"], d["lens"], 1200, sign * D ** -0.5, out,
                              ws, lse=lse, softcap=cap)
        assert m.moe_read_device_status(ws)[0] == 0
        got.append((out.clone(), lse.clone()))
    for o, s in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(s, got[0][1])


def capped_ref(case, scale, cap, window=0, exact=False):
    """out, lse and their bounds of a batch of one sequence, in fp64.  A score's error: that of its fp32
    products and sum, and 2^-20 of the score itself for the tangent (an exponential and a quotient
    of 2^-22 each, doubled by 1 - 2 / (1 + e^2y) where y is least, or ten roundings of a polynomial).
    Nothing grows with the cap.  ``exact``: the products are 0 or so far past the cap that the tangent
    of anything near them is 1."""
    n, L, G = case.new[0], case.lens_list[0], case.Hq // case.Hkv
    k, v = case.cached(0, case.k), case.cached(0, case.v)
    q = case.q[:n].double().view(n, case.Hkv, G, case.D).permute(1, 2, 0, 3)
    z = torch.einsum("hgnd,hkd->hgnk", q, k) * scale
    dz = torch.einsum("hgnd,hkd->hgnk", q.abs(), k.abs()) * abs(scale) * (case.D + 8) * U32
    z, dz = cap * torch.tanh(z / cap), dz * (not exact)
    seen = torch.arange(L)[None] <= torch.arange(L - n, L)[:, None]
    if window > 0:
        seen &= torch.arange(L)[None] > torch.arange(L - n, L)[:, None] - window
    dz = torch.where(seen, dz + z.abs() * 2.0 ** -20, 0.0)
    z = z.masked_fill(~seen, -math.inf)
    e = torch.logsumexp(z, -1)
    p = torch.exp(z - e[..., None])
    o, absv = (torch.einsum("hgnk,hkd->hgnd", p, x) for x in (v, v.abs()))
    u = half_step(case.dtype)
    rel = 2 * dz.amax(-1) + 2.0 ** -20 + (L + 64) * U32
    tol = (rel[..., None] + u) * absv
    tol = tol + u * (o.abs() + tol)
    lse_tol = dz.amax(-1) + 2.0 ** -20 + (L + 64) * U32 + 4 * U32 * e.abs()

    def put(x):
        return x.permute(2, 0, 1, *range(3, x.dim())).reshape(n, case.Hq, *x.shape[3:])
    return put(o), put(e), put(tol), put(lse_tol)


@pytest.mark.parametrize("new,L", [(1, 700), (3, 90), (90, 400)])
@pytest.mark.parametrize("cap", [1e3, 1e4, 1e5, 1e6, 1e9, 1e30])
@pytest.mark.parametrize("sign", [1, -1])
def test_far_caps(m, new, L, cap, sign):
    """A cap far beyond the scores leaves them as they are."""
    case = Batch([new], [L], 8, 2, 128, 16, torch.bfloat16, seed=L)
    scale = sign * 128 ** -0.5
    out, lse, code, _ = run_attn(m, case, softcap=cap, scale=scale)
    assert code == 0
    o, e, tol, lse_tol = capped_ref(case, scale, cap)
    within(lse, e, lse_tol, "lse")
    within(out, o, tol, "out")


@pytest.mark.parametrize("new,L", [(1, 700), (90, 400)])
@pytest.mark.parametrize("cap", [65.0, 300.0, 2000.0])
def test_scores_around_the_cap(m, new, L, cap):
    """Scores from far below the cap to past it."""
    for reach in (0.1, 0.5, 0.6, 3.0):
        case = Batch([new], [L], 8, 2, 64, 16, torch.bfloat16, seed=L)
        scale = 64 ** -0.5 * cap * reach / 3  # three standard deviations at reach * cap
        out, lse, code, _ = run_attn(m, case, softcap=cap, scale=scale)
        assert code == 0
        o, e, tol, lse_tol = capped_ref(case, scale, cap)
        within(lse, e, lse_tol, "lse")
        within(out, o, tol, "out")


@pytest.mark.parametrize("new,L,window", [(1, 500, 0), (1, 700, 130), (90, 400, 0), (300, 900, 200)])
@pytest.mark.parametrize("cap,scale", [(30.0, 0.1), (30.0, -0.1), (500.0, 0.1), (5.0, 2.0)])
@pytest.mark.parametrize("size", [1e19, 1e18])
def test_products_past_fp32(m, new, L, window, cap, scale, size):
    """Finite rows whose products leave fp32 (1e38 * 128) or come near its end: the cap brings them back
    to itself, in tiles that rows see whole and in others; keys of one sign for rows that see no other."""
    case = Batch([new], [L], 8, 2, 128, 16, torch.bfloat16, seed=L)
    case.q.fill_(size)
    for kinds in ((-1.0, 0.0, 1.0), (-1.0,), (1.0,)):
        for j in range(L):
            case.k[int(case.table[0, j // 16]), :, j % 16] = size * kinds[j * 7 % 11 % len(kinds)]
        out, lse, code, _ = run_attn(m, case, softcap=cap, scale=scale, window=window)
        assert code == 0
        o, e, tol, lse_tol = capped_ref(case, scale, cap, window, exact=True)
        within(lse, e, lse_tol, "lse")
        within(out, o, tol, "out")


def good_rows(case):
    """(sequence, row) of the new rows of sequences whose offsets and length are in range."""
    offs, lens = case.offs.tolist(), case.lens.tolist()
    most = case.table.shape[1] * case.page
    for b, (lo, hi, L) in enumerate(zip(offs, offs[1:], lens)):
        if 0 <= lo <= hi <= case.N and 0 <= L <= most:
            yield from ((b, r) for r in range(lo, hi))


def check_rope_in_part(m, case, code):
    """A batch whose description is wrong in part: recorded, the good sequences' rows right, and no
    other cache row touched."""
    r = run_rope(m, case, torch.arange(case.N, dtype=torch.int32)[None], 64)
    assert m.status_str(r["code"]) == code, r["code"]
    offs, lens = case.offs.tolist(), case.lens.tolist()
    kept = torch.ones(case.k.shape[:3], dtype=torch.bool)
    n = 0
    for b, row in good_rows(case):
        within(r["q_out"][row], r["q"][row], r["qe"][row], f"q of row {row}")
        j = lens[b] - (offs[b + 1] - row)
        pg = int(case.table[b, j // case.page]) if j >= 0 else -1
        if not 0 <= pg < case.P:
            continue
        at = (pg, slice(None), j % case.page)
        within(r["k"][at], r["k_ref"][row], r["ke"][row], f"k of row {row}")
        assert torch.equal(r["v"][at].double(), r["v_ref"][row])
        kept[at] = False
        n += 1
    for new, old in ((r["k"], case.k), (r["v"], case.v)):
        a, o = new[kept], old[kept]
        assert torch.equal(a.isnan(), o.isnan()) and torch.equal(a.nan_to_num(), o.nan_to_num())
    return n


@pytest.mark.parametrize("offs", [
    [0, 100, 3, 5], [0, -1, 3, 6], [4, 2, 4, 6], [1 << 30, 0, 3, 6], [2, 5, 0, 2], [2, 5, 0, 0, 1, 2],
    [0, 2, -5, 1 << 30, 2, 4, 6], [5, 6, 0, 1, 1, 3, 3, 5], [-(2 ** 31), 2 ** 31 - 1, 0, 6]], ids=str)
def test_rope_with_offsets_that_do_not_rise(m, offs):
    """The sequences between good offsets keep their rows, wherever the bad ones stand."""
    B = len(offs) - 1
    case = Batch([6] + [0] * (B - 1), [20 + b for b in range(B)], 4, 2, 64, 16, torch.float16)
    case.offs.copy_(torch.tensor(offs))
    assert check_rope_in_part(m, case, "MOE_ERR_CACHE_RANGE") > 0


def test_rope_with_one_bad_offset_among_many(m):
    """Rows of many warps, 200 sequences, one offset out of place."""
    for at, bad in ((0, 500), (1, 1 << 20), (57, -3), (100, 700), (199, 650), (200, 9)):
        case = Batch([3] * 200, [4 + b % 40 for b in range(200)], 4, 2, 64, 16, torch.float16)
        case.offs[at] = bad
        assert check_rope_in_part(m, case, "MOE_ERR_CACHE_RANGE") >= 3 * 100


@pytest.mark.parametrize("what,bad", [("page", -1), ("page", 1 << 30), ("page", -(2 ** 31)), ("length", -1),
                                      ("length", 49), ("length", 2 ** 31 - 1)])
def test_rope_writes_nothing_through_a_bad_page_or_length(m, what, bad):
    case = Batch([2, 3, 4], [20, 33, 40], 4, 2, 64, 16, torch.float16)
    if what == "page":
        case.table[1, 2] = bad  # the page of the last of the second sequence's three new tokens
    else:
        case.lens[1] = bad
    assert check_rope_in_part(m, case, "MOE_ERR_CACHE_RANGE") == (8 if what == "page" else 6)


@pytest.mark.parametrize("new,lens", [([1, 1, 1], [40, 33, 48]), ([40, 30, 20], [60, 33, 48])])
def test_a_graph_over_a_table_that_changes(m, new, lens):
    """Captured once; replayed with other pages and lengths, over which the rows are others."""
    cases = [Batch(new, [L - d for L in lens], 8, 2, 128, 16, torch.bfloat16, seed=20 + d) for d in (0, 3, 9)]
    pages, width = max(c.P for c in cases), max(c.table.shape[1] for c in cases)
    d = cases[0].dev(DEV)
    k, v = (torch.full((pages, 2, 16, 128), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = torch.full((3, width), 1 << 30, dtype=torch.int32, device=DEV)
    out = torch.empty_like(d["q"])
    lse = torch.empty(cases[0].N, 8, device=DEV)
    ws = m.alloc_attention_workspace(8, 2, 128, device=DEV)

    def show(case):
        k[:case.P].copy_(case.k), v[:case.P].copy_(case.v), d["q"].copy_(case.q), d["lens"].copy_(case.lens)
        table[:, :case.table.shape[1]].copy_(case.table)

    show(cases[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_attention_paged(d["q"], k, v, table, d["offs"], d["lens"], max(new), 128 ** -0.5, out, ws, lse=lse)
    for case in cases + cases[:1]:
        show(case)
        g.replay()
        assert m.moe_read_device_status(ws)[0] == 0
        o, e, tol, lse_tol = attention_ref(case, 128 ** -0.5)
        within(out, o, tol, "out")
        within(lse, e, lse_tol, "lse")


@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_of_a_row_of_zeros(m, eps):
    """0 / sqrt(eps): zeros, and with eps 0 NaN as the formula has it (the sum stays 0); other rows as ever."""
    x = torch.zeros(3, 512, device=DEV)
    x[1] = torch.randn(512, device=DEV)
    r = torch.zeros(3, 512, device=DEV)
    s, y = (torch.full((3, 512), 7.0, device=DEV) for _ in range(2))
    m.moe_add_rmsnorm(x, r, torch.ones(512, device=DEV), eps, sum_out=s, y=y)
    assert torch.equal(s, x)
    if eps == 0.0:
        assert bool(y[::2].isnan().all())
    else:
        assert bool((y[::2] == 0).all())
    want = norm_ref(x[1:2].cpu(), None, torch.ones(512), eps)[1]
    within(y[1:2], want, want.abs() * (512 / 2 + 8) * U32, "the row between")


def test_a_workspace_that_the_experts_have_used(m):
    """The single-token layer's tags lie where the parts of items are counted: recorded, not overlooked;
    initialised anew the workspace serves."""
    from quantized_routed_expert_02_gb300 import synth
    from tests.test_gpu_parity import layer_case, to_dev
    c = layer_case(synth.SHAPES["tiny"], 0, None)
    s, d = c["shape"], to_dev(c)
    ws = m.alloc_attention_workspace(8, 2, 128, device=DEV)
    assert ws.numel() >= m.moe_workspace_bytes(1, s.H, s.E, s.k, s.I)
    m.moe_layer(d["x"], d["Wr"], d["bias"], d["gate"], d["up"], d["down"], s.k, s.I, d["idx"], d["w"], d["y"], ws)
    assert m.moe_read_device_status(ws)[0] == 0
    case = Batch([1] * 32, [1500] * 32, 8, 2, 128, 16, torch.bfloat16, seed=3)  # parted, joined inside
    assert m.status_str(run_attn(m, case, ws=ws)[2]) == "MOE_ERR_WORKSPACE"
    m.moe_workspace_init(ws)
    out, lse, code, detail = run_attn(m, case, ws=ws)
    assert code == 0, (m.status_str(code), detail)
    o, e, tol, lse_tol = attention_ref(case, 128 ** -0.5)
    within(out, o, tol, "out")
    within(lse, e, lse_tol, "lse")


@pytest.mark.parametrize("new,lens", [([1, 1], [300, 1]), ([4, 3], [2, 90]), ([70, 150], [40, 900])])
@pytest.mark.parametrize("window", [(1 << 30) - 1, 1 << 30, 2 ** 31 - 1])
def test_windows_past_every_length(m, new, lens, window):
    """The widest windows hide nothing, also from tokens before the cache's start."""
    case = Batch(new, lens, 8, 2, 128, 16, torch.bfloat16, seed=5)
    plain = run_attn(m, case)
    wide = run_attn(m, case, window=window)
    assert wide[2] == 0
    used = sum(new)
    assert torch.equal(wide[0][:used], plain[0][:used]) and torch.equal(wide[1][:used], plain[1][:used])
