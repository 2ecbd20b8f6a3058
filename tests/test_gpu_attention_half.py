"""The attention half of a decoder block through the C ABI against 64-bit
references: moe_add_rmsnorm, moe_rope_append, moe_attention_paged."""
import math

import numpy as np
import pytest

from tests.block_cases import U32, Batch, attention_ref, half_step, inv_freq, norm_ref, rope_ref
from tests.test_gpu_parity import DEV, m  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

EPS = 1e-6


def within(got, want, tol, what):
    d = (got.double().cpu() - want).abs()
    bad = ~(d <= tol)
    bad &= ~((got.double().cpu() == want) & torch.isinf(want))
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, first at {bad.nonzero()[0].tolist()}, "
        f"worst excess {float((d - tol)[bad].nan_to_num(nan=math.inf).max()):.3e}")


# --------------------------------------------------------------------------
# moe_add_rmsnorm
# --------------------------------------------------------------------------
NORM = [(1, 256), (1, 2048), (3, 8), (5, 264), (2, 4096), (33, 768), (7, 2568), (2, 8192), (2, 16384), (1000, 512)]


@pytest.mark.parametrize("xt", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("yt", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,H", NORM)
def test_norm(m, T, H, xt, yt):
    types = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
    g = torch.Generator().manual_seed(T * 31 + H)
    x = torch.randn(T, H, generator=g).to(types[xt])
    r = 3 * torch.randn(T, H, generator=g)
    w = 1 + 0.3 * torch.randn(H, generator=g)
    s, y = norm_ref(x, r, w, EPS)
    so = torch.full((T, H), float("nan"), device=DEV)
    yo = torch.full((T, H), float("nan"), device=DEV, dtype=types[yt])
    m.moe_add_rmsnorm(x.to(DEV), r.to(DEV), w.to(DEV), EPS, sum_out=so, y=yo)
    torch.cuda.synchronize()
    within(so, s, U32 * s.abs(), "sum")
    # sum, squares and their sum (at most H/2 deep, halved by the root), root, quotient, two products
    rel = (H / 2 + 8) * U32
    u = half_step(types[yt])
    within(yo, y, y.abs() * rel + u * y.abs() * (1 + rel) + torch.finfo(types[yt]).smallest_normal * u, "y")


@pytest.mark.parametrize("T,H", [(1, 2048), (3, 256), (37, 4096), (2, 16384)])
def test_norm_q8k_is_the_quantiser(m, T, H):
    """The codes, scales and sums are those of moe_quantize_q8k on the fp32 rows, bit for bit;
    without y they are the same."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(T, H, generator=g)
    x[0, :256] = 0
    x = x.to(DEV)
    w = torch.randn(H, generator=g).to(DEV)
    e = lambda n, t: torch.full((T, n), 77, dtype=t, device=DEV)  # noqa: E731
    y = torch.empty(T, H, device=DEV)
    a = (e(H, torch.int8), e(H // 256, torch.float32), e(H // 32, torch.int32))
    b, c = tuple(t.clone() for t in a), tuple(t.clone() for t in a)
    m.moe_add_rmsnorm(x, None, w, EPS, y=y, q8k=a)
    m.moe_quantize_q8k(y, *b)
    m.moe_add_rmsnorm(x, None, w, EPS, q8k=c)
    torch.cuda.synchronize()
    for u, v, z in zip(a, b, c):
        assert torch.equal(u, v) and torch.equal(u, z)


def test_norm_edges(m):
    """Zero rows, eps 0, in-place sums, a row with an infinity or a NaN beside finite rows."""
    H = 512
    x = torch.randn(4, H, device=DEV)
    x[1] = 0
    x[2, 7] = float("inf")
    x[3, 500] = float("nan")
    w = torch.ones(H, device=DEV)
    y = torch.empty(4, H, device=DEV)
    m.moe_add_rmsnorm(x, None, w, EPS, y=y)
    s, want = norm_ref(x[:2].cpu(), None, w.cpu(), EPS)
    within(y[:2], want, want.abs() * (H / 2 + 8) * U32, "finite rows")
    assert torch.equal(y[2].isnan().nonzero().flatten().cpu(), torch.tensor([7]))
    assert bool(y[3].isnan().all())
    r = torch.randn(4, H, device=DEV)
    keep = r.clone()
    m.moe_add_rmsnorm(x, r, w, 0.0, sum_out=r, y=y)  # in place
    assert torch.equal(r[:2], (keep + x)[:2])
    z = torch.zeros(1, H, device=DEV)
    m.moe_add_rmsnorm(z, None, w, 0.0, sum_out=None, y=y[:1])
    torch.cuda.synchronize()


def test_norm_feeds_the_integer_experts(m):
    """moe_ffn_q8k_codes on the norm's codes is moe_ffn_q8k on its fp32 rows, bit for bit."""
    from quantized_routed_expert_02_gb300 import synth
    T, H, E, k, I = 5, 512, 8, 3, 256
    shape = synth.custom_shape(T, H, E, k, I, cfg_id=91)
    blobs = {n: torch.from_numpy(b).to(DEV) for n, b in synth.expert_blobs(shape, 0).items()}
    x = torch.randn(T, H, device=DEV)
    w = torch.rand(H, device=DEV) + 0.5
    y = torch.empty(T, H, device=DEV)
    q = (torch.empty(T, H, dtype=torch.int8, device=DEV), torch.empty(T, H // 256, device=DEV),
         torch.empty(T, H // 32, dtype=torch.int32, device=DEV))
    m.moe_add_rmsnorm(x, None, w, EPS, y=y, q8k=q)
    idx = torch.tensor(np.stack([np.random.default_rng(i).permutation(E)[:k] for i in range(T)]),
                       dtype=torch.int32, device=DEV)
    rw = torch.rand(T, k, device=DEV)
    ws = m.alloc_workspace(T, H, E, k, I, device=DEV)
    a, b = torch.empty(T, H, device=DEV), torch.empty(T, H, device=DEV)
    m.moe_ffn_q8k(y, idx, rw, blobs["gate"], blobs["up"], blobs["down"], E, I, a, ws)
    m.moe_ffn_q8k_codes(*q, idx, rw, blobs["gate"], blobs["up"], blobs["down"], E, I, b, ws)
    torch.cuda.synchronize()
    assert bool(a.abs().max() > 0) and torch.equal(a, b)


# --------------------------------------------------------------------------
# moe_rope_append
# --------------------------------------------------------------------------
def run_rope(m, case, pos, rot, axis=None, qk_norm=False, interleaved=False, seed=1):
    g = torch.Generator().manual_seed(seed)
    N, Hq, Hkv, D = case.N, case.Hq, case.Hkv, case.D
    qkv = torch.randn(N, (Hq + 2 * Hkv) * D, generator=g).to(case.dtype)
    qw = 1 + 0.3 * torch.randn(D, generator=g) if qk_norm else None
    kw = 1 + 0.3 * torch.randn(D, generator=g) if qk_norm else None
    f = inv_freq(rot)
    d = case.dev(DEV)
    q_out = torch.full((N, Hq, D), float("nan"), dtype=case.dtype, device=DEV)
    ws = m.alloc_attention_workspace(Hq, Hkv, D, device=DEV)
    up = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    m.moe_rope_append(qkv.to(DEV), pos.to(DEV), f.to(DEV), q_out, d["k"], d["v"], d["table"], d["offs"],
                      d["lens"], ws, axis=up(axis), q_norm_w=up(qw), k_norm_w=up(kw), eps=EPS,
                      interleaved=interleaved)
    code, detail = m.moe_read_device_status(ws)
    q, k, v, qe, ke = rope_ref(qkv, pos, f, axis, Hq, Hkv, D, qw, kw, EPS, interleaved)
    return dict(q_out=q_out.cpu(), k=d["k"].cpu(), v=d["v"].cpu(), q=q, k_ref=k, v_ref=v, qe=qe, ke=ke,
                code=code, detail=detail)


def check_rope(case, r):
    assert r["code"] == 0
    wk, wv = torch.zeros(case.k.shape[:3], dtype=torch.bool), None
    row = 0
    for b, (n, L) in enumerate(zip(case.new, case.lens_list)):
        within(r["q_out"][row:row + n], r["q"][row:row + n], r["qe"][row:row + n], f"q of sequence {b}")
        for i in range(n):
            j = L - n + i
            if j < 0:
                continue
            pg = int(case.table[b, j // case.page])
            within(r["k"][pg, :, j % case.page], r["k_ref"][row + i], r["ke"][row + i], f"k {b},{i}")
            assert torch.equal(r["v"][pg, :, j % case.page].double(), r["v_ref"][row + i])
            wk[pg, :, j % case.page] = True
        row += n
    # nothing else was written
    keep = ~wk
    for new, old in ((r["k"], case.k), (r["v"], case.v)):
        a, o = new[keep], old[keep]
        assert torch.equal(a.isnan(), o.isnan()) and torch.equal(a.nan_to_num(), o.nan_to_num())
    assert bool(r["q_out"][row:].isnan().all())  # rows of no sequence


ROPE = [
    # new, lens, Hq, Hkv, D, page, rot
    ([1], [1], 4, 1, 128, 16, 128),
    ([1], [700], 32, 4, 128, 16, 128),
    ([5, 0, 1, 17], [5, 9, 33, 40], 28, 4, 128, 32, 64),
    ([3, 2], [64, 65], 8, 8, 64, 64, 64),
    ([40, 1], [40, 256], 12, 2, 64, 128, 16),
    ([7], [300], 3, 1, 64, 256, 48),
    ([2000], [2100], 16, 2, 64, 16, 32),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("qk_norm", [False, True])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D,page,rot", ROPE)
def test_rope(m, new, lens, Hq, Hkv, D, page, rot, qk_norm, interleaved, dtype):
    case = Batch(new, lens, Hq, Hkv, D, page, dtype, seed=3, spare_rows=2)
    pos = torch.cat([torch.arange(L - n, L) for n, L in zip(new, lens)] + [torch.zeros(2, dtype=torch.long)])
    check_rope(case, run_rope(m, case, pos[None].to(torch.int32), rot, qk_norm=qk_norm, interleaved=interleaved))


@pytest.mark.parametrize("layout", ["runs", "turns"])
def test_rope_axes(m, layout):
    """Three axes, assigned to pairs in runs or in turns; far, negative and extreme positions."""
    case = Batch([9, 4], [9, 30], 8, 2, 128, 16, torch.bfloat16, seed=4)
    pos = torch.randint(0, 1 << 20, (3, case.N), generator=torch.Generator().manual_seed(2)).to(torch.int32)
    pos[0, 0], pos[1, 0], pos[2, 1], pos[0, 2] = 2 ** 31 - 1, -(2 ** 31), -5, 10_000_001
    axis = torch.arange(64) * 3 // 64 if layout == "runs" else torch.arange(64) % 3
    check_rope(case, run_rope(m, case, pos, 128, axis=axis.to(torch.int32), qk_norm=True))


def test_rope_more_tokens_than_cached(m):
    """kv_lens < n: the tokens before the cache's start are rotated, not cached."""
    case = Batch([5], [2], 4, 2, 64, 16, torch.float16)
    pos = torch.arange(5, dtype=torch.int32)[None]
    check_rope(case, run_rope(m, case, pos, 64))


def test_rope_bad_pages_and_lengths(m):
    """Out-of-range descriptions are recorded and nothing is written through them."""
    def spoiled(change):
        case = Batch([2, 3], [20, 33], 4, 2, 64, 16, torch.float16)
        change(case)
        r = run_rope(m, case, torch.zeros(1, case.N, dtype=torch.int32), 64)
        return case, r
    def same(a, o):
        return torch.equal(a.isnan(), o.isnan()) and torch.equal(a.nan_to_num(), o.nan_to_num())
    for bad in (-1, 1 << 30, 9):
        case, r = spoiled(lambda c: c.table.__setitem__((1, 1), bad))
        P = case.P
        if 0 <= bad < P:
            continue
        assert m.status_str(r["code"]) == "MOE_ERR_CACHE_RANGE" and r["detail"] == bad
    for L in (-1, 16 * 3 + 1, 2 ** 31 - 1):
        case, r = spoiled(lambda c: c.lens.__setitem__(1, L))
        assert m.status_str(r["code"]) == "MOE_ERR_CACHE_RANGE" and r["detail"] == L
    for o in ([0, 6, 5], [0, -1, 5], [0, 2, 99], [7, 8, 9]):
        case, r = spoiled(lambda c: c.offs.copy_(torch.tensor(o)))
        assert m.status_str(r["code"]) == "MOE_ERR_CACHE_RANGE", o


# --------------------------------------------------------------------------
# moe_attention_paged
# --------------------------------------------------------------------------
def run_attn(m, case, window=0, softcap=0.0, scale=None, most=None, ws=None, stream=None):
    scale = 1 / math.sqrt(case.D) if scale is None else scale
    d = case.dev(DEV)
    out = torch.full((case.N, case.Hq, case.D), float("nan"), dtype=case.dtype, device=DEV)
    lse = torch.full((case.N, case.Hq), float("nan"), device=DEV)
    ws = m.alloc_attention_workspace(case.Hq, case.Hkv, case.D, device=DEV) if ws is None else ws
    m.moe_attention_paged(d["q"], d["k"], d["v"], d["table"], d["offs"], d["lens"], most or case.most, scale,
                          out, ws, lse=lse, window=window, softcap=softcap)
    code, detail = m.moe_read_device_status(ws)
    return out, lse, code, detail


def check_attn(m, case, window=0, softcap=0.0, scale=None, most=None):
    out, lse, code, detail = run_attn(m, case, window, softcap, scale, most)
    assert code == 0, (m.status_str(code), detail)
    o, e, tol, lse_tol = attention_ref(case, 1 / math.sqrt(case.D) if scale is None else scale, window, softcap)
    used = sum(case.new)
    within(out[:used], o[:used], tol[:used], "out")
    within(lse[:used], e[:used], lse_tol[:used], "lse")
    assert bool(out[used:].isnan().all()) and bool(lse[used:].isnan().all())


ATTN = [
    # new, lens, Hq, Hkv, D, page
    ([1], [1], 4, 1, 128, 16),
    ([1], [93], 32, 4, 128, 16),
    ([1], [2049], 16, 2, 64, 64),
    ([1, 1, 1], [1, 17, 1000], 28, 4, 128, 32),
    ([1, 0, 1, 1], [5, 7, 129, 128], 8, 8, 64, 128),
    ([1] * 7, [3, 64, 65, 127, 255, 256, 257], 64, 4, 128, 256),
    ([6, 6, 5], [6, 300, 1111], 64, 4, 128, 16),
    ([2, 3, 1], [2, 50, 700], 12, 2, 64, 16),
    ([17], [17], 32, 4, 128, 16),
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
IDS = [f"B{len(a[0])}n{max(a[0])}L{max(a[1])}h{a[2]}k{a[3]}d{a[4]}p{a[5]}" for a in ATTN]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("window,softcap", [(0, 0.0), (1, 0.0), (37, 15.0)], ids=["plain", "window1", "win37cap"])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D,page", ATTN, ids=IDS)
def test_attention(m, new, lens, Hq, Hkv, D, page, window, softcap, dtype):
    case = Batch(new, lens, Hq, Hkv, D, page, dtype, seed=len(new) + max(lens), spare_rows=3)
    check_attn(m, case, window, softcap)


@pytest.mark.parametrize("most", [1, 4, 100000])
def test_attention_max_new_is_a_hint(m, most):
    """A wrong max_new gives the same results within the bounds."""
    check_attn(m, Batch([1, 40, 3], [500, 90, 3], 16, 2, 128, 16, torch.bfloat16), most=most)


@pytest.mark.parametrize("new,L", [(1, 5000), (40, 3000)])
def test_attention_large_scores(m, new, L):
    """Scores far apart (a one-hot softmax), rising and falling along the keys: the running maximum
    moves at every tile."""
    for sign in (1, -1):
        case = Batch([new], [L], 8, 2, 128, 32, torch.float16, seed=8)
        ramp = sign * torch.linspace(-3, 3, L)
        for j in range(L):
            case.k[int(case.table[0, j // 32]), :, j % 32] = ramp[j].half()
        case.q.fill_(1.0)
        check_attn(m, case)
        check_attn(m, case, scale=-0.05)


def test_attention_zero_scale_is_the_mean(m):
    check_attn(m, Batch([2, 1], [77, 300], 8, 2, 64, 16, torch.bfloat16), scale=0.0)


def test_attention_rows_past_the_end(m):
    """Infinities and NaN in the cache rows past each length do not reach the output."""
    for fill in (float("inf"), -float("inf"), float("nan"), 65504.0):
        case = Batch([1, 1, 20], [15, 100, 50], 16, 2, 128, 16, torch.float16, seed=2)
        for t in (case.k, case.v):
            t.nan_to_num_(nan=fill, posinf=fill, neginf=fill)
        check_attn(m, case)


@pytest.mark.parametrize("B,new,tile", [(1, 1, 64), (19, 1, 64), (40, 1, 64), (1, 70, 128), (9, 40, 128), (30, 90, 128)])
def test_attention_whole_and_parted(m, B, new, tile):
    """Lengths around those from which items are parted, one long sequence among short ones."""
    for tiles in (2, 3, 9, 10, 17):
        lens = [tiles * tile + d for d in (-1, 0, 1)] * B
        check_attn(m, Batch([new] * B, lens[:B], 8, 2, 64, 16, torch.bfloat16, seed=tiles))
    check_attn(m, Batch([new] * B, [new + 5] * (B - 1) + [40 * tile], 8, 2, 64, 16, torch.bfloat16))


@pytest.mark.parametrize("new,lens,page,D,cap", [
    ([1, 1, 1, 1], [900, 90, 129, 4000], 16, 128, 0.0), ([1, 5, 2], [700, 230, 64], 32, 64, 20.0),
    ([150, 1, 40], [900, 800, 45], 16, 128, 0.0), ([300, 33], [301, 2000], 64, 64, 20.0),
    ([20, 200], [1500, 700], 128, 128, 0.0), ([9, 130], [1500, 700], 256, 64, 0.0)])
def test_attention_pages_before_the_window(m, new, lens, page, D, cap):
    """Pages that no new token sees may be gone: their entries name nothing, their rows are NaN."""
    for window in (1, 70, 128):
        case = Batch(new, lens, 12, 3, D, page, torch.bfloat16, seed=window)
        o, e, tol, lse_tol = attention_ref(case, 1 / math.sqrt(D), window, cap)
        for b, (n, L) in enumerate(zip(new, lens)):
            gone = max(0, L - n - window + 1) // page
            for t in (case.k, case.v):
                t[case.table[b, :gone].long()] = float("nan")
            case.table[b, :gone] = -1
        out, lse, code, detail = run_attn(m, case, window=window, softcap=cap)
        assert code == 0, (m.status_str(code), detail)
        within(out, o, tol, "out")
        within(lse, e, lse_tol, "lse")


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("softcap", [0.0, 10.0])
def test_attention_nan_query(m, new, softcap):
    """A NaN in a query head reaches that row's output and lse, and no other."""
    case = Batch([new, new], [500, 900], 8, 2, 128, 16, torch.float16)
    o, e, tol, lse_tol = attention_ref(case, 1 / math.sqrt(128), 0, softcap)
    case.q[new // 2, 3, 5] = float("nan")
    out, lse, code, _ = run_attn(m, case, softcap=softcap)
    assert code == 0
    assert bool(out[new // 2, 3].isnan().all()) and bool(lse[new // 2, 3].isnan())
    for t in (out, lse, o, e):
        t[new // 2, 3] = 0.0
    within(out, o, tol, "out")
    within(lse, e, lse_tol, "lse")


def test_attention_bad_descriptions(m):
    """A page, length or offset out of range is recorded; the other sequences stay right."""
    for what, bad in (("table", -3), ("table", 1 << 30), ("lens", 1 << 30), ("lens", -1), ("lens", 49)):
        for new in ([1, 1, 1], [20, 30, 3]):
            case = Batch(new, [40, 33, 48], 8, 2, 128, 16, torch.bfloat16)
            o, e, tol, _ = attention_ref(case, 1 / math.sqrt(128))
            if what == "table":
                case.table[1, 1] = bad
            else:
                case.lens[1] = bad
            out, lse, code, detail = run_attn(m, case)
            assert m.status_str(code) == "MOE_ERR_CACHE_RANGE" and detail == bad
            for rows in (slice(0, new[0]), slice(new[0] + new[1], sum(new))):
                within(out[rows], o[rows], tol[rows], "a good sequence")
    for offs in ([0, 9, 5, 12], [0, -4, 5, 12], [0, 3, 5, 1 << 30], [1 << 30, 3, 4, 5]):
        case = Batch([3, 2, 7], [40, 33, 48], 8, 2, 128, 16, torch.bfloat16)
        case.offs.copy_(torch.tensor(offs))
        assert m.status_str(run_attn(m, case)[2]) == "MOE_ERR_CACHE_RANGE", offs


def test_attention_repeat_is_bitwise(m):
    for new, lens in (([1] * 5, [3000, 12, 900, 64, 7000]), ([300, 40], [2000, 2600])):
        case = Batch(new, lens, 32, 4, 128, 16, torch.bfloat16)
        ws = m.alloc_attention_workspace(32, 4, 128, device=DEV)
        a = run_attn(m, case, ws=ws)
        for _ in range(3):
            b = run_attn(m, case, ws=ws)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("seed", range(40))
def test_attention_drawn(m, seed):
    """Ragged batches, head layouts, pages, masks and scales drawn at random."""
    r = np.random.default_rng([7, seed])
    Hkv = int(r.choice([1, 2, 3, 4]))
    G = int(r.choice([1, 2, 3, 5, 7, 8, 16, 24, 40]))
    D, page = int(r.choice([64, 128])), int(r.choice([16, 32, 64, 128, 256]))
    B = int(r.integers(1, 7))
    most = int(r.choice([1, 1, 3, 20, 150]))
    new = [int(r.integers(0, most + 1)) for _ in range(B)]
    new[0] = max(1, new[0])
    lens = [int(max(0, n + r.integers(-3, 1) if r.random() < 0.2 else n + r.integers(0, 900))) for n in new]
    dtype = torch.float16 if r.random() < 0.5 else torch.bfloat16
    case = Batch(new, lens, Hkv * G, Hkv, D, page, dtype, seed=seed, spare_rows=int(r.integers(0, 3)))
    check_attn(m, case, window=int(r.choice([0, 0, 1, 17, 128, 300])), softcap=float(r.choice([0, 0, 3.0, 40.0])),
               scale=float(r.choice([D ** -0.5, D ** -0.5, -0.1, 0.3])))


@pytest.mark.parametrize("B,most", [(700, 1), (4096, 1), (300, 12)])
def test_attention_many_sequences(m, B, most):
    """More sequences than CTAs, most of them short, some empty."""
    r = np.random.default_rng(B)
    new = [int(x) for x in r.integers(0, most + 1, B)]
    lens = [n + int(x) for n, x in zip(new, r.integers(0, 40, B))]
    check_attn(m, Batch(new, lens, 8, 2, 64, 16, torch.bfloat16, seed=B))


def test_cache_past_32_bits(m):
    """A cache of over 2^31 values (and 2^32 bytes) per tensor: rows at its far end are written and read."""
    Hq, Hkv, D, page = 16, 4, 128, 64
    case = Batch([3, 40], [700, 130], Hq, Hkv, D, page, torch.bfloat16, seed=9)
    P = (1 << 31) // (Hkv * page * D) + case.P + 5
    far = {}
    for n in ("k", "v"):
        far[n] = torch.empty(P, Hkv, page, D, dtype=case.dtype, device=DEV)
        far[n][P - case.P:] = getattr(case, n).to(DEV)
    table = torch.where(case.table < case.P, case.table + (P - case.P), 1 << 30).to(DEV)
    ws = m.alloc_attention_workspace(Hq, Hkv, D, device=DEV)
    out = torch.full((case.N, Hq, D), float("nan"), dtype=case.dtype, device=DEV)
    for most in (1, 40):  # both kernels
        m.moe_attention_paged(case.q.to(DEV), far["k"], far["v"], table, case.offs.to(DEV), case.lens.to(DEV), most,
                              D ** -0.5, out, ws)
        o, _, tol, _ = attention_ref(case, D ** -0.5)
        within(out, o, tol, "out")
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(case.N, (Hq + 2 * Hkv) * D, generator=g).to(case.dtype)
    pos = torch.cat([torch.arange(L - n, L) for n, L in zip(case.new, case.lens_list)])[None].to(torch.int32)
    m.moe_rope_append(qkv.to(DEV), pos.to(DEV), inv_freq(D).to(DEV), out, far["k"], far["v"], table,
                      case.offs.to(DEV), case.lens.to(DEV), ws)
    assert m.moe_read_device_status(ws)[0] == 0
    q, k, v, qe, ke = rope_ref(qkv, pos, inv_freq(D), None, Hq, Hkv, D, None, None, EPS, False)
    r = dict(q_out=out.cpu(), k=far["k"][P - case.P:].cpu(), v=far["v"][P - case.P:].cpu(), q=q, k_ref=k, v_ref=v,
             qe=qe, ke=ke, code=0)
    check_rope(case, r)


def test_attention_in_a_graph_on_a_side_stream(m):
    """Captured once, replayed while the lengths and the table grow on the device."""
    case = Batch([1, 1], [64, 30], 16, 2, 128, 16, torch.bfloat16, seed=6)
    full = [64, 30]
    d = case.dev(DEV)
    out = torch.empty(2, 16, 128, dtype=case.dtype, device=DEV)
    ws = m.alloc_attention_workspace(16, 2, 128, device=DEV)
    side = torch.cuda.Stream()
    call = lambda: m.moe_attention_paged(d["q"], d["k"], d["v"], d["table"], d["offs"], d["lens"], 1,  # noqa: E731
                                         128 ** -0.5, out, ws)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call()
    for lens in ([1, 1], [17, 30], [64, 16]):
        case.lens_list, case.used = lens, [-(-L // 16) for L in lens]
        d["lens"].copy_(torch.tensor(lens))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        o, _, tol, _ = attention_ref(case, 128 ** -0.5)
        within(out, o, tol, f"lens {lens}")
    assert full == [64, 30]


def test_binding_checks(m):
    """Shapes, types and layouts that do not fit are refused before the library sees a pointer."""
    case = Batch([1], [20], 8, 2, 64, 16, torch.float16)
    d = case.dev(DEV)
    out = torch.empty_like(d["q"])
    ws = m.alloc_attention_workspace(8, 2, 64, device=DEV)
    def call(**k):
        a = dict(d, out=out) | k
        m.moe_attention_paged(a["q"], a["k"], a["v"], a["table"], a["offs"], a["lens"], 1, 0.1, a["out"], ws)
    call()
    with pytest.raises(TypeError):
        call(lens=d["lens"].long())
    with pytest.raises(TypeError):
        call(q=d["q"].float())
    with pytest.raises(ValueError):
        call(out=out[:, :4])
    with pytest.raises(ValueError):
        call(v=d["v"].transpose(1, 2))
    with pytest.raises(ValueError):
        call(k=d["k"].transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(m.MoeError):
        m.moe_attention_paged(d["q"], d["k"], d["v"], d["table"], d["offs"], d["lens"], 1, 0.1, out, ws[:128])
