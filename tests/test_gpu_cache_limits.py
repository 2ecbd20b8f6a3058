"""The calls on the cache in 8 bits and on drafted trees at the edges of what they promise: waits that run
out, what ran before, drawn batches, many sequences, queries that are not finite, windows and sinks past
every length, workspaces of the experts."""
import math

import numpy as np
import pytest

from tests.block_cases import Batch
from tests.cache_cases import Batch8, cache_ref, random_trees, tree_tensor
from tests.test_gpu_attention_half import within
from tests.test_gpu_cache import check_attn, run_attn
from tests.test_gpu_parity import DEV, m  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF16, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("codes", [False, True], ids=["16bit", "codes"])
@pytest.mark.parametrize("new,lens", [([1], [93]), ([1] * 32, [1500] * 32), ([1], [60000]), ([3, 1], [60, 40]),
                                      ([60], [100]), ([300] * 8, [900] * 8), ([900], [2500])])
def test_waits_that_run_out(m, new, lens, codes):
    """CTA 0 waits for an arrival that nobody makes: the call ends by itself, records MOE_ERR_TIMEOUT, and the
    workspace serves again once initialised."""
    kind = Batch8 if codes else Batch
    case = kind(new, lens, 8, 2, 128, 16, BF16, seed=11)
    tree = tree_tensor(random_trees(new), case.N, 29)
    ws = m.alloc_attention_workspace(8, 2, 128, device=DEV)
    try:
        m.moe_debug_set_wait_limit(20_000_000)      # 20 ms
        m.moe_debug_withhold_arrivals(1)
        assert m.status_str(run_attn(m, case, tree=tree, ws=ws)[2]) == "MOE_ERR_TIMEOUT"
    finally:
        m.moe_debug_withhold_arrivals(0)
        m.moe_debug_set_wait_limit(0)
    m.moe_workspace_init(ws)
    out, lse, code, detail = run_attn(m, case, tree=tree, ws=ws)
    assert code == 0, (m.status_str(code), detail)
    o, e, tol, lse_tol = cache_ref(case, 128 ** -0.5, trees=random_trees(new), words=29)
    within(out, o, tol, "out")
    within(lse, e, lse_tol, "lse")


@pytest.mark.parametrize("seed", range(60))
def test_drawn_batches(m, seed):
    """Ragged batches, layouts and masks drawn at random."""
    r = np.random.default_rng(seed)
    Hkv, G, D = int(r.integers(1, 5)), int(r.choice([1, 2, 3, 4, 5, 8, 12, 16, 32])), int(r.choice([64, 128]))
    page, B = int(r.choice([16, 32, 64, 128, 256])), int(r.integers(1, 9))
    top = int(r.choice([1, 1, 4, 40, 300]))
    new = [int(x) for x in r.integers(0, top + 1, B)]
    lens = [max(0, n + int(x)) for n, x in zip(new, r.integers(-3, int(r.choice([20, 400, 3000])), B))]
    kind = Batch8 if r.random() < 0.6 else Batch
    case = kind(new, lens, Hkv * G, Hkv, D, page, F16 if r.random() < 0.5 else BF16, seed=seed,
                spare_rows=int(r.integers(0, 3)))
    trees = random_trees(new, seed=seed, width=int(r.integers(1, 30)), empty=0.1) if r.random() < 0.5 else None
    check_attn(m, case, window=int(r.choice([0, 1, 17, 128, 300, 1000])), sinks=int(r.choice([0, 1, 5, 64, 200])),
               softcap=float(r.choice([0, 0, 3.0, 40.0, 500.0])), trees=trees, fill=-1,
               words=None if trees is None else int(r.integers(max(1, top // 64), 12)),
               scale=float(r.choice([D ** -0.5, D ** -0.5, -0.1, 0.3, 0.0])))


@pytest.mark.parametrize("codes", [False, True], ids=["16bit", "codes"])
@pytest.mark.parametrize("B,most", [(700, 1), (4096, 1), (300, 12)])
def test_many_sequences(m, B, most, codes):
    """More sequences than CTAs, most of them short, some empty."""
    r = np.random.default_rng(B)
    new = [int(x) for x in r.integers(0, most + 1, B)]
    lens = [n + int(x) for n, x in zip(new, r.integers(0, 40, B))]
    kind = Batch8 if codes else Batch
    case = kind(new, lens, 8, 2, 64, 16, BF16, seed=B)
    check_attn(m, case, trees=random_trees(new, seed=B), window=20, sinks=2)


@pytest.mark.parametrize("new,lens", [([1, 1], [300, 1]), ([4, 3], [2, 90]), ([70, 150], [40, 900])])
@pytest.mark.parametrize("window,sinks", [((1 << 30) - 1, 3), (2 ** 31 - 1, 2 ** 31 - 1), (7, 2 ** 31 - 1), (7, 1 << 30)])
def test_windows_and_sinks_past_every_length(m, new, lens, window, sinks):
    """They hide nothing; no index wraps."""
    for kind in (Batch, Batch8):
        case = kind(new, lens, 8, 2, 64, 16, F16, seed=3)
        for trees in (None, random_trees(new)):
            got = check_attn(m, case, window=window, sinks=sinks, trees=trees)
            plain = check_attn(m, case, trees=trees)
            assert float((got[1] - plain[1]).nan_to_num(neginf=0.0).abs().max()) < 1e-4


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_queries_that_are_not_finite(m, new, dtype):
    """An infinite or NaN query row is its own affair: the other rows and heads are as without it."""
    for kind in (Batch, Batch8):
        case = kind([new], [300], 8, 2, 64, 16, dtype, seed=2)
        trees = [1 << i for i in range(new)]
        o, e, tol, lse_tol = cache_ref(case, 0.125, trees=trees, words=2)
        bad = torch.zeros(new, 8, dtype=torch.bool)
        bad[0, 1], bad[new - 1, 6] = True, True
        case.q[0, 1, 5], case.q[new - 1, 6, 0] = math.inf, math.nan
        out, lse, code, _ = run_attn(m, case, tree=tree_tensor(trees, new, 2), scale=0.125)
        assert code == 0
        within(out.cpu()[~bad], o[~bad], tol[~bad], "out")
        within(lse.cpu()[~bad], e[~bad], lse_tol[~bad], "lse")
        assert bool((~lse.cpu()[bad].isfinite()).all()) and bool((~out.cpu()[bad].isfinite()).any(-1).all())


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_queries_of_many_sizes(m, new, dtype):
    """Rows far apart in size, elements of a row far apart, rows of zeros, the type's smallest values."""
    for kind in (Batch, Batch8):
        case = kind([new], [200], 8, 2, 128, 16, dtype, seed=4)
        f = torch.finfo(dtype)
        lo, hi = (-20, 12) if dtype is F16 else (-100, 90)
        for h in range(8):
            case.q[:, h] = (case.q[:, h].float() * 2.0 ** (lo + (hi - lo) * h // 8)).to(dtype)
        case.q[0, 0] = 0
        case.q[0, 1] = f.smallest_normal * f.eps
        case.q[0, 2, ::2] = (case.q[0, 2, ::2].float() * 2.0 ** -24).to(dtype)
        scale = 2.0 ** -12 if dtype is F16 else 2.0 ** -90
        check_attn(m, case, scale=scale, trees=[1 << i for i in range(new)], words=2)


def test_what_ran_before_leaves_no_trace(m):
    """Rows and keys that nobody has take what the call before left in shared memory: the result is the same bit
    for bit whatever that was."""
    for kind, new, G, D, cap in ((Batch8, [700, 300], 3, 128, 0.0), (Batch8, [40, 90], 7, 64, 5.0), (Batch8, [1, 1], 5, 128, 0.0),
                                 (Batch, [70, 30], 12, 128, 0.0), (Batch, [2, 1], 3, 64, 3.0)):
        case = kind(new, [1000, 905], 2 * G, 2, D, 16, BF16, seed=G)
        tree = tree_tensor(random_trees(new), case.N, 30)
        d, ws = case.dev(DEV), m.alloc_attention_workspace(2 * G, 2, D, device=DEV)
        got = []
        for size in (0.0, 30.0, 1000.0):
            for other in (Batch8([700, 600], [2100, 2000], 8, 2, D, 16, BF16, seed=1),
                          Batch([700, 1], [2100, 2000], 8, 2, D, 16, BF16, seed=1)):
                other.q *= size
                run_attn(m, other, ws=ws, tree=tree_tensor(random_trees(other.new), other.N, 30))
            got.append(run_attn(m, case, 500, cap, 7, tree, ws=ws, d=d))
            assert got[-1][2] == 0
        for o, s, _, _ in got[1:]:
            assert torch.equal(o, got[0][0]) and torch.equal(s, got[0][1])


def test_a_workspace_that_the_experts_have_used(m):
    """Where the FFN's tags would be taken for counts of parts, the call records it."""
    from quantized_routed_expert_02_gb300 import synth
    H, E, k, I = 2048, 16, 2, 768
    shape = synth.custom_shape(1, H, E, k, I, cfg_id=17)
    blobs = {n: torch.from_numpy(b).to(DEV) for n, b in synth.expert_blobs(shape, 0).items()}
    ws = torch.empty(max(m.moe_workspace_bytes(1, H, E, k, I), m.moe_attention_workspace_bytes(8, 2, 128)),
                     dtype=torch.uint8, device=DEV)
    m.moe_workspace_init(ws)
    idx, w = torch.empty(1, k, dtype=torch.int32, device=DEV), torch.empty(1, k, device=DEV)
    y = torch.empty(1, H, device=DEV)
    m.moe_layer(torch.randn(1, H, device=DEV), torch.randn(E, H, device=DEV) * 0.02, None, blobs["gate"], blobs["up"],
                blobs["down"], k, I, idx, w, y, ws)
    assert m.moe_read_device_status(ws)[0] == 0
    case = Batch8([1] * 40, [40] * 40, 8, 2, 128, 16, BF16)
    assert m.status_str(run_attn(m, case, ws=ws)[2]) == "MOE_ERR_WORKSPACE"
