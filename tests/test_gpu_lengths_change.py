"""Lengths that change under an attention call (a missing stream order): its warps leave together."""
import pytest

from tests.block_cases import Batch
from tests.cache_cases import Batch8, random_trees, tree_tensor
from tests.test_gpu_cache import check_attn, run_attn
from tests.test_gpu_parity import DEV, m  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("kind", ["chains", "trees", "codes"])
@pytest.mark.parametrize("D", [64, 128])
def test_warps_that_count_their_tiles_differently(m, kind, D):
    """What a changed length does to two warps of a row, by the test hook: the call ends by itself and records it, and the
    workspace serves again."""
    case = (Batch8 if kind == "codes" else Batch)([40] * 400, [50 + i % 90 for i in range(400)], 16, 2, D, 16,
                                                  torch.float16, seed=1)
    trees = random_trees(case.new) if kind == "trees" else None
    tree = None if trees is None else tree_tensor(trees, case.N, 2)
    ws = m.alloc_attention_workspace(16, 2, D, device=DEV)
    try:
        m.moe_debug_set_wait_limit(20_000_000)      # 20 ms
        m.moe_debug_withhold_arrivals(2)
        assert m.status_str(run_attn(m, case, tree=tree, ws=ws)[2]) == "MOE_ERR_CACHE_RANGE"
    finally:
        m.moe_debug_withhold_arrivals(0)
        m.moe_debug_set_wait_limit(0)
    m.moe_workspace_init(ws)
    check_attn(m, case, trees=trees, ws=ws)
