"""The attention half at the edges of what its entry points promise: waits that run out."""
import math

import pytest

from tests.block_cases import Batch, attention_ref
from tests.test_gpu_attention_half import run_attn, within
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


@pytest.mark.parametrize("G,D", [(3, 128), (7, 64), (12, 128)])
def test_what_ran_before_leaves_no_trace(m, G, D):
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
        m.moe_attention_paged(d["q"], d["k"], d["v"], d["table"], d["offs"], d["lens"], 1200, D ** -0.5, out, ws,
                              lse=lse)
        assert m.moe_read_device_status(ws)[0] == 0
        got.append((out.clone(), lse.clone()))
    for o, s in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(s, got[0][1])
