"""The limit of the device-side waits bounds the time that a call with a wait that runs out takes."""
import pytest

from quantized_routed_expert_02_gb300 import synth
from tests.cases import layer_case
from tests.test_gpu_parity import DEV, m, to_dev  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_grouped_gemm_waits_end_by_the_limit(m):
    """The down GEMM waits for rows that the gate/up launch never counts: no wait, neither for those nor
    for what follows from them, lasts longer than the limit (0.3 s, beside which the work is nothing)."""
    s = synth.custom_shape(64, 512, 16, 8, 256, cfg_id=93)
    case = layer_case(s, 0, (0, 31, 63))
    d = to_dev(case)
    ws = m.alloc_workspace(s.T, s.H, s.E, s.k, s.I, device=DEV)

    def call():
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        m.moe_layer(d["x"], d["Wr"], d["bias"], d["gate"], d["up"], d["down"], s.k, s.I, d["idx"], d["w"], d["y"], ws)
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b)

    call()
    try:
        m.moe_debug_set_wait_limit(300_000_000)
        m.moe_debug_withhold_arrivals(1)
        ms = call()
        code, detail = m.moe_read_device_status(ws)
        assert m.status_str(code) == "MOE_ERR_TIMEOUT" and detail in (18, 21), (code, detail)
        assert ms < 310.0, ms
    finally:
        m.moe_debug_withhold_arrivals(0)
        m.moe_debug_set_wait_limit(0)
