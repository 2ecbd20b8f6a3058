"""Scales of 8-bit codes: of either zero."""
import pytest

from tests.cache_cases import Batch8
from tests.test_gpu_cache import check_attn
from tests.test_gpu_parity import m  # noqa: F401

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
