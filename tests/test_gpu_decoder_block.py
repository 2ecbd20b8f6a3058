"""The example block: prompts in chunks and single tokens give what one call for the whole gives."""
import importlib.util
import os

import pytest

from tests.test_gpu_parity import m  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(m):  # noqa: F811
    spec = importlib.util.spec_from_file_location("decoder_block", os.path.join(ROOT, "examples", "decoder_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_example_runs(example, capsys):
    example.main()
    assert "cached tokens [308, 48]" in capsys.readouterr().out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_chunks_give_what_the_whole_gives(example, dtype):
    """The residual stream after the attention half of a prompt taken whole, in two chunks and token
    by token.  Each way rounds at most eight times to the 16-bit type on the way to the branch (norm,
    projection, rotation, scores' operands, weights, output, projection) and cancels nothing, so
    the branches agree to 2 * 8 half steps of their norm."""
    def take(pieces):
        block = example.Block(H=512, Hq=8, Hkv=2, D=64, E=4, k=2, I=256, B=1, max_len=128, dtype=dtype, seed=3)
        x = torch.randn(96, 512, generator=torch.Generator().manual_seed(5)).to("cuda")
        rows, at = [], 0
        for n in pieces:
            h = x[at:at + n].clone()
            block.step(h, [n])  # h is the residual stream after the attention half
            rows.append(h - x[at:at + n])
            at += n
        block.check()
        return torch.cat(rows)
    whole = take([96])
    bound = 2 * 8 * torch.finfo(dtype).eps / 2
    for pieces in ([50, 46], [90] + [1] * 6, [1] * 96):
        got = take(pieces)
        off = (got - whole).norm(dim=1) / whole.norm(dim=1)
        assert float(off.max()) <= bound, (pieces[:2], float(off.max()), bound)
