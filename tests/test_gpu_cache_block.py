"""The example block over the cache in 8 bits, with a window and sinks, and with drafted trees."""
import pytest

from tests.test_gpu_decoder_block import example  # noqa: F401
from tests.test_gpu_parity import m  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_example_runs_on_codes(example, capsys):  # noqa: F811
    example.main(codes=True)
    assert "cached tokens [312, 52]" in capsys.readouterr().out


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_an_accepted_path_is_a_chain(example, dtype, codes):  # noqa: F811
    """A prompt, a drafted tree, its accepted path kept, a token more: the branches of the path's nodes and of
    that token are those of the same tokens taken as a chain.  As for a prompt in chunks each way rounds at most
    eight times to the 16-bit type on the way to the branch; over codes a key or value whose own rounding differs
    by a step of the 16-bit projection moves to another code by at most one, a step of 1/127 of its head's
    largest value, against at most half a step of the type, 2^-9 of each value, before."""
    H = 512
    kw = dict(H=H, Hq=8, Hkv=2, D=64, E=4, k=2, I=256, B=1, max_len=128, dtype=dtype, seed=3, codes=codes, window=60,
              sinks=4)
    x = torch.randn(80, H, generator=torch.Generator().manual_seed(5)).to("cuda")

    def take(block, rows, **more):
        h = x[rows].clone()
        block.step(h, [len(rows)], **more)
        return h - x[rows]

    prompt, path, last = list(range(70)), [70, 72, 74], [75]
    drafted, chain = example.Block(**kw), example.Block(**kw)
    take(drafted, prompt)
    tree = take(drafted, [70, 71, 72, 73, 74], paths=[[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4]])
    drafted.keep([[0, 2, 4]])
    got = torch.cat([tree[[0, 2, 4]], take(drafted, last)])
    take(chain, prompt)
    want = torch.cat([take(chain, path), take(chain, last)])
    drafted.check()
    chain.check()
    assert drafted.lens == chain.lens == [74]
    off = (got - want).norm(dim=1) / want.norm(dim=1)
    bound = 2 * 8 * torch.finfo(dtype).eps / 2 + (1 / 127 if codes else 0)
    assert float(off.max()) <= bound, (off.tolist(), bound)
