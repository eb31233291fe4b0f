"""The longest sums of the operators in opt8_layers.h: whole numbers, whose sums are exact in any order,
and values of one sign, whose roundings would add up."""

import pytest
import torch

import layers_reference as lref
from precision_optimizer_step_amd import opt8_layers as ops

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible AMD GPU")
    torch.cuda.set_device(0)


def embedding_gradient(ids, dy, vocab, scale=1.0, old=None):
    """The fp32 gradient of dy, all on the GPU."""
    tokens, d = dy.shape
    out = torch.full((vocab, d), 77.0, device="cuda") if old is None else old
    work = torch.full((ops.opt8_embedding_workspace(tokens, vocab, d),), 255, dtype=torch.uint8, device="cuda")
    ops.opt8_embedding_backward(ops.make_embedding_grad(ids, dy, out, work, scale=scale, accumulate=old is not None))
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("tokens,d", [(1 << 22, 5), (300000, 130), (20000, 1025)])
def test_a_sum_of_one_sign_does_not_drift(tokens, d):
    """One id's tokens with the same dy, as a placeholder's or a small table's can be: at most 31 additions of
    32 bits in a chunk, the rounding of what the chunks give in 64 bits, and scale's."""
    row = 0.1 + torch.arange(d, device="cuda") * 0.37 % 0.8
    got = embedding_gradient(torch.full((tokens,), 2, device="cuda"), row.expand(tokens, d).contiguous(), 4, 0.7)
    scale = float(torch.tensor(0.7, dtype=F32))
    want = row.cpu().double() * tokens * scale
    lref.check("dtable", got[2], want, (31 + 2 + 1e-3) * lref.U * want)
    assert bool((got[[0, 1, 3]] == 0).all())
