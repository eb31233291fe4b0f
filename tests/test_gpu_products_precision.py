"""How much of a sum the 8-bit product keeps, on sums that cancel, and its scales out to the
ends of the range that the header gives."""

import pytest
import torch

import products_device_reference as dev
import products_reference as ref
from precision_optimizer_step_amd import opt8_products as ops

pytestmark = pytest.mark.gpu

E4, E5, BF = torch.float8_e4m3fn, torch.float8_e5m2, torch.bfloat16
ROW, TILE = ops.OPT8_FP8_BLOCK_ROW, ops.OPT8_FP8_BLOCK_TILE


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible AMD GPU")
    torch.cuda.set_device(0)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def quantized(x, kind, block):
    rows, cols = x.shape
    tile = block == TILE
    q = torch.empty(rows, cols, dtype=torch.uint8, device="cuda").view(kind)
    s = torch.empty(ref.ceil128(cols), ref.ceil128(rows) if tile else rows, device="cuda")
    ops.opt8_fp8_quantize(ops.make_fp8_quant(x, q, s, block=block))
    return q, s


def values(rows, cols, loud, g):
    """Normal values, with `loud` one column in a hundred twenty times as large, as activations have."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    if loud:
        x[:, torch.rand(cols, device="cuda", generator=g) < 0.01] *= 20
    return x


@pytest.mark.parametrize("kind", [E4, E5])
@pytest.mark.parametrize("loud", [False, True])
@pytest.mark.parametrize("block_b", [ROW, TILE])
@pytest.mark.parametrize("m,n,k", [(16, 512, 2048), (128, 256, 1024), (128, 128, 4096), (1001, 2560, 512)])
def test_what_is_cut_from_sums_that_cancel(m, n, k, block_b, loud, kind):
    """[A A'] [B -B']^T with A' and B' the columns of A and B in another order inside each block of
    128: zero, but the groups of 8 consecutive k that the instruction adds are others in the second
    half, so what is left is what the two halves cut off (with fp32's rounding of the blocks' sums).

    Bound, in the mean square over all results: a group cuts less than 2^-13 of its largest term from
    each of the 7 others; the signs of what is cut are those of random terms, so squares add:
    7 * 2^-26 * sum over groups of the largest term's square.  Sums of blocks: their number times 2^-24
    of a result's size.  With the 2-norm of all terms for that size, the whole is below 3.3e-4 of
    it (7^(1/2) 2^-13, were each group's largest term all of it): a sixth of bf16's largest rounding."""
    g = gen(m + k + loud)
    a, sa = quantized(values(m, k, loud, g), kind, ROW)
    b, sb = quantized(values(n, k, False, g) * 0.02, E4, block_b)
    order = torch.cat([torch.randperm(128, device="cuda", generator=g) + 128 * i for i in range(k // 128)])
    bytes_a, bytes_b = a.view(torch.uint8), b.view(torch.uint8)
    both_a = torch.cat([bytes_a, bytes_a[:, order]], 1).view(kind)
    both_b = torch.cat([bytes_b, bytes_b[:, order] ^ 0x80], 1).view(E4)
    sa, sb = torch.cat([sa, sa]), torch.cat([sb, sb])
    c = torch.empty(m, n, dtype=BF, device="cuda")
    ops.opt8_fp8_matmul(ops.make_fp8_product(both_a, sa, both_b, sb, c, block_b=block_b))
    torch.cuda.synchronize()
    tops = torch.zeros((), dtype=torch.float64, device="cuda")
    x, y = dev.decode(both_a, sa, False).abs(), dev.decode(both_b, sb, block_b == TILE).abs()
    for at in range(0, 2 * k, 8):
        top = x[:, at, None] * y[None, :, at]
        for j in range(1, 8):
            top = torch.maximum(top, x[:, at + j, None] * y[None, :, at + j])
        tops += (top ** 2).sum()
    size = ((x ** 2) @ (y ** 2).t()).sum()
    cut = (c.double() ** 2).sum() ** 0.5
    blocks = 2 * ref.ceil128(k)
    assert float(cut) <= float((7 * 2.0 ** -26 * tops) ** 0.5 + blocks * 2.0 ** -24 * size ** 0.5) * (1 + ref.half_step(BF))
    assert float(cut) <= 3.3e-4 * float(size ** 0.5)
    assert float(cut) > 0          # something is cut: the sums are not exact


@pytest.mark.parametrize("m", [5, 90])
@pytest.mark.parametrize("block_b", [ROW, TILE])
@pytest.mark.parametrize("ea,eb", [(-126, 0), (0, -126), (-126, 126), (-126, 127), (127, -126), (127, 0), (0, 127), (60, 67),
                                   (-63, -63), (120, -126), (-100, 90), (64, 63)])
def test_scales_whose_product_is_a_normal_number(m, block_b, ea, eb):
    """Powers of two for scales, far out each, whose product is 2^-126 to 2^127; at most one
    nonzero product in each result, so results are exact, and 0 where there is none."""
    g = gen(m)
    n, k = 70, 256
    at = torch.randint(0, k, (m,), device="cuda", generator=g)
    a = torch.zeros(m, k, device="cuda")
    a[torch.arange(m, device="cuda"), at] = 1.0
    b = torch.randint(-1, 2, (n, k), device="cuda", generator=g).float()
    sa = torch.full((2, m), 2.0 ** ea, device="cuda")
    sb = torch.full((2, 1 if block_b == TILE else n), 2.0 ** eb, device="cuda")
    c = torch.empty(m, n, dtype=BF, device="cuda")
    qa, qb = a.to(E4), b.to(E4)
    ops.opt8_fp8_matmul(ops.make_fp8_product(qa, sa, qb, sb, c, block_b=block_b))
    torch.cuda.synchronize()
    assert torch.equal(c.double(), (a.double() @ b.double().t()) * 2.0 ** (ea + eb))
