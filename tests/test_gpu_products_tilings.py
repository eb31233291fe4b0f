"""Every kernel of the operators at sizes that run it (products_shapes.py, which a CPU test holds
against the library's choice), in every type, with random values and ragged ends."""

import pytest
import torch

import products_device_reference as dev
import products_reference as ref
import products_shapes as shapes
from precision_optimizer_step_amd import opt8_products as ops

pytestmark = pytest.mark.gpu

ACT = {"silu": ops.OPT8_ACT_SILU, "gelu": ops.OPT8_ACT_GELU, "gelu_tanh": ops.OPT8_ACT_GELU_TANH}
BF, HF = torch.bfloat16, torch.float16
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
ROW, TILE = ops.OPT8_FP8_BLOCK_ROW, ops.OPT8_FP8_BLOCK_TILE


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible AMD GPU")
    torch.cuda.set_device(0)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def held(values, dtype, each=8):
    """The values in rows a multiple of 16 bytes apart, NaN behind each row."""
    rows, cols = values.shape
    store = torch.full((rows, -(-cols // each) * each + each), float("nan"), device="cuda").to(dtype)
    store[:, :cols] = values.to(dtype)
    return store[:, :cols]


def outputs(dtype, *sizes):
    """Results with one row and eight columns of 77 behind them."""
    stores = [torch.full((r + 1, c + 8), 77.0, dtype=dtype, device="cuda") for r, c in sizes]
    return stores, [s[:r, :c] for s, (r, c) in zip(stores, sizes)]


def untouched(store, t):
    return bool((store[t.shape[0]:] == 77).all()) and bool((store[:, t.shape[1]:] == 77).all())


def block(rows, d, f, dtype, seed):
    g = gen(seed)
    return [held(torch.randn(r, c, device="cuda", generator=g) * s, dtype)
            for r, c, s in ((rows, d, 1.0), (f, d, d ** -0.5), (f, d, d ** -0.5))]


def check_forward(rows, d, f, dtype, act, save, seed):
    x, wg, wu = block(rows, d, f, dtype, seed)
    stores, (h, g, u) = outputs(dtype, (rows, f), (rows, f), (rows, f))
    ops.opt8_gated_ffn_forward(ops.make_gated_ffn(x, wg, wu, h, g if save else None, u if save else None, act=ACT[act]))
    torch.cuda.synchronize()
    want, err = dev.gated(x, wg, wu, act)
    for name, got, store, w, e in zip(("h", "gate", "up"), (h, g, u), stores, want, err):
        if name != "h" and not save:
            assert bool((store == 77).all())
            continue
        worst = dev.worst(got, w, e, dtype)
        assert worst <= 1.0, f"{name}: error is {worst} times its bound"
        assert untouched(store, got), f"{name}: written outside"


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("at", range(len(shapes.GATED)), ids=lambda i: "x".join(map(str, shapes.GATED[i][0])))
def test_gated_forward_in_every_tiling(at, dtype):
    check_forward(*shapes.GATED[at][0], dtype, list(ACT)[at % 3], True, at)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("at", range(len(shapes.GATED)), ids=lambda i: "x".join(map(str, shapes.GATED[i][0])))
def test_gated_backward_in_every_tiling(at, dtype):
    rows, d, f = shapes.GATED[at][0]
    act = list(ACT)[(at + 1) % 3]
    x, wg, wu = block(rows, d, f, dtype, 100 + at)
    g = gen(200 + at)
    dh, gate, up = (held(torch.randn(rows, f, device="cuda", generator=g), dtype) for _ in range(3))
    stores, outs = outputs(dtype, (rows, d), (f, d), (f, d))
    need = ops.opt8_gated_ffn_workspace(rows, d, f)
    work = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")    # NaN patterns
    ops.opt8_gated_ffn_backward(ops.make_gated_ffn_grad(dh, x, wg, wu, gate, up, *outs, work[:need], act=ACT[act]))
    torch.cuda.synchronize()
    assert bool((work[need:] == 0xFF).all()), "written behind the workspace"
    del work
    want, err = dev.gated_grad(dh, x, wg, wu, gate, up, act, dtype)
    for name, got, store, w, e in zip(("dx", "dw_gate", "dw_up"), outs, stores, want, err):
        worst = dev.worst(got, w, e, dtype)
        assert worst <= 1.0, f"{name}: error is {worst} times its bound"
        assert untouched(store, got), f"{name}: written outside"


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows", [1, 5, 16])
@pytest.mark.parametrize("d", shapes.FEW_GATED_D)
def test_gated_forward_of_few_rows_at_depth(rows, d, dtype):
    for f, act, save in ((100, "silu", True), (77, "gelu", False), (4097, "gelu_tanh", True)):
        check_forward(rows, d, f, dtype, act, save, rows * 10000 + d)


def check_product(m, n, k, kind, block_b, seed):
    g = gen(seed)
    tile = block_b == TILE
    a, b = (held(torch.randn(r, k, device="cuda", generator=g) * 8, t, 16) for r, t in ((m, kind), (n, E4)))
    kb = ref.ceil128(k)
    sa = torch.exp(torch.randn(kb, m, device="cuda", generator=g))
    sb = torch.exp(torch.randn(kb, ref.ceil128(n) if tile else n, device="cuda", generator=g))
    (store,), (c,) = outputs(BF, (m, n))
    ops.opt8_fp8_matmul(ops.make_fp8_product(a, sa, b, sb, c, block_b=block_b))
    torch.cuda.synchronize()
    want, bound = dev.product(a, sa, b, sb, tile)
    worst = dev.worst(c, want, bound, BF)
    assert worst <= 1.0, f"error is {worst} times its bound"
    assert untouched(store, c)


@pytest.mark.parametrize("kind", [E4, E5])
@pytest.mark.parametrize("block_b", [ROW, TILE])
@pytest.mark.parametrize("m", [1, 7, 16])
@pytest.mark.parametrize("k", shapes.FEW_PRODUCT_K)
def test_product_of_few_rows_at_depth(m, k, block_b, kind):
    for n in (16, 129, 1000):
        check_product(m, n, k, kind, block_b, m * 10000 + k)


@pytest.mark.parametrize("kind", [E4, E5])
@pytest.mark.parametrize("block_b", [ROW, TILE])
@pytest.mark.parametrize("at", range(len(shapes.PRODUCTS)), ids=lambda i: "x".join(map(str, shapes.PRODUCTS[i][0])))
def test_product_in_every_tiling(at, block_b, kind):
    check_product(*shapes.PRODUCTS[at][0], kind, block_b, at)
