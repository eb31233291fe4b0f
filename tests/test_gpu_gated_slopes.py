"""The gated block's slopes at the ends of bfloat16's range, and its gradients against differences
within bounds that wrong gradients do not meet."""

import itertools

import pytest
import torch

import products_reference as ref
from precision_optimizer_step_amd import opt8_products as ops

pytestmark = pytest.mark.gpu

ACT = {"silu": ops.OPT8_ACT_SILU, "gelu": ops.OPT8_ACT_GELU, "gelu_tanh": ops.OPT8_ACT_GELU_TANH}
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible AMD GPU")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("act", list(ACT))
def test_products_of_far_apart_factors(act):
    """dg = dh * slope * up, where two of the three leave fp32's normal numbers together although
    all three do not.  Results of 2^-110 to 2^110 only, so that neither bf16's nor the product's
    own ends matter.  x = 1 makes dw_gate and dw_up the rounded dg and du.

    Error: slopes and values are off by at most |argument| 2^-23 + 2^-20 (the exponential's
    argument is rounded to fp32; exponential and reciprocal by the hardware), the argument below 25;
    three products 2^-24 each, and one rounding to bf16."""
    gates = {"silu": (-24.0, -10.0, 3.0), "gelu": (-7.0, -3.0, 2.0), "gelu_tanh": (-5.5, -3.0, 2.0)}[act]
    exps = (-120, -100, -60, -20, 0, 20, 60, 70, 100, 120)
    rows = [(2.0 ** a * 1.25, g, 2.0 ** b * 1.5) for a, g, b in itertools.product(exps, gates, exps)]
    dh, gate, up = (torch.tensor([r[i] for r in rows], dtype=BF) for i in range(3))
    v, s = ref.act(gate.double(), act)
    want_g, want_u = dh.double() * s * up.double(), dh.double() * v

    def inside(x):
        return (x.abs() > 2.0 ** -110) & (x.abs() < 2.0 ** 110)
    # where dh * slope, or dh * up, leaves fp32
    assert int((((dh.double() * s).abs() < 2.0 ** -140) & inside(want_g)).sum()) >= 2
    assert int((((dh.double() * up.double()).abs() > 2.0 ** 130) & inside(want_g)).sum()) >= 2
    f = dh.numel()
    x = torch.zeros(1, 8, dtype=BF, device="cuda")
    x[:, 0] = 1.0
    w = torch.zeros(f, 8, dtype=BF, device="cuda")
    dwg, dwu = torch.empty_like(w), torch.empty_like(w)
    work = torch.empty(ops.opt8_gated_ffn_workspace(1, 8, f), dtype=torch.uint8, device="cuda")
    store = [torch.zeros(1, -(-f // 8) * 8, dtype=BF, device="cuda")[:, :f] for _ in range(3)]
    for to, src in zip(store, (dh, gate, up)):
        to.copy_(src[None])
    ops.opt8_gated_ffn_backward(ops.make_gated_ffn_grad(store[0], x, w, w.clone(), store[1], store[2], None, dwg, dwu, work,
                                                        act=ACT[act]))
    torch.cuda.synchronize()
    rel = 25 * 2.0 ** -23 + 2.0 ** -20 + 4 * 2.0 ** -24
    for name, got, want in (("dg", dwg, want_g), ("du", dwu, want_u)):
        k = inside(want)
        worst = ref.worst(got[k.cuda(), 0], want[k], ref.rounded(want[k], want[k].abs() * rel, BF))
        assert worst <= 1.0, f"{name}: error is {worst} times its bound"


@pytest.mark.parametrize("act", list(ACT))
def test_no_gradient_stays_none(act):
    """dh = 0 gives dg = du = 0 beside the largest up and gates of either sign."""
    top = torch.finfo(BF).max
    gate = torch.tensor([[-1e30, -20.0, -1.0, 0.0, 1.5, 2.0, 20.0, 1e30]], dtype=BF, device="cuda")
    f = gate.shape[1]
    x = torch.ones(1, 8, dtype=BF, device="cuda")
    w = torch.zeros(f, 8, dtype=BF, device="cuda")
    dwg, dwu = torch.full_like(w, 3.0), torch.full_like(w, 3.0)
    work = torch.empty(ops.opt8_gated_ffn_workspace(1, 8, f), dtype=torch.uint8, device="cuda")
    for up in (top, -top):
        ops.opt8_gated_ffn_backward(ops.make_gated_ffn_grad(torch.zeros_like(gate), x, w, w.clone(), gate,
                                                            torch.full_like(gate, up), None, dwg, dwu, work, act=ACT[act]))
        torch.cuda.synchronize()
        assert bool((dwg == 0).all()) and bool((dwu == 0).all())
