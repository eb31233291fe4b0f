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


def value_64(x, wg, wu, act):
    """h in 64 bits: the activation's value alone, no slope."""
    return ref.act(x @ wg.t(), act)[0] * (x @ wu.t())


def differences(x, wg, wu, c, act, e=1e-4):
    """Central differences of sum(h * c) by every element of x, w_gate and w_up.  An element of x
    moves its own row of h alone and one of a weight its own column, so a column of the input is
    moved at once and h * c summed by rows or by columns."""
    out = []
    for at, src in enumerate((x, wg, wu)):
        grad = torch.empty_like(src)
        for j in range(src.shape[1]):
            sums = []
            for sign in (1, -1):
                args = [x, wg, wu]
                args[at] = src.clone()
                args[at][:, j] += sign * e
                sums.append((value_64(*args, act) * c).sum(1 if at == 0 else 0))
            grad[:, j] = (sums[0] - sums[1]) / (2 * e)
        out.append(grad)
    return out


def difference_bounds(x, wg, wu, c, act):
    """Bounds of the kernels' gradients against the exact ones of sum(h * c).

    The backward pass reads g and u rounded to bf16 (after fp32 sums): half a step and gamma(d) of
    the magnitudes.  It takes act and its slope there; |slope| <= 1.13 and |second derivative| <=
    0.82 (0.5 for silu, 2 phi(0) = 0.798 and a little more for gelu and its tanh form) carry the
    difference over.  dg and du are rounded once to bf16, then summed in fp32 and rounded once.
    The slope comes from differences of the value.  The differences themselves are off by e^2/6 of
    a third derivative (a sum of up to 70 c u act''' x^3, below 300: 5e-7) and by rounding (1e-11)."""
    half = ref.half_step(BF)
    g, u = x @ wg.t(), x @ wu.t()
    n, d = x.shape
    f = wg.shape[0]
    v = ref.act(g, act)[0]
    s = (ref.act(g + 1e-5, act)[0] - ref.act(g - 1e-5, act)[0]) / 2e-5
    X, G, U, C = (t.abs() for t in (x, wg, wu, c))
    eg, eu = ((X @ w.t()) * ref.gamma(d) for w in (G, U))
    eg, eu = eg + half * (g.abs() + eg), eu + half * (u.abs() + eu)
    slope_err, value_err = 0.82 * eg + 2.0 ** -18, 1.13 * eg + 2.0 ** -18
    dg, du = (c * u * s).abs(), (c * v).abs()
    fg = C * (u.abs() * slope_err + eu * (s.abs() + slope_err)) + 2.0 ** -22 * dg
    fu = C * value_err + 2.0 ** -22 * du
    fg, fu = fg + half * (dg + fg), fu + half * (du + fu)
    ag, au = dg + fg, du + fu
    ex = fg @ G + fu @ U + (ag @ G + au @ U) * ref.gamma(2 * f + 128)
    ew = [e.t() @ X + (m.t() @ X) * ref.gamma(n) for e, m in ((fg, ag), (fu, au))]
    return [ref.rounded(t, b, BF) + 1e-6 for t, b in zip(differences(x, wg, wu, c, act), [ex] + ew)]


def inputs(rows, d, f, seed):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(r, k, generator=g) * s).to(BF) for r, k, s in
            ((rows, d, 1.0), (f, d, d ** -0.5), (f, d, d ** -0.5), (rows, f, 1.0))]


@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("rows,d,f", [(40, 48, 56), (9, 72, 33), (70, 17, 24)])
def test_every_gradient_against_differences(act, rows, d, f):
    """Element by element.  The bounds are an eighth of the gradients or less (in the 2-norm, over
    each of the three), so that no gradient, gradients of the other sign, twice the gradient and
    a slope without its second term all leave them, which is checked here on the 64-bit form."""
    x, wg, wu, c = inputs(rows, d, f, 3 * rows + d)
    wide = [t.double() for t in (x, wg, wu, c)]
    want, bound = differences(*wide, act), difference_bounds(*wide, act)
    X, G, U, C = wide
    slope_of_p = ref.act(X @ G.t(), act)[0] / (X @ G.t())           # act(g)/g: the slope without its second term
    for at, (w, b) in enumerate(zip(want, bound)):
        assert float(b.norm()) <= float(w.norm()) / 8
        for wrong in (torch.zeros_like(w), -w, 2 * w):
            assert float(((wrong - w).abs() / b).max()) > 2.0, at
    bare = C * (X @ U.t()) * slope_of_p
    assert float(((bare.t() @ X - want[1]).abs() / bound[1]).max()) > 2.0

    def held(t):
        store = torch.zeros(t.shape[0], -(-t.shape[1] // 8) * 8, dtype=BF, device="cuda")
        store[:, :t.shape[1]] = t.cuda()
        return store[:, :t.shape[1]]
    xs, gs, us, cs = (held(t) for t in (x, wg, wu, c))
    h, gate, up = (held(torch.zeros(rows, f)) for _ in range(3))
    ops.opt8_gated_ffn_forward(ops.make_gated_ffn(xs, gs, us, h, gate, up, act=ACT[act]))
    outs = [torch.empty(*t.shape, dtype=BF, device="cuda") for t in (x, wg, wu)]
    work = torch.empty(ops.opt8_gated_ffn_workspace(rows, d, f), dtype=torch.uint8, device="cuda")
    ops.opt8_gated_ffn_backward(ops.make_gated_ffn_grad(cs, xs, gs, us, gate, up, *outs, work, act=ACT[act]))
    torch.cuda.synchronize()
    for name, got, w, b in zip(("dx", "dw_gate", "dw_up"), outs, want, bound):
        worst = ref.worst(got, w, b)
        assert worst <= 1.0, f"{name}: error is {worst} times its bound"
