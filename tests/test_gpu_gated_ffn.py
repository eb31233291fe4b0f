"""Gated feed-forward block, forward and backward, against 64-bit forms and differences,
and one training step through it, the 8-bit products and the optimizer."""

import numpy as np
import pytest
import torch

import products_reference as ref
from precision_optimizer_step_amd import opt8, opt8_products as ops

pytestmark = pytest.mark.gpu

ACT = {"silu": ops.OPT8_ACT_SILU, "gelu": ops.OPT8_ACT_GELU, "gelu_tanh": ops.OPT8_ACT_GELU_TANH}
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible AMD GPU")
    torch.cuda.set_device(0)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def room(rows, cols, dtype, extra=0, fill=77.0):
    """[rows, cols] with rows a multiple of 8 elements (plus extra) apart and one row behind."""
    store = torch.full((rows + 1, -(-cols // 8) * 8 + extra), fill, dtype=dtype, device="cuda")
    return store, store[:rows, :cols]


def untouched(store, rows, cols, fill=77.0):
    return bool((store[rows] == fill).all()) and bool((store[:, cols:] == fill).all())


def inputs(rows, d, f, dtype, seed, extra=0):
    g = gen(seed)
    out = []
    for r, c, s in ((rows, d, 1.0), (f, d, d ** -0.5), (f, d, d ** -0.5)):
        _, t = room(r, c, dtype, extra, fill=float("nan"))   # what lies behind a row is never used
        t.copy_((torch.randn(r, c, generator=g) * s).to(dtype))
        out.append(t)
    return out


# The fast exponential and reciprocal: 2^-20 of the activation's value or slope; gelu's erfc, 2^-20 too.
ACT_ERR = 2.0 ** -20


def forward_reference(x, wg, wu, act):
    """h, g, u in 64 bits and bounds of their fp32 forms: the sums' own, carried through act
    (whose slope is at most 1.13 in magnitude)."""
    X, G, U = (t.double().cpu() for t in (x, wg, wu))
    g, u = X @ G.t(), X @ U.t()
    eg, eu = (X.abs() @ G.abs().t()) * ref.gamma(x.shape[1]), (X.abs() @ U.abs().t()) * ref.gamma(x.shape[1])
    v, _ = ref.act(g, act)
    ev = 1.13 * eg + ACT_ERR * (v.abs() + 2.0 ** -20 * g.abs())
    eh = ev * (u.abs() + eu) + v.abs() * eu + 2.0 ** -24 * (v * u).abs()
    return (v * u, g, u), (eh, eg, eu)


def check_forward(rows, d, f, dtype=BF, act="silu", save=True, seed=0, extra=0):
    x, wg, wu = inputs(rows, d, f, dtype, seed, extra)
    hs, h = room(rows, f, dtype, extra)
    gs, g = room(rows, f, dtype, extra)
    us, u = room(rows, f, dtype, extra)
    ops.opt8_gated_ffn_forward(ops.make_gated_ffn(x, wg, wu, h, g if save else None, u if save else None, act=ACT[act]))
    torch.cuda.synchronize()
    want, err = forward_reference(x, wg, wu, act)
    for name, got, store, w, e in zip(("h", "gate", "up"), (h, g, u), (hs, gs, us), want, err):
        if name != "h" and not save:
            assert bool((store == 77).all())
            continue
        worst = ref.worst(got, w, ref.rounded(w, e, dtype))
        assert worst <= 1.0, f"{name}: error is {worst} times its bound"
        assert untouched(store, rows, f), f"{name}: written outside"
    return h


@pytest.mark.parametrize("rows", [1, 2, 16, 17, 33, 64, 65, 129, 300])
@pytest.mark.parametrize("f", [1, 16, 72, 130])
def test_forward_rows_and_width(rows, f):
    check_forward(rows, 256, f, seed=rows * 100 + f)


@pytest.mark.parametrize("d", [1, 7, 8, 9, 31, 32, 63, 64, 65, 100, 128, 500])
@pytest.mark.parametrize("rows", [3, 90])
def test_forward_depths(rows, d):
    check_forward(rows, d, 100, seed=d, extra=8)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("save", [True, False])
@pytest.mark.parametrize("rows,f", [(5, 200), (100, 200), (2050, 3360)])
def test_forward_types_and_activations(dtype, act, save, rows, f):
    """(2050 rows and 3360 columns take the largest tiles.)"""
    check_forward(rows, 192, f, dtype, act, save, seed=3)


def test_activations_far_from_zero():
    """g from -60 to 60, and beyond where the exponential overflows: no NaN, the limits exact."""
    for act in ACT:
        vals = torch.cat([torch.linspace(-60, 60, 241), torch.tensor([-3e4, -200.0, 200.0, 3e4])]).to(BF)
        f = vals.numel()
        for rows in (1, 80):
            x = torch.zeros(rows, 8, dtype=BF, device="cuda")
            x[:, 0] = 1.0
            wg = torch.zeros(f, 8, dtype=BF, device="cuda")
            wg[:, 0] = vals.cuda()
            wu = torch.zeros(f, 8, dtype=BF, device="cuda")
            wu[:, 0] = 1.0
            h = torch.empty(rows, f, dtype=BF, device="cuda")
            ops.opt8_gated_ffn_forward(ops.make_gated_ffn(x, wg, wu, h, act=ACT[act]))
            torch.cuda.synchronize()
            g = vals.double()
            v, _ = ref.act(g, act)
            # sigmoid and erfc by fp32: 2^-20 relative of the value down to where fp32's exponential
            # leaves the normal numbers (2^-126); the argument's own rounding (x log2 e, y of the
            # tanh form: |y| 2^-22 absolute in the exponent) adds |arg| 2^-21
            arg = g.abs() + (g * g if act != "silu" else 0) + (0.08 * g.abs() ** 3 if act == "gelu_tanh" else 0)
            err = v.abs() * (2.0 ** -18 + arg.clamp_max(200.0) * 2.0 ** -20) + g.abs() * 2.0 ** -125
            for r in range(rows):
                assert ref.worst(h[r], v, ref.rounded(v, err, BF)) <= 1.0


def grad_reference(dh, x, wg, wu, g, u, act, dtype):
    """64-bit gradients and the bounds of their fp32 forms from dg, du rounded once to `dtype`."""
    H, X, G, U, g, u = (t.double().cpu() for t in (dh, x, wg, wu, g, u))
    v, s = ref.act(g, act)
    dg, du = H * u * s, H * v
    # fp32 dg, du: the activation's error (absolute 2^-20 of 1.13 for a slope near its zero) and two
    # products; then half a step of the type
    fg = (H * u).abs() * (2.0 ** -18) + 4 * 2.0 ** -24 * dg.abs()
    fu = H.abs() * (v.abs() * 2.0 ** -18 + g.abs() * 2.0 ** -30) + 4 * 2.0 ** -24 * du.abs()
    eg, eu = ref.rounded(dg, fg, dtype), ref.rounded(du, fu, dtype)
    n, f = H.shape
    ag, au = dg.abs() + eg, du.abs() + eu
    dx = dg @ G + du @ U
    ex = eg @ G.abs() + eu @ U.abs() + (ag @ G.abs() + au @ U.abs()) * ref.gamma(2 * f + 128)
    dwg, dwu = dg.t() @ X, du.t() @ X
    ewg = eg.t() @ X.abs() + (ag.t() @ X.abs()) * ref.gamma(n)
    ewu = eu.t() @ X.abs() + (au.t() @ X.abs()) * ref.gamma(n)
    return (dx, dwg, dwu), (ex, ewg, ewu)


def check_backward(rows, d, f, dtype=BF, act="silu", dx=True, dw=True, seed=0, extra=0):
    x, wg, wu = inputs(rows, d, f, dtype, seed, extra)
    g = gen(seed + 1)
    saved = []
    for _ in range(3):
        _, t = room(rows, f, dtype, extra, fill=float("nan"))
        t.copy_(torch.randn(rows, f, generator=g).to(dtype))
        saved.append(t)
    dh, gate, up = saved
    sx, ox = room(rows, d, dtype, extra)
    sg, og = room(f, d, dtype, extra)
    su, ou = room(f, d, dtype, extra)
    need = ops.opt8_gated_ffn_workspace(rows, d, f)
    work = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")    # NaN patterns
    ops.opt8_gated_ffn_backward(ops.make_gated_ffn_grad(dh, x, wg, wu, gate, up, ox if dx else None, og if dw else None,
                                                        ou if dw else None, work[:need], act=ACT[act]))
    torch.cuda.synchronize()
    want, err = grad_reference(dh, x, wg, wu, gate, up, act, dtype)
    for name, got, store, w, e, on, r in zip(("dx", "dw_gate", "dw_up"), (ox, og, ou), (sx, sg, su), want, err,
                                             (dx, dw, dw), (rows, f, f)):
        if not on:
            assert bool((store == 77).all())
            continue
        worst = ref.worst(got, w, ref.rounded(w, e, dtype))
        assert worst <= 1.0, f"{name}: error is {worst} times its bound"
        assert untouched(store, r, d), f"{name}: written outside"
    assert bool((work[need:] == 0xFF).all()), "written behind the workspace"
    return ox, og, ou


@pytest.mark.parametrize("rows", [1, 2, 63, 64, 65, 128, 200])
@pytest.mark.parametrize("d,f", [(8, 8), (100, 72), (200, 130), (129, 257)])
def test_backward_sizes(rows, d, f):
    check_backward(rows, d, f, seed=rows + d)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("act", list(ACT))
def test_backward_types_and_activations(dtype, act):
    check_backward(150, 96, 160, dtype, act, seed=4, extra=8)


@pytest.mark.parametrize("act", list(ACT))
def test_slopes_of_gates_whose_square_overflows(act):
    """bf16 reaches past the square root of fp32's largest number: the slope is 0 or 1 there, and
    a slope of 0 keeps dg at 0 where dh * u alone would overflow."""
    far = [-3e38, -1e30, -1e20, -1e19, -1e15, -1e4, 1e4, 1e15, 1e19, 1e20, 1e30, 3e38]
    gates = torch.tensor([far + [-1e4] * 4], dtype=BF)
    ones = torch.ones_like(gates)
    big = ones.clone()
    big[:, 12:] = 1e20
    f = gates.shape[1]
    x = torch.zeros(1, 8, dtype=BF, device="cuda")
    x[:, 0] = 1.0
    w = torch.zeros(f, 8, dtype=BF, device="cuda")
    dwg, dwu = torch.empty_like(w), torch.empty_like(w)
    work = torch.empty(ops.opt8_gated_ffn_workspace(1, 8, f), dtype=torch.uint8, device="cuda")
    ops.opt8_gated_ffn_backward(ops.make_gated_ffn_grad(big.cuda(), x, w, w.clone(), gates.cuda(), big.cuda(), None, dwg, dwu,
                                                        work, act=ACT[act]))
    torch.cuda.synchronize()
    v, s = ref.act(gates.double(), act)
    # slopes of exactly 0 or 1 and values of exactly 0 or g: every product is exact
    assert torch.equal(dwg[:, 0].double().cpu(), s[0])
    assert torch.equal(dwu[:, 0].double().cpu(), v[0])


@pytest.mark.parametrize("dx,dw", [(True, False), (False, True)])
def test_backward_of_one_side(dx, dw):
    check_backward(90, 64, 100, dx=dx, dw=dw, seed=5)


@pytest.mark.parametrize("rows,d,f", [(4100, 3200, 192), (300, 2600, 2700)])
def test_backward_largest_tiles(rows, d, f):
    """Enough tiles of dx, or of the weights' gradients, for the largest tile."""
    check_backward(rows, d, f, seed=6)


@pytest.mark.parametrize("rows,f", [(17, 4000), (130, 4100), (500, 4104), (1500, 4104), (2050, 4104)])
def test_forward_every_tile_size(rows, f):
    """64 x 64 tiles with four teams of waves and with two, 128 x 128 with two and with one, and
    256 x 256, at depths that give the teams different numbers of steps, and none to some."""
    for d in (60, 129, 320):
        check_forward(rows, d, f, seed=d)


@pytest.mark.parametrize("rows,d,f", [(1, 128, 4096), (64, 130, 4096), (70, 1000, 2080), (500, 1024, 1100), (17, 9, 3000)])
def test_backward_with_a_long_sum_for_dx(rows, d, f):
    """dx from several parts of its contraction (2f), some shorter than others."""
    assert ops.opt8_gated_ffn_workspace(rows, d, f) > rows * 4 * (-(-f // 64) * 64)
    check_backward(rows, d, f, seed=rows)


@pytest.mark.parametrize("rows,d,f", [(600, 2100, 700), (1100, 2100, 500), (1, 700, 300), (3000, 130, 260)])
def test_backward_every_tile_size(rows, d, f):
    check_backward(rows, d, f, seed=8)


def test_backward_of_no_rows_clears_the_weights_gradients():
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    w = torch.randn(96, 64, generator=gen(0)).to(BF).cuda()
    n = torch.empty(0, 96, dtype=BF, device="cuda")
    a, b = torch.full_like(w, 5.0), torch.full_like(w, 5.0)
    ops.opt8_gated_ffn_backward(ops.make_gated_ffn_grad(n, e, w, w, n, n, e.clone(), a, b,
                                                        torch.empty(0, dtype=torch.uint8, device="cuda")))
    ops.opt8_gated_ffn_forward(ops.make_gated_ffn(e, w, w, n.clone()))
    ops.opt8_gated_ffn_backward(ops.make_gated_ffn_grad(n, e, w, w, n, n, e.clone(), None, None,
                                                        torch.empty(0, dtype=torch.uint8, device="cuda")))
    ops.opt8_gated_ffn_forward(ops.make_gated_ffn(e, w, w, n.clone(), n.clone(), n.clone()))
    torch.cuda.synchronize()
    assert bool((a == 0).all()) and bool((b == 0).all())


@pytest.mark.parametrize("act", list(ACT))
def test_gradients_against_differences(act):
    """The kernels' gradients of sum(h * c) against central differences of the 64-bit form,
    along random directions of x and of both weights.  The gradients carry the rounding of g,
    u, dg, du and of themselves: five half steps of bf16 relative to sum|terms|."""
    rows, d, f = 40, 48, 56
    x, wg, wu = inputs(rows, d, f, BF, 9)
    c = torch.randn(rows, f, generator=gen(10)).to(BF).cuda()
    h, g, u = (torch.empty(rows, f, dtype=BF, device="cuda") for _ in range(3))
    ops.opt8_gated_ffn_forward(ops.make_gated_ffn(x, wg, wu, h, g, u, act=ACT[act]))
    dx, dg, du = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    work = torch.empty(ops.opt8_gated_ffn_workspace(rows, d, f), dtype=torch.uint8, device="cuda")
    ops.opt8_gated_ffn_backward(ops.make_gated_ffn_grad(c, x, wg, wu, g, u, dx, dg, du, work, act=ACT[act]))
    torch.cuda.synchronize()
    X, G, U, C = (t.double().cpu() for t in (x, wg, wu, c))

    def value(X, G, U):
        return float((ref.act(X @ G.t(), act)[0] * (X @ U.t()) * C).sum())
    for at, (grad, src) in enumerate(((dx, X), (dg, G), (du, U))):
        v = torch.randn(src.shape, generator=gen(20 + at), dtype=torch.float64)
        e = 1e-5
        args = [X, G, U]
        args[at] = src + e * v
        hi = value(*args)
        args[at] = src - e * v
        diff = (hi - value(*args)) / (2 * e)
        got = grad.double().cpu()
        # |dg| and |du| terms behind each gradient, all magnitudes: a bound on what half steps act on
        A = [t.abs() for t in (X, G, U, C)]
        gg, uu = X @ G.t(), X @ U.t()
        val, slope = ref.act(gg, act)
        tg, tu = A[3] * uu.abs() * (slope.abs() + 1.0 * gg.abs()), A[3] * (val.abs() + 1.13 * gg.abs())
        mags = (tg @ A[1] + tu @ A[2], tg.t() @ A[0], tu.t() @ A[0])[at]
        assert abs(float((got * v).sum()) - diff) <= 5 * ref.half_step(BF) * float((mags * v.abs()).sum())


def test_other_stream_and_graph():
    rows, d, f = 130, 128, 200
    x, wg, wu = inputs(rows, d, f, BF, 11)
    h, g, u, dh = (torch.empty(rows, f, dtype=BF, device="cuda") for _ in range(4))
    dh.copy_(torch.randn(rows, f, generator=gen(1)))
    dx, dg, du = torch.empty(rows, d, dtype=BF, device="cuda"), torch.empty_like(wg), torch.empty_like(wu)
    work = torch.empty(ops.opt8_gated_ffn_workspace(rows, d, f), dtype=torch.uint8, device="cuda")
    a = ops.make_gated_ffn(x, wg, wu, h, g, u)
    b = ops.make_gated_ffn_grad(dh, x, wg, wu, g, u, dx, dg, du, work)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ops.opt8_gated_ffn_forward(a, stream=side)
    ops.opt8_gated_ffn_backward(b, stream=side)
    side.synchronize()
    outs = (h, g, u, dx, dg, du)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.opt8_gated_ffn_forward(a)
        ops.opt8_gated_ffn_backward(b)
    for k in range(3):
        x.copy_(torch.randn(rows, d, generator=gen(40 + k)))
        for t in outs:
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in outs]
        for t in outs:
            t.fill_(6.0)
        ops.opt8_gated_ffn_forward(a)
        ops.opt8_gated_ffn_backward(b)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(first, outs))


def test_training_step_through_every_operator():
    """x -> gated block -> h in 8 bits -> product with w_down -> loss gradient dy -> 8-bit
    gradients of w_down and h -> gated backward -> AdamW on the three weights.  The gradients
    are compared with the same chain in 64 bits; the optimizer's result with the step the
    oracle takes on these gradients."""
    import oracle
    rows, d, f = 137, 128, 256
    x, wg, wu = inputs(rows, d, f, BF, 50)
    x, wg, wu = x.contiguous(), wg.contiguous(), wu.contiguous()
    wd = (torch.randn(d, f, generator=gen(51)) * f ** -0.5).to(BF).cuda()
    dy = torch.randn(rows, d, generator=gen(52)).to(BF).cuda()
    E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
    TILE, ROW = ops.OPT8_FP8_BLOCK_TILE, ops.OPT8_FP8_BLOCK_ROW

    def quantized(t, kind, block):
        r, c = t.shape
        tile = block == TILE
        q = torch.empty(r, -(-c // 16) * 16, dtype=kind, device="cuda")[:, :c]
        qt = torch.empty(c, -(-r // 16) * 16, dtype=kind, device="cuda")[:, :r]
        s = torch.empty(ref.ceil128(c), ref.ceil128(r) if tile else r, device="cuda")
        st = torch.empty(ref.ceil128(r), ref.ceil128(c) if tile else c, device="cuda")
        ops.opt8_fp8_quantize(ops.make_fp8_quant(t, q, s, qt, st, block=block))
        return q, s, qt, st
    h, g, u = (torch.empty(rows, f, dtype=BF, device="cuda") for _ in range(3))
    ops.opt8_gated_ffn_forward(ops.make_gated_ffn(x, wg, wu, h, g, u))
    qh, sh, qht, sht = quantized(h, E4, ROW)
    qd, sd, qdt, sdt = quantized(wd, E4, TILE)
    y = torch.empty(rows, d, dtype=BF, device="cuda")
    ops.opt8_fp8_matmul(ops.make_fp8_product(qh, sh, qd, sd, y))
    qy, sy, qyt, syt = quantized(dy, E5, ROW)
    dh, dwd = torch.empty_like(h), torch.empty_like(wd)
    ops.opt8_fp8_matmul(ops.make_fp8_product(qy, sy, qdt, sdt, dh))
    ops.opt8_fp8_matmul(ops.make_fp8_product(qyt, syt, qht, sht, dwd, block_b=ROW))
    dx, dg, du = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    work = torch.empty(ops.opt8_gated_ffn_workspace(rows, d, f), dtype=torch.uint8, device="cuda")
    ops.opt8_gated_ffn_backward(ops.make_gated_ffn_grad(dh, x, wg, wu, g, u, dx, dg, du, work))
    opt8.opt8_init_codebooks()
    descs, before, states = [], [], []
    for i, (p, gr) in enumerate(((wg, dg), (wu, du), (wd, dwd))):
        n = p.numel()
        nb = -(-n // 2048)
        m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
        m.fill_(127)
        am, av = (torch.zeros(nb, device="cuda") for _ in range(2))
        before.append(p.view(torch.int16).cpu().numpy().view(np.uint16).reshape(-1).copy())
        states.append((m, v, am, av))
        descs.append(opt8.make_tensor(p.view(-1), gr.view(-1), m, v, am, av, tensor_id=i))
    opt8.opt8_adamw_step(descs, opt8.make_hparams(1e-3, weight_decay=0.01, step=1, seed=3))
    torch.cuda.synchronize()

    # 64 bits, no rounding in between; e4m3 half step 2^-4, e5m2 2^-3 relative, random signs: the
    # relative 2-norm error of a product of two rounded factors stays below the sum of half steps
    X, D, DY = x.double().cpu(), wd_of(before[2], d, f), dy.double().cpu()
    G0, U0 = (wd_of(b, f, d) for b in before[:2])
    val, slope = ref.act(X @ G0.t(), "silu")
    H = val * (X @ U0.t())
    DH = DY @ D
    DG, DU = DH * (X @ U0.t()) * slope, DH * val
    for got, want in ((y, H @ D.t()), (dh, DH), (dwd, DY.t() @ H), (dx, DG @ G0 + DU @ U0), (dg, DG.t() @ X), (du, DU.t() @ X)):
        rel = float((got.double().cpu() - want).norm() / want.norm())
        assert rel <= 2.0 ** -3 + 2.0 ** -4, rel
    hp = oracle.Hparams(lr=1e-3, weight_decay=0.01, step=1, seed=3)
    for i, (p, gr) in enumerate(((wg, dg), (wu, du), (wd, dwd))):
        n = p.numel()
        bits = gr.view(torch.int16).cpu().numpy().view(np.uint16).reshape(-1)
        nb = -(-n // 2048)
        want = oracle.step_tensor(oracle.MODE_8BIT, before[i], bits, np.full(n, 127, np.uint8), np.zeros(n, np.uint8),
                                  np.zeros(nb, np.float32), np.zeros(nb, np.float32), hp, tensor_id=i)
        assert np.array_equal(p.view(torch.int16).cpu().numpy().view(np.uint16).reshape(-1), want[0])


def wd_of(bits, rows, cols):
    return torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16).double().view(rows, cols)


def test_projections_as_halves_of_one_matrix():
    """gate and up side by side in one [rows, 2f] matrix, forward and back; both weights in one [2f, d]."""
    rows, d, f = 150, 64, 104
    x, _, _ = inputs(rows, d, f, BF, 60)
    w = (torch.randn(2 * f, d, generator=gen(61)) * d ** -0.5).to(BF).cuda()
    both = torch.zeros(rows, 2 * f, dtype=BF, device="cuda")
    h, g, u = (torch.empty(rows, f, dtype=BF, device="cuda") for _ in range(3))
    ops.opt8_gated_ffn_forward(ops.make_gated_ffn(x, w[:f], w[f:], h, both[:, :f], both[:, f:]))
    h2 = torch.empty_like(h)
    ops.opt8_gated_ffn_forward(ops.make_gated_ffn(x, w[:f].clone(), w[f:].clone(), h2, g, u))
    torch.cuda.synchronize()
    assert torch.equal(h, h2) and torch.equal(both[:, :f], g) and torch.equal(both[:, f:], u)
    work = torch.empty(ops.opt8_gated_ffn_workspace(rows, d, f), dtype=torch.uint8, device="cuda")
    res = []
    for gate, up in ((both[:, :f], both[:, f:]), (g, u)):
        dx, dw = torch.empty(rows, d, dtype=BF, device="cuda"), torch.empty(2 * f, d, dtype=BF, device="cuda")
        ops.opt8_gated_ffn_backward(ops.make_gated_ffn_grad(h, x, w[:f], w[f:], gate, up, dx, dw[:f], dw[f:], work))
        torch.cuda.synchronize()
        res.append((dx, dw))
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_offsets_past_32_bits():
    """Projections, their gradients and the workspace of over 2^31 elements."""
    rows, d, f = 140003, 64, 16400
    x, wg, wu = inputs(rows, d, f, BF, 70)
    x, wg, wu = x.contiguous(), wg.contiguous(), wu.contiguous()
    h, g, u = (torch.empty(rows, f, dtype=BF, device="cuda") for _ in range(3))
    ops.opt8_gated_ffn_forward(ops.make_gated_ffn(x, wg, wu, h, g, u))
    torch.cuda.synchronize()
    for r in (slice(0, 30), slice(rows - 30, rows)):
        want, err = forward_reference(x[r], wg, wu, "silu")
        for got, w, e in zip((h, g, u), want, err):
            assert ref.worst(got[r], w, ref.rounded(w, e, BF)) <= 1.0
    # gradients: dh nonzero in the first and last rows only, so that 64-bit sums stay short
    h.zero_()
    for r in (slice(0, 30), slice(rows - 30, rows)):
        h[r] = torch.randn(30, f, generator=gen(71)).to(BF)
    dx, dg, du = torch.empty(rows, d, dtype=BF, device="cuda"), torch.empty_like(wg), torch.empty_like(wu)
    work = torch.empty(ops.opt8_gated_ffn_workspace(rows, d, f), dtype=torch.uint8, device="cuda")
    ops.opt8_gated_ffn_backward(ops.make_gated_ffn_grad(h, x, wg, wu, g, u, dx, dg, du, work))
    torch.cuda.synchronize()
    keep = torch.cat([torch.arange(30), torch.arange(rows - 30, rows)]).cuda()
    want, err = grad_reference(h[keep], x[keep], wg, wu, g[keep], u[keep], "silu", BF)
    assert ref.worst(dx[keep], want[0], ref.rounded(want[0], err[0], BF)) <= 1.0
    assert bool((dx[30:rows - 30] == 0).all())
    for got, w, e in ((dg, want[1], err[1]), (du, want[2], err[2])):
        assert ref.worst(got, w, ref.rounded(w, e, BF)) <= 1.0
