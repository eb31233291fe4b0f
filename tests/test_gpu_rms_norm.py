"""RMS norm with residual and 8-bit codes, and its backward pass, against 64-bit forms and differences."""

import pytest
import torch

import layers_reference as lref
import products_reference as ref
from precision_optimizer_step_amd import opt8_layers as ops

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
EPS = float(torch.tensor(1e-6, dtype=F32))


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible AMD GPU")
    torch.cuda.set_device(0)


def values(rows, cols, dtype, g, extra=0, head=0, scale=1.0):
    _, t = lref.room(rows, cols, dtype, extra, fill=float("nan"), head=head)   # what lies between rows is never used
    t.copy_((torch.randn(rows, cols, generator=g) * scale).to(dtype))
    return t


def code_room(rows, d, kind, extra=0):
    store = torch.full((rows + 1, -(-d // 16) * 16 + extra), 99, dtype=torch.uint8, device="cuda")
    return store, store.view(kind)[:rows, :d]


# every width that a kernel ends at, and one past it
WIDTHS = [1, 7, 128, 129, 512, 513, 1024, 1025, 2048, 2051, 4096, 4100, 8192, 8200, 16384, 16391, 40000]


def forward(rows, d, dtype, wtype=None, residual=True, kind=E4, extra=0, head=0, seed=0, in_place=None):
    g = torch.Generator().manual_seed(seed)
    x, w = values(rows, d, dtype, g, extra, head), (1 + 0.2 * torch.randn(d, generator=g)).to(wtype or dtype).cuda()
    r = values(rows, d, dtype, g, extra, head, scale=2.0) if residual else None
    ys, y = lref.room(rows, d, dtype, extra, head=head)
    ss, s = lref.room(rows, d, dtype, extra, head=head)
    qs, q = code_room(rows, d, kind, 16 if extra else 0)
    scale, rstd = torch.empty(ref.ceil128(d), rows, device="cuda"), torch.empty(rows, device="cuda")
    want = lref.norm(x.cpu(), w.cpu(), EPS, r.cpu() if residual else None)
    if in_place is not None:
        s = x if in_place == "x" else r
    ops.opt8_rms_norm_forward(ops.make_rms_norm(x, w, y=y, q=q, scale=scale, rstd=rstd, residual=r, sum=s if residual else None, eps=EPS))
    torch.cuda.synchronize()
    if residual:
        lref.check("sum", s, *want["sum"])
    lref.check("y", y, *want["n"])
    lref.check("rstd", rstd, *want["rstd"])
    assert lref.untouched(ys, y) and (in_place or not residual or lref.untouched(ss, s))
    codes = qs.cpu()
    assert bool((codes[:, d:] == 99).all()) and bool((codes[rows] == 99).all())
    if dtype == F32:
        # y holds what was encoded: the same codes and scales, bit for bit
        c, sc = ref.quantize(y, kind, False)
        assert torch.equal(sc, scale.cpu()) and torch.equal(c, codes[:rows, :d])
    else:
        n, err = want["n"]
        top = torch.zeros(ref.ceil128(d), rows, dtype=torch.float64)
        for b in range(ref.ceil128(d)):
            top[b] = n[:, 128 * b:128 * b + 128].abs().amax(1)
        ws = (top / ref.FMAX[kind]).clamp_min(2.0 ** -126)
        rel = (err / n.abs().clamp_min(1e-300)).max()
        lref.check("scale", scale, ws, (rel + 2 * lref.U) * ws, F32)
        got, by = ref.decode(q.view(torch.uint8).cpu().view(kind), scale, False), scale.cpu().double()[torch.arange(d) // 128].t()
        small = torch.finfo(kind).smallest_normal * torch.finfo(kind).eps
        # half a step of the code or of the smallest codes; n's own error, 1/scale and the product with it
        bound = ref.half_step(kind) * n.abs() + small / 2 * by + (err + 3 * lref.U * n.abs()) * (1 + ref.half_step(kind))
        assert bool(((got - n).abs() <= bound * (1 + 1e-6)).all())


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype,wtype", [(BF, BF), (HF, F32), (F32, F32)])
def test_forward(d, dtype, wtype):
    rows = 37 if d <= 4100 else 5
    forward(rows, d, dtype, wtype)
    forward(rows, d, dtype, wtype, residual=False, kind=E5, extra=3, head=1, seed=1)


@pytest.mark.parametrize("rows,d", [(1, 4096), (1, 20000), (300, 128), (1111, 64), (9, 4096)])
@pytest.mark.parametrize("where", ["x", "residual"])
def test_sum_in_an_operand_s_place(rows, d, where):
    forward(rows, d, BF, in_place=where)


@pytest.mark.parametrize("outputs", [("y",), ("rstd",), ("sum",), ("q", "scale"), ("sum", "rstd")])
@pytest.mark.parametrize("d", [100, 1600, 17000])
def test_outputs_on_their_own(outputs, d):
    """Each output alone has the bits that it has among all."""
    g = torch.Generator().manual_seed(0)
    x, r, w = values(6, d, BF, g), values(6, d, BF, g), torch.ones(d, dtype=BF, device="cuda")

    def outs():
        return dict(y=torch.zeros(6, d, dtype=BF, device="cuda"), sum=torch.zeros(6, d, dtype=BF, device="cuda"), q=code_room(6, d, E4)[1],
                    scale=torch.zeros(ref.ceil128(d), 6, device="cuda"), rstd=torch.zeros(6, device="cuda"))
    a, b = outs(), outs()
    ops.opt8_rms_norm_forward(ops.make_rms_norm(x, w, residual=r, **a))
    ops.opt8_rms_norm_forward(ops.make_rms_norm(x, w, residual=r, **{k: b[k] for k in outputs}))
    for k in outputs:
        assert torch.equal(*(t[k].contiguous().view(torch.uint8) for t in (a, b)))


def test_rows_of_zeros_infinities_and_nan():
    """Each row by itself: zeros stay zeros with eps, NaN and infinities keep to their row."""
    x = torch.ones(5, 300, dtype=BF, device="cuda")
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 200] = float("inf")
    w = torch.ones(300, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(5, device="cuda")
    q, s = code_room(5, 300, E4)[1], torch.empty(3, 5, device="cuda")
    ops.opt8_rms_norm_forward(ops.make_rms_norm(x, w, y=y, q=q, scale=s, rstd=rstd, eps=EPS))
    assert bool((y[0] == 0).all()) and bool((q[0].float() == 0).all()) and bool((s[:, 0] == 2.0 ** -126).all())
    assert abs(float(rstd[0]) - EPS ** -0.5) <= 1e3 * 4 * lref.U
    assert bool(y[1].isnan().all()) and bool(rstd[1].isnan()) and bool(q[1].float().isnan().all())
    # 1 / sqrt(inf) = 0: finite values give 0, the infinite one 0 * inf
    assert float(rstd[2]) == 0 and bool(y[2, 200].isnan()) and int((y[2] == 0).sum()) == 299
    for r in (3, 4):
        assert abs(float(rstd[r]) - 1) <= 2 * EPS and bool(((y[r].float() - 1).abs() <= 2.0 ** -8).all())
    ops.opt8_rms_norm_forward(ops.make_rms_norm(x[:1], w, y=y[:1], rstd=rstd[:1], eps=0.0))
    assert float(rstd[0]) == float("inf") and bool(y[0].isnan().all())


def backward(rows, d, dtype, wtype=None, out=None, dsum=True, extra=0, head=0, seed=0, in_place=None, sides="both"):
    g = torch.Generator().manual_seed(seed)
    x, dy = values(rows, d, dtype, g, extra, head), values(rows, d, dtype, g, extra, head)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(wtype or dtype).cuda()
    ds = values(rows, d, dtype, g, extra, head) if dsum else None
    rstd = (x.float().square().mean(1) + EPS).rsqrt()
    (wx, ex), (ww, ew) = lref.norm_grad(dy.cpu(), x.cpu(), w.cpu(), rstd.cpu(), ds.cpu() if dsum else None)
    store, dx = lref.room(rows, d, dtype, extra, head=head)
    if in_place:
        dx = dy if in_place == "dy" else ds
    dw = torch.full((d + 2,), 77.0, dtype=out or dtype, device="cuda")
    work = torch.full((ops.opt8_rms_norm_workspace(rows, d) + 64,), 255, dtype=torch.uint8, device="cuda")
    ops.opt8_rms_norm_backward(ops.make_rms_norm_grad(dy, x, w, rstd, None if sides == "dweight" else dx, None if sides == "dx" else dw[:d],
                                                      work, dsum=ds))
    torch.cuda.synchronize()
    if sides != "dweight":
        lref.check("dx", dx, wx, ex)
        assert in_place or lref.untouched(store, dx)
    if sides != "dx":
        lref.check("dweight", dw[:d], ww, ew)
    assert bool((dw[d:] == 77).all()) and bool((work[-64:] == 255).all())
    return dx, dw


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype,wtype,out", [(BF, BF, BF), (HF, F32, F32), (F32, F32, F32)])
def test_backward(d, dtype, wtype, out):
    rows = 37 if d <= 4100 else 9
    backward(rows, d, dtype, wtype, out)
    backward(rows, d, dtype, wtype, out, dsum=False, extra=3, head=1, seed=1)


@pytest.mark.parametrize("rows,d", [(1, 1), (1, 4096), (17, 64), (4000, 48), (2500, 1600), (700, 9000), (200, 17000)])
@pytest.mark.parametrize("sides", ["both", "dx", "dweight"])
def test_backward_of_few_and_many_rows(rows, d, sides):
    backward(rows, d, BF, out=F32, sides=sides)


@pytest.mark.parametrize("d", [64, 4096, 16384, 17000])
@pytest.mark.parametrize("where", ["dy", "dsum"])
def test_dx_in_an_operand_s_place(d, where):
    backward(1300 if d < 5000 else 20, d, BF, in_place=where)


@pytest.mark.parametrize("rows,d", [(1 << 22, 3), (2, 1 << 20)])
def test_the_most_and_the_widest_rows(rows, d):
    forward(rows, d, BF, kind=E5)
    backward(rows, d, BF, out=F32)


def test_backward_gives_the_same_bits():
    a, b = backward(3000, 200, F32), backward(3000, 200, F32)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_backward_without_rows_stores_zeros():
    e = torch.empty(0, 50, device="cuda")
    dw = torch.ones(50, device="cuda")
    ops.opt8_rms_norm_backward(ops.make_rms_norm_grad(e, e, dw.clone(), torch.empty(0, device="cuda"), e, dw, torch.empty(0, dtype=torch.uint8, device="cuda")))
    assert bool((dw == 0).all())


def test_backward_against_differences():
    """dx and dweight in fp32 against central differences of the 64-bit norm, element by element.
    With steps of 2^-12 and third derivatives below 8 the differences are off by less than 2^-22 (times
    a row's summed |dy| for dx), their arithmetic by less than 2^-40."""
    g = torch.Generator().manual_seed(2)
    rows, d, step = 3, 24, 2.0 ** -12
    x, dy, w = (torch.randn(*s, generator=g) for s in ((rows, d), (rows, d), (d,)))
    w = 1 + 0.2 * w

    def loss(x, w):
        t = x.double()
        return (t * (t.square().mean(1, keepdim=True) + EPS) ** -0.5 * w.double() * dy.double()).sum(1)
    rstd = (x.cuda().square().mean(1) + EPS).rsqrt()
    dx, dw = torch.empty(rows, d, device="cuda"), torch.empty(d, device="cuda")
    work = torch.empty(ops.opt8_rms_norm_workspace(rows, d), dtype=torch.uint8, device="cuda")
    ops.opt8_rms_norm_backward(ops.make_rms_norm_grad(dy.cuda(), x.cuda(), w.cuda(), rstd, dx, dw, work))
    (_, ex), (_, ew) = lref.norm_grad(dy, x, w, rstd.cpu())
    reach = dy.abs().sum(1).max() * 2.0 ** -22
    for j in range(d):
        e = torch.zeros(d, dtype=torch.float64)
        e[j] = step
        diff = (loss(x.double() + e, w) - loss(x.double() - e, w)) / (2 * step)
        # rstd is the fp32 one: 8 U of its own rounding steps reach dx twice
        assert bool(((dx[:, j].cpu().double() - diff).abs() <= ex[:, j] + reach + 16 * lref.U * dy.abs().sum(1)).all())
        diff = ((loss(x, w.double() + e) - loss(x, w.double() - e)) / (2 * step)).sum()
        assert abs(float(dw[j]) - float(diff)) <= float(ew[j]) + float(reach) + 16 * lref.U * float((dy * x).abs()[:, j].sum() * rstd.max())


def test_offsets_past_32_bits():
    """Rows whose distance makes the last ones lie past 2^32 bytes."""
    rows, d, ld = 70001, 96, 40000
    x = torch.empty(rows * ld, dtype=BF, device="cuda").view(rows, ld)[:, :d]
    x.copy_((torch.arange(rows, device="cuda") % 7 + 1)[:, None].expand(rows, d))
    w, y, rstd = torch.ones(d, dtype=BF, device="cuda"), torch.empty(rows, d, dtype=BF, device="cuda"), torch.empty(rows, device="cuda")
    ops.opt8_rms_norm_forward(ops.make_rms_norm(x, w, y=y, rstd=rstd))
    assert bool(((y.float() - 1).abs() <= 2.0 ** -7).all())
    dw, work = torch.empty(d, device="cuda"), torch.empty(ops.opt8_rms_norm_workspace(rows, d), dtype=torch.uint8, device="cuda")
    dx = torch.empty(rows * ld, dtype=BF, device="cuda").view(rows, ld)[:, :d]
    ops.opt8_rms_norm_backward(ops.make_rms_norm_grad(y, x, w, rstd, dx, dw, work))
    # h and y are ones but for rounding: each of the columns sums to the rows
    assert bool(((dw - rows).abs() <= rows * 2.0 ** -7).all()) and bool((dx.abs() <= 2.0 ** -6).all())


@pytest.mark.parametrize("rows,d", [(300, 64), (37, 4096), (9, 16384), (20, 17000)])
def test_dweight_alone_has_no_use_for_dsum(rows, d):
    """The same bits with a dsum of NaN as without one, and as beside dx."""
    g = torch.Generator().manual_seed(4)
    x, dy, w, ds = values(rows, d, BF, g), values(rows, d, BF, g), torch.ones(d, dtype=BF, device="cuda"), torch.full((rows, d), float("nan"), dtype=BF, device="cuda")
    rstd, work = (x.float().square().mean(1) + EPS).rsqrt(), torch.empty(ops.opt8_rms_norm_workspace(rows, d), dtype=torch.uint8, device="cuda")
    got = []
    for dx, dsum in [(None, None), (None, ds), (torch.empty_like(x), ds)]:
        dw = torch.full((d,), 7.0, device="cuda")
        ops.opt8_rms_norm_backward(ops.make_rms_norm_grad(dy, x, w, rstd, dx, dw, work, dsum=dsum))
        got.append(dw)
    assert bool(got[0].isfinite().all()) and torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("d", [1, 7, 128, 500, 1000, 2048, 4096, 8192, 16384, 20000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_whose_squares_leave_fp32(d, dtype):
    """Without eps the norm does not change with its row's size: rows of 2^-125 to 2^125, whose squares are
    0 or infinite in 32 bits, have the formula's values; smaller ones have an infinite rstd, as zeros have."""
    g = torch.Generator().manual_seed(6)
    sizes = torch.tensor([-125.0, -100, -80, -75, -64, -63, -40, 0, 40, 63, 64, 80, 100, 121])
    x = torch.rand(len(sizes), d, generator=g) * 0.5 + 0.75
    x = (x * torch.where(torch.rand(x.shape, generator=g) < 0.5, -1.0, 1.0) * 2.0 ** sizes[:, None]).to(dtype).cuda()
    w = torch.ones(d, dtype=dtype, device="cuda")
    for residual in (None, x * 0.5):
        y, s, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(len(sizes), device="cuda")
        ops.opt8_rms_norm_forward(ops.make_rms_norm(x, w, y=y, rstd=rstd, residual=residual, sum=None if residual is None else s, eps=0.0))
        want = lref.norm(x.cpu(), w.cpu(), 0.0, None if residual is None else residual.cpu())
        lref.check("rstd", rstd, *want["rstd"])
        lref.check("y", y, *want["n"])
    small = torch.full((2, d), 2.0 ** -131, dtype=dtype, device="cuda")
    small[1] = 0
    ops.opt8_rms_norm_forward(ops.make_rms_norm(small, w, rstd=rstd[:2], eps=0.0))
    assert rstd[:2].tolist() == [float("inf")] * 2


@pytest.mark.parametrize("rows,d", [(300, 128), (37, 4096), (5, 20000)])
def test_rstd_is_rounded_once(rows, d):
    """Half a step of fp32 and what 64-bit sums leave of it."""
    x = values(rows, d, BF, torch.Generator().manual_seed(7), scale=3.0)
    rstd = torch.empty(rows, device="cuda")
    ops.opt8_rms_norm_forward(ops.make_rms_norm(x, torch.ones(d, dtype=BF, device="cuda"), rstd=rstd, eps=EPS))
    want = (x.double().square().mean(1) + EPS) ** -0.5
    assert bool(((rstd.double() - want).abs() <= lref.U * (1 + 2.0 ** -20) * want).all())
