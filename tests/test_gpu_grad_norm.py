"""Norm and clipping of a list of gradients against 64-bit forms."""

import ctypes
import math
import struct

import pytest
import torch

import layers_reference as lref
from precision_optimizer_step_amd import opt8, opt8_layers as ops

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible AMD GPU")
    torch.cuda.set_device(0)


def scratch():
    return (torch.full((1,), 7.0, dtype=torch.float64, device="cuda"), torch.full((1,), 7.0, device="cuda"),
            torch.full((ops.OPT8_GRAD_WORKSPACE,), 255, dtype=torch.uint8, device="cuda"))


def clip(grads, outs, max_norm):
    squares, norm, work = scratch()
    call = ops.make_grads(ops.opt8_grad_table(grads, outs), squares, norm, work, max_norm=max_norm)
    ops.opt8_grad_norm(call)
    first = float(norm)
    norm.fill_(3.0)
    ops.opt8_grad_clip(call)
    torch.cuda.synchronize()
    assert float(norm) == first or (math.isnan(first) and math.isnan(float(norm)))
    return float(squares), first


def check(sizes, dtype, to, share, scale=1.0, head=0, seed=0):
    """share: of the norm that is allowed; to: type of the places, or None for in place."""
    g = torch.Generator().manual_seed(seed)
    stores, grads, outs, places = [], [], [], []
    for i, n in enumerate(sizes):
        kind = dtype[i % len(dtype)]
        store, t = lref.room(1, n, kind, head=head)
        t.copy_((torch.randn(1, n, generator=g) * scale).to(kind))
        stores.append(store)
        grads.append(t.reshape(n))
        place, o = lref.room(1, n, to[i % len(to)] or kind, head=head)
        own = to[i % len(to)] is not None
        places.append((place, o) if own else None)
        outs.append(o.reshape(n) if own else None)
    before = [t.clone() for t in grads]
    want = math.fsum(float(t.double().square().sum()) for t in before)
    most = share * math.sqrt(want)
    squares, norm = clip(grads, outs, most)
    # each square is exact in 64 bits, their sum off by 2^-53 an addition on paths of under 2^14 of them
    assert abs(squares - want) <= 2.0 ** -38 * want
    assert abs(norm - math.sqrt(want)) <= 2.0 ** -24 * math.sqrt(want) * (1 + 2.0 ** -10)
    factor = min(1.0, most / (math.sqrt(want) + 1e-6))
    for i, (t, o, p) in enumerate(zip(before, outs, places)):
        got = grads[i] if o is None else o
        if factor == 1.0 and got.dtype == t.dtype:
            assert torch.equal(got, t), i
        exact = t.cpu().double() * factor
        lref.check(f"gradient {i}", got, exact, 3 * lref.U * exact.abs())       # the factor's rounding and the product's
        if o is not None:
            assert torch.equal(grads[i], t) and lref.untouched(*p)
        assert lref.untouched(stores[i], grads[i].view(1, -1))


@pytest.mark.parametrize("sizes", [[1], [5, 1, 8192, 8193], [100000], [0, 7, 0], [3] * 500, [2049, 8191, 16384, 16385, 40000]])
@pytest.mark.parametrize("dtype,to", [((BF,), (None,)), ((F32,), (BF,)), ((HF, F32, BF), (None, BF, F32, HF)), ((F32,), (F32, None))])
@pytest.mark.parametrize("share", [0.3, 4.0])
def test_norm_and_clipping(sizes, dtype, to, share):
    check(sizes, dtype, to, share)
    check(sizes, dtype, to, share, head=1, scale=0.01, seed=1)


def test_more_pieces_than_workgroups():
    check([8192 * 5000 + 3, 11], (BF,), (None,), 0.5)


def test_an_empty_list():
    assert clip([], None, 1.0) == (0.0, 0.0)
    assert clip([torch.empty(0, device="cuda")], [torch.empty(0, dtype=BF, device="cuda")], 1.0) == (0.0, 0.0)


@pytest.mark.parametrize("value", [3e38, 1e-38, 1e30, 1e-30])
def test_values_whose_squares_leave_fp32(value):
    n = 1 if value > 1e38 else 9
    for kind in (BF, F32):
        t = torch.full((n,), value, dtype=kind, device="cuda")
        v = float(t[0])
        squares, norm = clip([t], None, v)
        assert abs(squares - n * v * v) <= 2.0 ** -50 * n * v * v
        assert abs(norm - math.sqrt(n) * v) <= 2.0 ** -23 * math.sqrt(n) * v
        factor = min(1.0, v / (math.sqrt(n) * v + 1e-6))
        # below fp32's normal numbers (1e-38 x a small factor) a rounding is half of the smallest number
        lref.check("clipped", t, torch.full((n,), v * factor, dtype=torch.float64), torch.full((n,), 3 * lref.U * v * factor + 2.0 ** -149))


def test_norms_that_are_zero_infinite_or_nan():
    z = torch.zeros(100, dtype=BF, device="cuda")
    assert clip([z], None, 1.0) == (0.0, 0.0) and bool((z == 0).all())
    t = torch.ones(100, dtype=BF, device="cuda")
    t[5] = float("inf")
    assert clip([t], None, 1.0)[1] == math.inf
    assert bool(t[5].isnan()) and int((t == 0).sum()) == 99
    t = torch.ones(100, dtype=BF, device="cuda")
    t[5] = float("nan")
    assert math.isnan(clip([t], None, 1.0)[1]) and bool(t.isnan().all())
    t = torch.ones(100, device="cuda")
    clip([t], None, 0.0)
    assert bool((t == 0).all())


def test_a_factor_of_one_keeps_every_bit():
    """NaN patterns and negative zeros in place; only the norm is read from `squares`."""
    bits = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).cuda()
    t = bits.view(BF).clone()
    squares, norm, work = scratch()
    squares.fill_(0.25)
    ops.opt8_grad_clip(ops.make_grads(ops.opt8_grad_table([t]), squares, norm, max_norm=0.75))
    assert torch.equal(t.view(torch.int16), bits) and float(norm) == 0.5
    ops.opt8_grad_clip(ops.make_grads(ops.opt8_grad_table([t]), squares, max_norm=0.25))
    want = bits.view(BF).double() * (0.25 / (0.5 + 1e-6))
    fine = want.isfinite()
    lref.check("clipped", t[fine], want[fine], 3 * lref.U * want[fine].abs() + 2.0 ** -149)
    assert torch.equal(t.isnan(), want.isnan())


def test_the_squares_of_other_ranks_count():
    """What ranks hold is added up in `squares` between the two calls."""
    parts = [torch.randn(5000, generator=torch.Generator().manual_seed(i)).cuda() for i in range(2)]
    whole = parts[0].clone(), parts[1].clone()
    clip(list(whole), None, 2.0)
    calls = [(t, *scratch()) for t in parts]
    descs = [ops.make_grads(ops.opt8_grad_table([t]), s, n, w, max_norm=2.0) for t, s, n, w in calls]
    for d in descs:
        ops.opt8_grad_norm(d)
    total = calls[0][1] + calls[1][1]
    for (_, s, _, _), d in zip(calls, descs):
        s.copy_(total)
        ops.opt8_grad_clip(d)
    for a, b in zip(parts, whole):      # the sums' order differs: a factor apart by a rounding at most
        assert bool(((a - b).abs() <= 4 * lref.U * b.abs()).all())


def test_more_than_2_to_32_bytes():
    n = (1 << 31) + 12345
    t = torch.zeros(n, dtype=BF, device="cuda")
    at = [0, 8191, 8192, (1 << 31) - 1, 1 << 31, n - 1]
    t[torch.tensor(at, device="cuda")] = 2.0
    squares, norm = clip([t], None, 1.0)
    assert squares == 4.0 * len(at)
    factor = float(torch.tensor(1.0 / (math.sqrt(squares) + 1e-6), dtype=F32))
    assert torch.equal(t[torch.tensor(at, device="cuda")].cpu(), torch.full((len(at),), 2.0 * factor).to(BF))
    assert int(t.count_nonzero()) == len(at)


def test_overlaps_are_refused():
    t = torch.zeros(100, device="cuda")
    for grads, outs in [([t, t], None), ([t[:60], t[50:]], None), ([t[:50]], [t[25:75]]), ([t[:50], t[50:]], [t[50:], None])]:
        with pytest.raises(opt8.Opt8Error, match="overlap"):
            ops.opt8_grad_table(grads, outs)
    ops.opt8_grad_table([t[:50], t[50:]])
    ops.opt8_grad_table([t], [t])


@pytest.mark.parametrize("most", [0.5, 1e9])
def test_a_table_that_held_a_longer_list(most):
    """A table's memory is used again for a shorter list: what the longer one left behind its pieces does not count."""
    long = [torch.full((n,), 2.0, dtype=BF, device="cuda") for n in (8192 * 3, 100, 8193)]
    outs = [torch.full((g.numel(),), 7.0, device="cuda") for g in long]
    short, place = torch.ones(300, device="cuda"), torch.zeros(300, device="cuda")
    fns = ops._functions()

    def listed(grads, places):
        entries = [v for g, o in zip(grads, places) for v in (g.data_ptr(), o.data_ptr(), g.numel(), ops._TYPE[g.dtype], ops._TYPE[o.dtype])]
        return struct.pack("=" + "QQqii" * len(grads), *entries)
    size = fns["opt8_grad_table_bytes"](listed(long, outs), 3)
    assert size == 24 * 7
    memory = bytearray(size)
    at = (ctypes.c_char * size).from_buffer(memory)
    assert fns["opt8_grad_table"](listed(long, outs), 3, at, size) == opt8.OPT8_OK
    assert fns["opt8_grad_table"](listed([short], [place]), 1, at, size) == opt8.OPT8_OK
    squares, norm, work = scratch()
    call = ops.make_grads(torch.frombuffer(memory, dtype=torch.uint8).cuda(), squares, norm, work, max_norm=most)
    ops.opt8_grad_norm(call)
    assert float(squares) == 300.0
    ops.opt8_grad_clip(call)
    factor = min(1.0, most / (math.sqrt(300.0) + 1e-6))
    assert torch.equal(place, torch.full_like(place, factor)) and bool((short == 1).all())
    assert all(bool((g == 2).all()) for g in long) and all(bool((o == 7).all()) for o in outs)


def test_nothing_past_a_table_s_bytes_is_read():
    """A call that names a part of its table takes the pieces in that part, by a factor of 1 too."""
    g, o = torch.ones(8192 * 4, device="cuda"), torch.zeros(8192 * 4, device="cuda")
    table = ops.opt8_grad_table([g], [o])
    squares, norm, work = scratch()
    call = ops.make_grads(table[:24 * 3], squares, norm, work, max_norm=1e9)
    ops.opt8_grad_norm(call)
    assert float(squares) == 2 * 8192
    ops.opt8_grad_clip(call)
    assert bool((o[:2 * 8192] == 1).all()) and bool((o[2 * 8192:] == 0).all())
