"""8-bit block-scaled quantiser and matrix product against plain forms: codes and scales
bit for bit, products exactly where they are whole numbers and within a derived bound elsewhere."""

import pytest
import torch

import products_reference as ref
from precision_optimizer_step_amd import opt8, opt8_products as ops

pytestmark = pytest.mark.gpu

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
ROW, TILE = ops.OPT8_FP8_BLOCK_ROW, ops.OPT8_FP8_BLOCK_TILE
GUARD = 0xA5


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible AMD GPU")
    torch.cuda.set_device(0)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def up16(n):
    return -(-n // 16) * 16


def code_room(rows, cols, kind, extra=0):
    """[rows, cols] codes in rows up16(cols) + extra apart; every byte holds the guard."""
    store = torch.full((rows, up16(cols) + extra), GUARD, dtype=torch.uint8, device="cuda")
    return store, store.view(kind)[:, :cols]


def run_quantize(x, kind, block, q=True, t=True, extra=0):
    rows, cols = x.shape
    tile = block == TILE
    out = {}
    kw = {}
    if q:
        out["q_store"], kw["q"] = code_room(rows, cols, kind, extra)
        kw["scale"] = torch.full((ref.ceil128(cols), ref.ceil128(rows) if tile else rows), -1.0, device="cuda")
    if t:
        out["t_store"], kw["qt"] = code_room(cols, rows, kind, extra)
        kw["scale_t"] = torch.full((ref.ceil128(rows), ref.ceil128(cols) if tile else cols), -1.0, device="cuda")
    ops.opt8_fp8_quantize(ops.make_fp8_quant(x, block=block, **kw))
    torch.cuda.synchronize()
    out.update(kw)
    return out


def same_codes(got, want):
    """NaN codes may differ in their sign bit; all others are equal."""
    g = got.view(torch.uint8).cpu()
    w = want
    nan_g, nan_w = got.cpu().float().isnan(), want.view(got.dtype).float().isnan()
    return bool(torch.equal(nan_g, nan_w)) and bool(torch.equal(g[~nan_g], w[~nan_w]))


def check_quantize(x, kind, block, **kw):
    out = run_quantize(x, kind, block, **kw)
    tile = block == TILE
    for codes, scale, store, src in (("q", "scale", "q_store", x), ("qt", "scale_t", "t_store", x.t())):
        if codes not in out:
            continue
        want, ws = ref.quantize(src, kind, tile)
        assert torch.equal(out[scale].cpu(), ws), f"{scale} differs"
        assert same_codes(out[codes], want), f"{codes} differs"
        pad = out[store][:, src.shape[1]:]
        assert bool((pad == GUARD).all()), "bytes behind a row were written"


SHAPES = [(1, 1), (1, 128), (1, 4096), (3, 129), (128, 128), (127, 257), (129, 127), (300, 1000), (8, 16), (257, 31)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("block", [ROW, TILE])
@pytest.mark.parametrize("kind", [E4, E5])
def test_quantize_shapes(rows, cols, block, kind):
    x = torch.randn(rows, cols, generator=gen(rows * 1000 + cols)).bfloat16().cuda()
    check_quantize(x, kind, block)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("q,t", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("block", [ROW, TILE])
def test_quantize_types_and_outputs(dtype, q, t, block):
    x = (torch.randn(200, 333, generator=gen(5)) * 3).to(dtype).cuda()
    check_quantize(x, E4, block, q=q, t=t, extra=32)


def test_quantize_values_over_the_whole_range():
    """Tiny and huge magnitudes, subnormal maxima, zero blocks, ties between codes."""
    x = torch.zeros(8, 512)
    x[0] = torch.randn(512, generator=gen(1)) * 1e-38
    x[1] = torch.randn(512, generator=gen(2)) * 1e-44
    x[2] = torch.randn(512, generator=gen(3)) * 1e37
    x[3, :128] = 2.0 ** -149
    x[4] = torch.exp(torch.randn(512, generator=gen(4)) * 20)
    x[5] = torch.arange(512) / 512 * 448
    x[6, ::7] = -448.0
    for kind in (E4, E5):
        for block in (ROW, TILE):
            check_quantize(x.cuda(), kind, block)


def test_quantize_nan_and_infinity():
    x = torch.randn(4, 384, generator=gen(9))
    x[0, 5] = float("nan")
    x[1, 130] = float("inf")
    x[2, 300] = float("-inf")
    x[2, 301] = float("nan")
    x[3, 0:128] = float("nan")
    check_quantize(x.cuda(), E4, ROW)
    out = run_quantize(x.cuda(), E4, ROW)
    assert torch.isinf(out["scale"][1, 1]) and out["q"][1, 128:256].float().nan_to_num(7.0)[2] == 7.0
    assert float(out["q"][1, 128].float()) == 0.0


def test_quantize_strided_input_and_unaligned_start():
    base = torch.randn(70, 401, generator=gen(3)).bfloat16().cuda()
    check_quantize(base[:, 1:300], E4, ROW)          # rows 401 apart, start 2 bytes off
    check_quantize(base[::2, :400], E5, TILE)
    wide = torch.randn(70, 408, generator=gen(4)).bfloat16().cuda()
    check_quantize(wide[:, :399], E4, ROW)           # aligned rows, ragged end


# ----------------------------------------------------------------------------- product
def operands(m, n, k, a_kind, tile, seed, extra=0):
    g = gen(seed)
    sa, a = code_room(m, k, a_kind, extra)
    sb, b = code_room(n, k, E4, extra)
    # the guard's bytes behind each row are NaN in neither format, but change any sum they enter
    a.copy_((torch.randn(m, k, generator=g) * 8).to(a_kind))
    b.copy_((torch.randn(n, k, generator=g) * 8).to(E4))
    kb = ref.ceil128(k)
    scale_a = torch.exp(torch.randn(kb, m, generator=g)).cuda()
    scale_b = torch.exp(torch.randn(kb, ref.ceil128(n) if tile else n, generator=g)).cuda()
    return a, scale_a, b, scale_b


def check_exact(m, n, k, a_kind=E4, tile=True, seed=0, extra=0):
    """Codes -1, 0 and 1 (few of them) and scales 1, 2 and 4: every partial sum is a whole number
    below 256, so the kernel's result is the definition's, bit for bit."""
    g = gen(seed)
    _, a = code_room(m, k, a_kind, extra)
    _, b = code_room(n, k, E4, extra)
    few = min(1.0, 24.0 / k)
    a.copy_((torch.randint(0, 2, (m, k), generator=g) * 2 - 1).float().to(a_kind))
    b.copy_(((torch.rand(n, k, generator=g) < few).float() * torch.randint(-1, 2, (n, k), generator=g)).to(E4))
    kb = ref.ceil128(k)
    sa = 2.0 ** torch.randint(0, 2, (kb, m), generator=g).float().cuda()
    sb = 2.0 ** torch.randint(0, 2, (kb, ref.ceil128(n) if tile else n), generator=g).float().cuda()
    c = torch.full((m, n), 77.0, dtype=torch.bfloat16, device="cuda")
    ops.opt8_fp8_matmul(ops.make_fp8_product(a, sa, b, sb, c, block_b=TILE if tile else ROW))
    torch.cuda.synchronize()
    want = ref.decode(a, sa, False) @ ref.decode(b, sb, tile).t()
    assert float(want.abs().max()) <= 256
    assert torch.equal(c.double().cpu(), want)


def check_product(m, n, k, a_kind=E4, tile=True, out=torch.bfloat16, seed=0, extra=0, ldc_extra=0):
    a, sa, b, sb = operands(m, n, k, a_kind, tile, seed, extra)
    store = torch.full((m + 1, n + ldc_extra), 77.0, dtype=out, device="cuda")
    c = store[:m, :n]
    ops.opt8_fp8_matmul(ops.make_fp8_product(a, sa, b, sb, c, block_b=TILE if tile else ROW))
    torch.cuda.synchronize()
    want, bound = ref.product(a, sa, b, sb, tile)
    w = ref.worst(c, want, ref.rounded(want, bound, out))
    assert w <= 1.0, f"error is {w} times its bound"
    assert bool((store[m] == 77).all()) and bool((store[:, n:] == 77).all()), "written outside c"
    return c


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 33, 64, 65, 128, 200, 257])
@pytest.mark.parametrize("n", [1, 16, 100, 129, 384])
def test_product_rows_and_columns(m, n):
    check_exact(m, n, 256, seed=m * 1000 + n)
    check_product(m, n, 256, seed=m * 1000 + n)


@pytest.mark.parametrize("k", [1, 15, 16, 17, 112, 127, 128, 129, 200, 255, 256, 257, 640, 1000])
@pytest.mark.parametrize("m", [5, 70])
@pytest.mark.parametrize("tile", [True, False])
def test_product_depths(m, k, tile):
    check_exact(m, 130, k, tile=tile, seed=k, extra=16)
    check_product(m, 130, k, tile=tile, seed=k, extra=16)


@pytest.mark.parametrize("a_kind", [E4, E5])
@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n", [(3, 48), (40, 200), (150, 260)])
def test_product_types(a_kind, tile, out, m, n):
    check_product(m, n, 320, a_kind=a_kind, tile=tile, out=out, seed=7)


@pytest.mark.parametrize("a_kind", [E4, E5])
@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("k", [128, 200, 333, 700])
def test_product_largest_tiles(a_kind, tile, k):
    check_exact(3601, 3610, k, a_kind=a_kind, tile=tile, seed=8)


@pytest.mark.parametrize("a_kind", [E4, E5])
@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("m,n", [(2001, 4090), (1001, 4090), (501, 4090), (130, 4090)])
def test_product_every_tile_size(a_kind, tile, m, n):
    """128 x 128 with one team of waves and with two, 64 x 64 with two and with four; each at
    depths that give the teams different numbers of steps, and none to some."""
    for k in (100, 300, 520, 1153):
        check_exact(m, n, k, a_kind=a_kind, tile=tile, seed=k)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
def test_product_result_strides(out):
    for ldc_extra in (0, 1, 3, 8):
        check_product(90, 77, 160, out=out, seed=2, ldc_extra=ldc_extra)
        check_product(9, 77, 160, out=out, seed=2, ldc_extra=ldc_extra)


def test_product_ignores_what_lies_behind_a_row():
    """NaN bytes behind each row's k do not reach the result."""
    for m in (4, 90):
        for k in (100, 121, 130):
            a, sa, b, sb = operands(m, 70, k, E4, True, 3)
            for x in (a, b):
                base = x.as_strided((x.shape[0], x.stride(0)), (x.stride(0), 1)).view(torch.uint8)
                base[:, k:] = 0x7F
            c = torch.empty(m, 70, dtype=torch.bfloat16, device="cuda")
            ops.opt8_fp8_matmul(ops.make_fp8_product(a, sa, b, sb, c))
            torch.cuda.synchronize()
            want, bound = ref.product(a, sa, b, sb, True)
            assert ref.worst(c, want, ref.rounded(want, bound, torch.bfloat16)) <= 1.0


def test_product_nan_stays_in_its_row_and_column():
    for m in (20, 100):
        a, sa, b, sb = operands(m, 80, 300, E4, True, 4)
        a.view(torch.uint8)[3, 290] = 0x7F
        b.view(torch.uint8)[50, 7] = 0x7F
        c = torch.empty(m, 80, dtype=torch.bfloat16, device="cuda")
        ops.opt8_fp8_matmul(ops.make_fp8_product(a, sa, b, sb, c))
        torch.cuda.synchronize()
        nan = c.isnan().cpu()
        want = torch.zeros(m, 80, dtype=torch.bool)
        want[3, :] = True
        want[:, 50] = True
        assert torch.equal(nan, want)


def test_product_of_nothing():
    a, sa, b, sb = operands(5, 40, 128, E4, True, 1)
    none = torch.empty(5, 0, device="cuda").to(E4)
    c = torch.full((5, 40), 3.0, dtype=torch.bfloat16, device="cuda")
    empty = torch.empty(0, 5, device="cuda")
    ops.opt8_fp8_matmul(ops.make_fp8_product(none, empty, torch.empty(40, 0, device="cuda").to(E4),
                                             torch.empty(0, 1, device="cuda"), c))
    torch.cuda.synchronize()
    assert bool((c == 0).all())
    c = torch.full((100, 140), 3.0, dtype=torch.bfloat16, device="cuda")
    ops.opt8_fp8_matmul(ops.make_fp8_product(torch.empty(100, 0, device="cuda").to(E4), torch.empty(0, 100, device="cuda"),
                                             torch.empty(140, 0, device="cuda").to(E4), torch.empty(0, 2, device="cuda"), c))
    torch.cuda.synchronize()
    assert bool((c == 0).all())
    ops.opt8_fp8_matmul(ops.make_fp8_product(a[:0], torch.empty(1, 0, device="cuda"), b, sb, torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")))
    ops.opt8_fp8_matmul(ops.make_fp8_product(a, sa, b[:0], torch.empty(1, 0, device="cuda"), torch.empty(5, 0, dtype=torch.bfloat16, device="cuda")))
    torch.cuda.synchronize()


def test_same_call_gives_the_same_bits():
    for m in (7, 300):
        assert torch.equal(check_product(m, 500, 1024, seed=11), check_product(m, 500, 1024, seed=11))


def test_quantised_linear_layer_forward_and_gradients():
    """The three products of a layer from one quantisation of each matrix, tokens odd: within
    the error of rounding each operand to 8 bits (half a step of e4m3 2^-4, of e5m2 2^-3)."""
    g = gen(12)
    tokens, d, f = 137, 256, 384
    x, w, dy = (torch.randn(*s, generator=g).bfloat16().cuda() for s in ((tokens, d), (f, d), (tokens, f)))
    qx, qw, qy = run_quantize(x, E4, ROW), run_quantize(w, E4, TILE), run_quantize(dy, E5, ROW)
    y, dx, dw = (torch.empty(*s, dtype=torch.bfloat16, device="cuda") for s in ((tokens, f), (tokens, d), (f, d)))
    ops.opt8_fp8_matmul(ops.make_fp8_product(qx["q"], qx["scale"], qw["q"], qw["scale"], y))
    ops.opt8_fp8_matmul(ops.make_fp8_product(qy["q"], qy["scale"], qw["qt"], qw["scale_t"], dx))
    ops.opt8_fp8_matmul(ops.make_fp8_product(qy["qt"], qy["scale_t"], qx["qt"], qx["scale_t"], dw, block_b=ROW))
    torch.cuda.synchronize()
    X, W, Y = x.double().cpu(), w.double().cpu(), dy.double().cpu()
    e4, e5 = ref.half_step(E4), ref.half_step(E5)
    # values far below their block's largest lose more than half a relative step (subnormal codes):
    # half the smallest e4m3 number 2^-9 of a scale max/448, half of e5m2's 2^-16 of max/57344
    t4 = 2.0 ** -10 / 448 * 5.5
    t5 = 2.0 ** -17 / 57344 * 5.5

    def bound(a, b, ea, eb, ta, tb):
        A, B = a.abs(), b.abs()
        da, db = A * ea + ta, B * eb + tb
        # and the product's own: its cut (at most 7/8 * 8 * 2^-13 of sum|terms|) and bf16's half step
        return A @ db + da @ B + da @ db + (A @ B) * (7 * 2.0 ** -13 + 2.0 ** -8)
    assert ref.worst(y, X @ W.t(), bound(X, W.t(), e4, e4, t4, t4)) <= 1.0
    assert ref.worst(dx, Y @ W, bound(Y, W, e5, e4, t5, t4)) <= 1.0
    assert ref.worst(dw, Y.t() @ X, bound(Y.t(), X, e5, e4, t5, t4)) <= 1.0


def test_other_stream_and_graph():
    """A call on a side stream, and a captured one replayed over new inputs."""
    a, sa, b, sb = operands(100, 260, 384, E4, True, 21)
    c = torch.empty(100, 260, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(100, 384, generator=gen(22)).bfloat16().cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p, q = ops.make_fp8_product(a, sa, b, sb, c), ops.make_fp8_quant(x, a, sa)
    ops.opt8_fp8_quantize(q, stream=side)
    ops.opt8_fp8_matmul(p, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.opt8_fp8_quantize(q)
        ops.opt8_fp8_matmul(p)
    for k in range(3):
        x.copy_(torch.randn(100, 384, generator=gen(30 + k)))
        c.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        replayed = c.clone()
        c.fill_(6.0)
        ops.opt8_fp8_quantize(q)
        ops.opt8_fp8_matmul(p)
        torch.cuda.synchronize()
        assert torch.equal(replayed, c)
        want, bound = ref.product(a, sa, b, sb, True)
        assert ref.worst(c, want, ref.rounded(want, bound, torch.bfloat16)) <= 1.0


def test_library_refusals_reach_the_caller():
    a, sa, b, sb = operands(4, 16, 128, E4, True, 1)
    c = torch.empty(4, 16, dtype=torch.bfloat16, device="cuda")
    p = ops.make_fp8_product(a, sa, b, sb, c)
    p.c = p.a
    with pytest.raises(opt8.Opt8Error) as e:
        ops.opt8_fp8_matmul(p)
    assert e.value.status == opt8.OPT8_E_ALIAS


def test_offsets_past_32_bits():
    """x, codes and results of over 2^31 elements: the last rows are as those of a small call."""
    rows, cols, n = 70003, 32784, 32784
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    qt_store, qt = code_room(cols, rows, E4)
    q = torch.empty(rows, cols, dtype=torch.uint8, device="cuda").view(E4)
    s, st = torch.empty(ref.ceil128(cols), rows, device="cuda"), torch.empty(ref.ceil128(rows), cols, device="cuda")
    ops.opt8_fp8_quantize(ops.make_fp8_quant(x, q, s, qt, st))
    torch.cuda.synchronize()
    tail = x[-83:]                       # the last block of rows (70003 = 546 * 128 + 115) ends here
    want, ws = ref.quantize(tail, E4, False)
    assert torch.equal(q[-83:].view(torch.uint8).cpu(), want) and torch.equal(s[:, -83:].cpu(), ws)
    want, ws = ref.quantize(x[-115:].t()[-40:], E4, False)
    assert torch.equal(qt[-40:, -115:].view(torch.uint8).cpu(), want) and torch.equal(st[-1:, -40:].cpu(), ws)
    del x, qt, qt_store
    k = 144
    a = q.as_strided((rows, k), (cols, 1), cols - k)       # the last columns: rows of q, far apart
    b = q.as_strided((n, k), (cols, 1), 16)
    sa, sb = torch.ones(2, rows, device="cuda"), torch.ones(2, ref.ceil128(n), device="cuda")
    a_own = torch.empty(rows + 1, cols, dtype=torch.uint8, device="cuda").view(E4)   # owns what lies behind the last row
    a_own.view(torch.uint8)[:rows].copy_(q.view(torch.uint8))
    a = a_own.as_strided((rows, k), (cols, 1), cols - k)
    b = a_own.as_strided((n, k), (cols, 1), 16)
    del q
    c = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    ops.opt8_fp8_matmul(ops.make_fp8_product(a, sa, b, sb, c))
    torch.cuda.synchronize()
    for r in (slice(0, 40), slice(rows - 60, rows)):
        want, bound = ref.product(a[r], sa[:, r], b[-50:], torch.ones(2, 1, device="cuda"), True)
        assert ref.worst(c[r, -50:], want, ref.rounded(want, bound, torch.bfloat16)) <= 1.0


def test_two_streams_at_once():
    """Different calls on two streams without order between them: each as alone."""
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    sets = [operands(300, 500, 1024, E4, True, s) for s in (31, 32)]
    alone = []
    for a, sa, b, sb in sets:
        c = torch.empty(300, 500, dtype=torch.bfloat16, device="cuda")
        ops.opt8_fp8_matmul(ops.make_fp8_product(a, sa, b, sb, c))
        alone.append(c)
    torch.cuda.synchronize()
    outs = [torch.zeros_like(c) for c in alone]
    torch.cuda.synchronize()
    for _ in range(20):
        for side, (a, sa, b, sb), c in zip(sides, sets, outs):
            ops.opt8_fp8_matmul(ops.make_fp8_product(a, sa, b, sb, c), stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(alone, outs))


@pytest.mark.parametrize("rows,cols", [(0, 5), (5, 0), (0, 0)])
def test_quantize_of_nothing(rows, cols):
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for block in (ROW, TILE):
        run_quantize(x, E4, block)


def test_the_longest_rows():
    """k at its limit (2^22), and rows 2^23 bytes apart: the last tile row's offsets end below 2^31."""
    check_exact(2, 17, 1 << 22, seed=1)
    check_exact(20, 17, 1 << 22, seed=2)
    far, m, k = 1 << 23, 270, 300
    store = torch.zeros(m, far, dtype=torch.uint8, device="cuda")
    a = store.view(E4)[:, :k]
    a.copy_(torch.randint(-1, 2, (m, k), generator=gen(3)).float().to(E4))
    b = torch.randint(-1, 2, (40, 304), generator=gen(4)).float().to(E4).cuda()[:, :k]
    c = torch.empty(m, 40, dtype=torch.bfloat16, device="cuda")
    sa, sb = torch.ones(3, m, device="cuda"), torch.ones(3, 1, device="cuda")
    ops.opt8_fp8_matmul(ops.make_fp8_product(a, sa, b, sb, c))
    torch.cuda.synchronize()
    assert torch.equal(c.double().cpu(), a.float().double().cpu() @ b.float().double().cpu().t())
