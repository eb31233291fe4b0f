"""The operators of opt8_layers.h in calls over 128 MB, which read 16-bit rows past the caches, against
the same rows in small calls or against whole numbers; and by the sort, captured and beside errors of other calls."""

import ctypes

import pytest
import torch

import products_reference as ref
from precision_optimizer_step_amd import opt8, opt8_layers as ops
from test_gpu_layers_calls import Step
from test_gpu_layers_long_sums import embedding_gradient, exact_gradient, ids_of, whole

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
E4 = torch.float8_e4m3fn
LARGE = 128 << 20


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible AMD GPU")
    torch.cuda.set_device(0)


def normal(rows, d, dtype, seed, extra=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.full((rows, d + extra), float("nan"), dtype=dtype, device="cuda")[:, :d]
    return t.copy_(torch.randn(rows, d, device="cuda", generator=g))


def bits(t):
    return t.contiguous().view(torch.uint8)


WIDTHS = [100, 128, 512, 1000, 2048, 4096, 4100, 8192, 12001, 16384, 20000]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("residual", [True, False])
def test_the_norm_of_many_rows(d, dtype, residual):
    """Every output has the bits that its rows have in small calls."""
    rows = LARGE // (d * (6 if residual else 4)) + 300
    x, r = normal(rows, d, dtype, 0, extra=d % 3), normal(rows, d, dtype, 1) if residual else None
    w = normal(1, d, dtype, 2)[0].contiguous()

    def outs(n):
        return dict(y=torch.zeros(n, d, dtype=dtype, device="cuda"), sum=torch.zeros(n, d, dtype=dtype, device="cuda") if residual else None,
                    q=torch.zeros(n, -(-d // 16) * 16, dtype=torch.uint8, device="cuda").view(E4)[:, :d], scale=torch.zeros(ref.ceil128(d), n, device="cuda"),
                    rstd=torch.zeros(n, device="cuda"))
    large = outs(rows)
    ops.opt8_rms_norm_forward(ops.make_rms_norm(x, w, residual=r, **large))
    step = rows // 5
    for a in range(0, rows, step):
        n = min(step, rows - a)
        small = outs(n)
        ops.opt8_rms_norm_forward(ops.make_rms_norm(x[a:a + n], w, residual=None if r is None else r[a:a + n], **small))
        for k, v in small.items():
            if v is not None:
                other = large[k][:, a:a + n] if k == "scale" else large[k][a:a + n]
                assert torch.equal(bits(v), bits(other)), (k, a)
    assert bool(large["rstd"].isfinite().all()) and float(large["y"].float().abs().sum()) > 0


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dsum", [True, False])
def test_the_norm_s_gradient_of_many_rows(d, dtype, dsum):
    """dx has the bits that its rows have in small calls; dweight of whole numbers is exact."""
    rows = LARGE // (d * (8 if dsum else 6)) + 300
    x, dy, ds = normal(rows, d, dtype, 3), normal(rows, d, dtype, 4, extra=d % 3), normal(rows, d, dtype, 5) if dsum else None
    w, rstd = normal(1, d, dtype, 6)[0].contiguous(), normal(rows, 1, F32, 7).abs()[:, 0].contiguous() + 0.5
    dx, dw = torch.zeros(rows, d, dtype=dtype, device="cuda"), torch.zeros(d, device="cuda")
    work = torch.empty(ops.opt8_rms_norm_workspace(rows, d), dtype=torch.uint8, device="cuda")
    ops.opt8_rms_norm_backward(ops.make_rms_norm_grad(dy, x, w, rstd, dx, dw, work, dsum=ds))
    step = rows // 5
    for a in range(0, rows, step):
        n = min(step, rows - a)
        small = torch.zeros(n, d, dtype=dtype, device="cuda")
        ops.opt8_rms_norm_backward(ops.make_rms_norm_grad(dy[a:a + n], x[a:a + n], w, rstd[a:a + n], small, None, dsum=None if ds is None else ds[a:a + n]))
        assert torch.equal(bits(small), bits(dx[a:a + n])), a
    x, dy, rstd = whole(rows, d, dtype, 1, 8), whole(rows, d, dtype, 3, 9, extra=d % 3), torch.ones_like(rstd)
    want = torch.zeros(d, dtype=torch.float64, device="cuda")
    for a in range(0, rows, 4096):
        want += (dy[a:a + 4096].double() * x[a:a + 4096].double()).sum(0)
    ops.opt8_rms_norm_backward(ops.make_rms_norm_grad(dy, x, w, rstd, dx, dw, work, dsum=ds))
    assert torch.equal(dw.double(), want) and float(want.abs().sum()) > 0


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("tokens,vocab,d,kind,accumulate", [(20001, 50257, 1030, "frequent", False), (3000, 70000, 1024, "padded", False),
                                                            (70000, 300, 1001, "even", True), (40000, 5, 2048, "one", True)])
def test_the_gradient_of_many_tokens(dtype, tokens, vocab, d, kind, accumulate):
    assert 2 * d * (tokens + (tokens if accumulate else vocab)) > LARGE
    ids, dy = ids_of(tokens, vocab, kind, 12), whole(tokens, d, dtype, 3, 13, extra=d % 3)
    dy[ids < 0] = float("nan")
    old = whole(vocab, d, F32, 3, 14).contiguous() if accumulate else None
    want = exact_gradient(ids, dy, vocab, old)
    assert torch.equal(embedding_gradient(ids, dy, vocab, old=old).double(), want)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_the_norm_of_a_list_of_many_values(dtype):
    """Whole numbers in every place: their squares' sum is exact."""
    grads = [whole(1, n, dtype, 3, 15 + i)[0].contiguous() for i, n in enumerate((30000001, 8192, 5, 40000003, 7))]
    assert 2 * sum(g.numel() for g in grads) > LARGE
    squares, norm = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(1, device="cuda")
    work = torch.empty(ops.OPT8_GRAD_WORKSPACE, dtype=torch.uint8, device="cuda")
    ops.opt8_grad_norm(ops.make_grads(ops.opt8_grad_table(grads), squares, norm, work))
    assert float(squares) == sum(float(g.double().square().sum()) for g in grads) > 0


def test_the_sorted_gradient_captured_and_replayed():
    """With more tokens than find their like without the sort: three launches in a graph, replayed with new ids
    and eager work between, give the eager bits, on a workspace that holds another batch's."""
    s = Step(6, tokens=300)
    s.run()
    torch.cuda.synchronize()
    wide = torch.zeros(s.sizes[1], s.sizes[2], dtype=BF, device="cuda")

    def part():
        ops.opt8_embedding_backward(ops.make_embedding_grad(s.dids, s.dx, s.acc["table"], s.work[3], scale=4.0))
        ops.opt8_embedding_backward(ops.make_embedding_grad(s.dwhere, s.dx, s.acc["place"], s.work[4], accumulate=True))
        ops.opt8_embedding_backward(ops.make_embedding_grad(s.dids, s.dsum, wide, s.work[3]))
    part()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            part()
    torch.cuda.synchronize()
    g = torch.Generator().manual_seed(16)
    outs = (s.acc["table"], s.acc["place"], wide)
    for i in range(4):
        ids = torch.randint(-1, s.sizes[1], (300,), generator=g)
        if i == 2:
            ids[20:290] = 17       # one id over many chunks
        s.dids.copy_(ids)
        s.dx.copy_(torch.randn(s.dx.shape, generator=g))
        kept = s.acc["place"].clone()
        part()
        torch.cuda.synchronize()
        eager = [t.clone() for t in outs]
        for t in outs:
            t.fill_(9)
        s.acc["place"].copy_(kept)
        s.work[3].fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, outs)), i


def test_an_error_that_another_call_left_is_not_the_sorted_gradient_s():
    path = next(line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line)
    hip = ctypes.CDLL(path)
    ids, dy = ids_of(300, 50, "frequent", 17), normal(300, 40, F32, 18)
    out, work = torch.zeros(50, 40, device="cuda"), torch.empty(ops.opt8_embedding_workspace(300, 50, 40), dtype=torch.uint8, device="cuda")
    call = ops.make_embedding_grad(ids, dy, out, work)
    ops.opt8_embedding_backward(call)
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    try:
        left = hip.hipSetDevice(9999)
        rc = ops.opt8_embedding_backward(call, check=False)
        message, found = opt8.opt8_last_error(), hip.hipGetLastError()
    finally:
        hip.hipGetLastError()
    torch.cuda.synchronize()
    assert left != 0 and found == left and (rc, message) == (opt8.OPT8_OK, "")
    assert torch.equal(out, want) and float(want.abs().sum()) > 0
