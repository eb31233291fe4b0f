"""The operators of opt8_layers.h together, as a training step uses them; captured and replayed; on
two streams at once; beside errors that other calls left."""

import ctypes

import numpy as np
import pytest
import torch

import layers_reference as lref
from precision_optimizer_step_amd import opt8, opt8_layers as ops, opt8_products as products

pytestmark = pytest.mark.gpu

BF, E4, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible AMD GPU")
    torch.cuda.set_device(0)


def codes(rows, cols):
    return torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.uint8, device="cuda").view(E4)[:, :cols]


class Step:
    """One block of a language model between its tokens and its optimizer: embedding with places,
    norm with codes, gated feed-forward block, norm with the residual, an 8-bit head, and back."""

    def __init__(self, seed, tokens=96, vocab=500, places=64, d=160, f=256):
        g = torch.Generator().manual_seed(seed)

        def w(*s, by=1.0):
            return (torch.randn(*s, generator=g) * by).to(BF).cuda()

        def o(*s, kind=BF):
            return torch.zeros(*s, dtype=kind, device="cuda")
        self.sizes = tokens, vocab, d, f
        self.ids = torch.randint(0, vocab, (tokens,), generator=g)
        self.ids[-7:] = -1
        self.where = torch.arange(tokens) % places
        self.p = dict(table=w(vocab, d, by=0.1), place=w(places, d, by=0.1), n1=1 + w(d, by=0.1), n2=1 + w(d, by=0.1),
                      gate=w(f, d, by=d ** -0.5), up=w(f, d, by=d ** -0.5))
        self.p = {k: v.to(BF) for k, v in self.p.items()}
        self.g = {k: torch.zeros_like(v) for k, v in self.p.items()}
        self.acc = {k: torch.zeros_like(v, dtype=F32) for k, v in self.p.items() if k in ("table", "place", "n1", "n2")}
        self.dids, self.dwhere = self.ids.cuda(), self.where.cuda()
        self.x, self.y1, self.h, self.gt, self.ut = o(tokens, d), o(tokens, d), o(tokens, f), o(tokens, f), o(tokens, f)
        self.r1, self.r2, self.s2, self.y2 = o(tokens, kind=F32), o(tokens, kind=F32), o(tokens, d), o(tokens, d)
        self.back = w(d, f, by=f ** -0.5)            # down projection, held fixed, as codes
        self.qw, self.sw = codes(d, f), o(-(-f // 128), -(-d // 128), kind=F32)
        self.qh, self.sh = codes(tokens, f), o(-(-f // 128), tokens, kind=F32)
        self.down = o(tokens, d)
        self.q2, self.sq2 = codes(tokens, d), o(-(-d // 128), tokens, kind=F32)
        self.dy = w(tokens, d, by=0.01)
        self.dsum, self.dh, self.dx1, self.dx = o(tokens, d), o(tokens, f), o(tokens, d), o(tokens, d)
        self.work = [o(n, kind=torch.uint8) for n in (
            products.opt8_gated_ffn_workspace(tokens, d, f), ops.opt8_rms_norm_workspace(tokens, d), ops.opt8_rms_norm_workspace(tokens, d),
            ops.opt8_embedding_workspace(tokens, vocab, d), ops.opt8_embedding_workspace(tokens, places, d), ops.OPT8_GRAD_WORKSPACE)]
        self.squares, self.norm = o(1, kind=torch.float64), o(1, kind=F32)
        names = list(self.p)
        self.table = ops.opt8_grad_table([self.acc.get(k, self.g[k]) for k in names], [self.g[k] if k in self.acc else None for k in names])
        products.opt8_fp8_quantize(products.make_fp8_quant(self.back, self.qw, self.sw, block=products.OPT8_FP8_BLOCK_TILE))

    def run(self):
        p, g, a = self.p, self.g, self.acc
        ops.opt8_embedding_forward(ops.make_embedding(self.dids, p["table"], self.x, scale=4.0, place_ids=self.dwhere, place_table=p["place"]))
        ops.opt8_rms_norm_forward(ops.make_rms_norm(self.x, p["n1"], y=self.y1, rstd=self.r1))
        products.opt8_gated_ffn_forward(products.make_gated_ffn(self.y1, p["gate"], p["up"], self.h, self.gt, self.ut))
        products.opt8_fp8_quantize(products.make_fp8_quant(self.h, self.qh, self.sh))
        products.opt8_fp8_matmul(products.make_fp8_product(self.qh, self.sh, self.qw, self.sw, self.down))
        ops.opt8_rms_norm_forward(ops.make_rms_norm(self.down, p["n2"], y=self.y2, q=self.q2, scale=self.sq2, rstd=self.r2, residual=self.x, sum=self.s2))
        # back: dy of y2; the down projection's gradient for h by a plain product
        ops.opt8_rms_norm_backward(ops.make_rms_norm_grad(self.dy, self.s2, p["n2"], self.r2, self.dsum, a["n2"], self.work[1]))
        torch.matmul(self.dsum, self.back, out=self.dh)
        products.opt8_gated_ffn_backward(products.make_gated_ffn_grad(self.dh, self.y1, p["gate"], p["up"], self.gt, self.ut, self.dx1, g["gate"],
                                                                      g["up"], self.work[0]))
        ops.opt8_rms_norm_backward(ops.make_rms_norm_grad(self.dx1, self.x, p["n1"], self.r1, self.dx, a["n1"], self.work[2], dsum=self.dsum))
        ops.opt8_embedding_backward(ops.make_embedding_grad(self.dids, self.dx, a["table"], self.work[3], scale=4.0))
        ops.opt8_embedding_backward(ops.make_embedding_grad(self.dwhere, self.dx, a["place"], self.work[4]))
        grads = ops.make_grads(self.table, self.squares, self.norm, self.work[5], max_norm=0.05)
        ops.opt8_grad_norm(grads)
        ops.opt8_grad_clip(grads)

    def outputs(self):
        return [t.clone().reshape(-1).view(torch.uint8) for t in (self.x, self.y1, self.s2, self.y2, self.q2.contiguous(), self.sq2, self.dsum, self.dx, self.squares,
                                                                  self.norm, *self.acc.values(), *(self.g[k] for k in self.acc))]


def test_a_step_from_tokens_to_the_optimizer():
    """Every operator's outputs from the inputs that it was given, and the optimizer's step with the
    clipped gradients: the parameters that the oracle has too."""
    import oracle
    s = Step(0)
    s.run()
    torch.cuda.synchronize()
    c = lambda t: t.cpu()   # noqa: E731
    eps = float(torch.tensor(1e-6, dtype=F32))
    lref.check("x", s.x, *lref.embedding(s.ids, c(s.p["table"]), 4.0, s.where, c(s.p["place"])))
    lref.check("y1", s.y1, *lref.norm(c(s.x), c(s.p["n1"]), eps)["n"])
    want = lref.norm(c(s.down), c(s.p["n2"]), eps, c(s.x))
    lref.check("s2", s.s2, *want["sum"])
    lref.check("y2", s.y2, *want["n"])
    (wx, ex), (ww, ew) = lref.norm_grad(c(s.dy), c(s.s2), c(s.p["n2"]), c(s.r2))
    lref.check("dsum", s.dsum, wx, ex)
    lref.check("dn2", s.acc["n2"], ww, ew)
    (wx, ex), (ww, ew) = lref.norm_grad(c(s.dx1), c(s.x), c(s.p["n1"]), c(s.r1), c(s.dsum))
    lref.check("dx", s.dx, wx, ex)
    lref.check("dn1", s.acc["n1"], ww, ew)
    tokens, vocab, d, _ = s.sizes
    lref.check("dtable", s.acc["table"], *lref.embedding_grad(s.ids, c(s.dx), vocab, 4.0))
    lref.check("dplace", s.acc["place"], *lref.embedding_grad(s.where, c(s.dx), len(s.p["place"]), 1.0))
    norm = float(s.squares) ** 0.5
    assert norm > 0.05
    for k, a in s.acc.items():
        exact = c(a).double() * (0.05 / (norm + 1e-6))
        lref.check("g " + k, s.g[k], exact, 3 * lref.U * exact.abs())
    # the step reads the clipped gradients
    opt8.opt8_init_codebooks()
    hp = opt8.make_hparams(1e-2, weight_decay=0.01, step=1, seed=3)
    n = vocab * d
    state = dict(m=torch.full((n,), 127, dtype=torch.uint8, device="cuda"), v=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                 am=torch.zeros(-(-n // 2048), device="cuda"), av=torch.zeros(-(-n // 2048), device="cuda"))
    before = c(s.p["table"]).view(torch.int16).numpy().view(np.uint16).reshape(-1).copy()
    opt8.opt8_adamw_step([opt8.make_tensor(s.p["table"], s.g["table"], state["m"], state["v"], state["am"], state["av"])], hp)
    torch.cuda.synchronize()
    bits = c(s.g["table"]).view(torch.int16).numpy().view(np.uint16).reshape(-1)
    want = oracle.step_tensor(oracle.MODE_8BIT, before, bits, np.full(n, 127, np.uint8), np.zeros(n, np.uint8), np.zeros(-(-n // 2048), np.float32),
                              np.zeros(-(-n // 2048), np.float32), oracle.Hparams(lr=1e-2, weight_decay=0.01, step=1, seed=3), tensor_id=0)
    assert np.array_equal(c(s.p["table"]).view(torch.int16).numpy().view(np.uint16).reshape(-1), want[0])


def test_captured_and_replayed():
    """A graph of the operators, replayed with new inputs and eager work between, gives the eager bits.
    (torch's own product, which the step has in its middle, is run before.)"""
    s = Step(1)
    s.run()
    torch.cuda.synchronize()
    p, a = s.p, s.acc

    def part():
        ops.opt8_embedding_forward(ops.make_embedding(s.dids, p["table"], s.x, scale=4.0, place_ids=s.dwhere, place_table=p["place"]))
        ops.opt8_rms_norm_forward(ops.make_rms_norm(s.down, p["n2"], y=s.y2, q=s.q2, scale=s.sq2, rstd=s.r2, residual=s.x, sum=s.s2))
        ops.opt8_rms_norm_backward(ops.make_rms_norm_grad(s.dy, s.s2, p["n2"], s.r2, s.dsum, a["n2"], s.work[1]))
        ops.opt8_embedding_backward(ops.make_embedding_grad(s.dids, s.dsum, a["table"], s.work[3], scale=4.0))
        ops.opt8_embedding_backward(ops.make_embedding_grad(s.dwhere, s.dsum, a["place"], s.work[4], accumulate=True))
        grads = ops.make_grads(s.table, s.squares, s.norm, s.work[5], max_norm=0.05)
        ops.opt8_grad_norm(grads)
        ops.opt8_grad_clip(grads)
    part()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            part()
    torch.cuda.synchronize()
    g = torch.Generator().manual_seed(5)
    for i in range(4):
        s.dids.copy_(torch.randint(-1, s.sizes[1], (s.sizes[0],), generator=g))
        s.dy.copy_(torch.randn(s.dy.shape, generator=g) * 0.01 * (i + 1))
        kept = a["place"].clone(), {k: v.clone() for k, v in s.g.items()}
        part()
        torch.cuda.synchronize()
        eager = s.outputs()
        for t in (s.x, s.y2, s.s2, s.dsum, a["table"], a["n2"]):
            t.fill_(9)
        a["place"].copy_(kept[0])
        for k, v in kept[1].items():
            s.g[k].copy_(v)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(eager, s.outputs())), i


def test_two_streams_at_once():
    """Two models on two streams, each with its own buffers and workspaces, give the bits that each gives alone."""
    steps = [Step(2), Step(3, tokens=300, d=96)]
    want = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        want.append(s.outputs())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, stream in zip(steps, streams):
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                s.run()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            assert all(torch.equal(x, y) for x, y in zip(w, s.outputs()))


def every_call():
    s = Step(4)
    s.run()
    grads = ops.make_grads(s.table, s.squares, s.norm, s.work[5], max_norm=0.05)
    return s, [
        ("embedding", ops.opt8_embedding_forward, ops.make_embedding(s.dids, s.p["table"], s.x), (s.x,)),
        ("embedding gradient", ops.opt8_embedding_backward, ops.make_embedding_grad(s.dids, s.dx, s.acc["table"], s.work[3]), (s.acc["table"],)),
        ("norm", ops.opt8_rms_norm_forward, ops.make_rms_norm(s.down, s.p["n2"], y=s.y2), (s.y2,)),
        ("norm gradient", ops.opt8_rms_norm_backward, ops.make_rms_norm_grad(s.dy, s.s2, s.p["n2"], s.r2, s.dsum, s.acc["n2"], s.work[1]), (s.dsum, s.acc["n2"])),
        ("gradients' norm", ops.opt8_grad_norm, grads, (s.squares, s.norm)),
        ("clipping", ops.opt8_grad_clip, grads, (s.g["table"],)),
    ]


def test_an_error_that_another_call_left_is_not_the_launch_s():
    path = next(line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line)
    hip = ctypes.CDLL(path)
    s, calls = every_call()
    for name, call, desc, outs in calls:
        call(desc)
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        if name == "clipping":
            s.squares.copy_(torch.tensor([4.0]))
            call(desc)
            want = [t.clone() for t in outs]
            s.squares.copy_(torch.tensor([4.0]))
        torch.cuda.synchronize()
        try:
            left = hip.hipSetDevice(9999)
            rc = call(desc, check=False)
            message = opt8.opt8_last_error()
            found = hip.hipGetLastError()
        finally:
            hip.hipGetLastError()
        torch.cuda.synchronize()
        assert left != 0 and found == left, name
        assert (rc, message) == (opt8.OPT8_OK, ""), name
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), name


def test_a_call_after_the_current_device_changed(monkeypatch):
    _, calls = every_call()
    torch.cuda.synchronize()
    for name, call, desc, outs in calls:
        before = [t.clone() for t in outs]
        with monkeypatch.context() as m:
            m.setattr(torch.cuda, "current_device", lambda: 1)
            with pytest.raises(ValueError, match="cuda:0.*current device is cuda:1"):
                call(desc)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, before)), name
        assert call(desc) == opt8.OPT8_OK
