"""The operators between a language model's weights and their gradients, as cases to measure: block-scaled 8-bit
floating point (quantiser and matrix product) and the gated feed-forward block (forward and backward).

`run` computes each in elementary torch operations in 32 bits, or (`own`) through the package's entry points.
Widths are those of the workload lists (1024/4096, 1600/6400, 2560/10240, 4096/16384) and generic ones.
"""
import math

import torch

own = False

BLOCK = 128
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
LARGEST = 8192 * 4096 * 16384     # rows x width x width of the largest listed cases


def blocks(n):
    return -(-n // BLOCK)


def round16(n):
    return -(-n // 16) * 16


def listed():
    return [
        # one token's activations before an 8-bit product: latency
        dict(name="quantize-one-token", op="quantize", rows=1, cols=4096, tile=False, both=False, x="bf16", fmt="e4m3"),
        # a ragged batch's output gradient, in both orientations (for the input's and the weight's gradient)
        dict(name="quantize-gradient", op="quantize", rows=4001, cols=10240, tile=False, both=True, x="bf16", fmt="e5m2"),
        # the largest weight after an optimizer step, for the forward product and for the input's gradient
        dict(name="quantize-weight", op="quantize", rows=16384, cols=4096, tile=True, both=True, x="bf16", fmt="e4m3"),
        # one token through the widest projection: the weight is read once
        dict(name="product-one-token", op="product", m=1, n=16384, k=4096, tile=True, out="bf16", fmt="e4m3"),
        # a short prompt through a down projection
        dict(name="product-short", op="product", m=333, n=2560, k=10240, tile=True, out="bf16", fmt="e4m3"),
        # a training batch through the widest projection
        dict(name="product-forward", op="product", m=8192, n=16384, k=4096, tile=True, out="bf16", fmt="e4m3"),
        # a weight's gradient over an odd number of tokens: both operands scaled by rows
        dict(name="product-weight-grad", op="product", m=10240, n=2560, k=4093, tile=False, out="bf16", fmt="e5m2"),
        # one token through the gated block: both weights are read once
        dict(name="gated-one-token", op="gated", rows=1, d=4096, f=16384, act="silu", x="bf16", save=False),
        # an odd batch in fp16, with what the backward pass needs
        dict(name="gated-odd", op="gated", rows=777, d=1600, f=6400, act="gelu", x="fp16", save=True),
        # a training batch
        dict(name="gated-forward", op="gated", rows=8192, d=4096, f=16384, act="silu", x="bf16", save=True),
        # the backward pass of a small batch and of a training batch
        dict(name="gated-backward-small", op="gated-grad", rows=500, d=1024, f=4096, act="gelu_tanh", x="bf16"),
        dict(name="gated-backward", op="gated-grad", rows=8192, d=4096, f=16384, act="silu", x="bf16"),
    ]


def _spread(rng, low, high, multiple=1):
    """A whole number between low and high, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / multiple)) * multiple))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "gated", "gated-grad"])
    if op == "quantize":
        return dict(op=op, rows=_spread(rng, 1, 16384), cols=_spread(rng, 128, 16384, 16), tile=rng.random() < 0.4,
                    both=rng.random() < 0.6, x=rng.choice(["bf16", "bf16", "fp16", "fp32"]), fmt=rng.choice(["e4m3", "e5m2"]))
    while True:
        if op == "product":
            tile = rng.random() < 0.6
            c = dict(op=op, m=_spread(rng, 1, 16384), n=_spread(rng, 64, 16384),
                     k=_spread(rng, 128, 16384, 16) if tile else _spread(rng, 128, 16384), tile=tile,
                     out=rng.choice(["bf16", "bf16", "fp16"]), fmt=rng.choice(["e4m3", "e5m2"]))
            size = c["m"] * c["n"] * c["k"]
        else:
            c = dict(op=op, rows=_spread(rng, 1 if op == "gated" else 64, 16384), d=_spread(rng, 256, 4096, 8),
                     f=_spread(rng, 512, 16384, 8), act=rng.choice(["silu", "gelu", "gelu_tanh"]),
                     x=rng.choice(["bf16", "bf16", "fp16"]))
            if op == "gated":
                c["save"] = rng.random() < 0.5
            size = c["rows"] * c["d"] * c["f"]
        if size <= LARGEST // 2:
            return c


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(rows, cols, gen, scale=1.0):
    """Normal values with some channels far larger than the others, as activations have."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    loud = torch.rand(cols, device="cuda", generator=gen) < 0.01
    return x * torch.where(loud, 20.0, 1.0) * scale


def _encode(x, fmt, tile):
    """8-bit codes and scales of x (scales [blocks of columns, rows or blocks of rows])."""
    rows, cols = x.shape
    kb, rb = blocks(cols), blocks(rows)
    p = torch.zeros(rb * BLOCK if tile else rows, kb * BLOCK, device=x.device)
    p[:rows, :cols] = x
    if tile:
        top = p.view(rb, BLOCK, kb, BLOCK).abs().amax((1, 3))
    else:
        top = p.view(rows, kb, BLOCK).abs().amax(2)
    # tensors on both sides of each division: by a Python number torch multiplies by its rounded inverse
    scale = (top / torch.full_like(top, FMAX[fmt])).clamp_min(2.0 ** -126)
    by = torch.ones_like(scale) / scale
    by = by.repeat_interleave(BLOCK, 1)[:, :cols]
    if tile:
        by = by.repeat_interleave(BLOCK, 0)[:rows]
    return (x * by).to(F8[fmt]), scale.t().contiguous()


def _padded(q):
    """The same codes with rows a multiple of 16 bytes apart."""
    rows, cols = q.shape
    store = torch.zeros(rows, round16(cols), device=q.device, dtype=torch.uint8)
    store[:, :cols] = q.view(torch.uint8)
    return store.view(q.dtype)[:, :cols]


def _room(rows, cols, dtype):
    """An output with rows a multiple of 16 bytes apart."""
    each = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.empty(rows, -(-cols // each) * each, device="cuda", dtype=dtype)[:, :cols]


def prepare(case, seed):
    gen = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "quantize":
        r, c, tile = case["rows"], case["cols"], case["tile"]
        small = 1e-3 if case["fmt"] == "e5m2" else 0.02 if tile else 1.0
        s["x"] = _activations(r, c, gen, small).to(TYPES[case["x"]])
        s["q"] = _room(r, c, F8[case["fmt"]])
        s["scale"] = torch.empty(blocks(c), blocks(r) if tile else r, device="cuda")
        s["qt"] = s["scale_t"] = None
        if case["both"]:
            s["qt"] = _room(c, r, F8[case["fmt"]])
            s["scale_t"] = torch.empty(blocks(r), blocks(c) if tile else c, device="cuda")
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        a = _activations(m, k, gen, 1e-3 if case["fmt"] == "e5m2" else 1.0)
        b = torch.randn(n, k, device="cuda", generator=gen) * 0.02 if case["tile"] else _activations(n, k, gen)
        s["a"], s["scale_a"] = _encode(a, case["fmt"], False)
        s["b"], s["scale_b"] = _encode(b, "e4m3", case["tile"])
        if k % 16:
            s["a"], s["b"] = _padded(s["a"]), _padded(s["b"])
        s["c"] = torch.empty(m, n, device="cuda", dtype=TYPES[case["out"]])
    else:
        r, d, f, t = case["rows"], case["d"], case["f"], TYPES[case["x"]]
        s["x"] = torch.randn(r, d, device="cuda", generator=gen).to(t)
        s["w_gate"] = (torch.randn(f, d, device="cuda", generator=gen) / math.sqrt(d)).to(t)
        s["w_up"] = (torch.randn(f, d, device="cuda", generator=gen) / math.sqrt(d)).to(t)
        if op == "gated":
            s["h"] = torch.empty(r, f, device="cuda", dtype=t)
            s["gate"] = torch.empty(r, f, device="cuda", dtype=t) if case["save"] else None
            s["up"] = torch.empty(r, f, device="cuda", dtype=t) if case["save"] else None
        else:
            # what the forward pass left: both projections, rounded to the type
            s["gate"] = torch.randn(r, f, device="cuda", generator=gen).to(t)
            s["up"] = torch.randn(r, f, device="cuda", generator=gen).to(t)
            # half precision trains with a scaled loss, so its gradients stay among the normal numbers
            s["dh"] = (torch.randn(r, f, device="cuda", generator=gen) * (1.0 if case["x"] == "fp16" else 1e-3)).to(t)
            s["dx"] = torch.empty(r, d, device="cuda", dtype=t)
            s["dw_gate"] = torch.empty(f, d, device="cuda", dtype=t)
            s["dw_up"] = torch.empty(f, d, device="cuda", dtype=t)
            # scratch memory of the backward pass: two arrays like `gate`, and room for partial sums
            s["scratch"] = torch.empty(2 * 2 * r * f + (64 << 20), device="cuda", dtype=torch.uint8)
    return s


def _decoded(q, scale, tile):
    """The 32-bit values that codes and scales stand for."""
    rows, cols = q.shape
    by = scale.t().repeat_interleave(BLOCK, 1)[:, :cols]
    if tile:
        by = by.repeat_interleave(BLOCK, 0)[:rows]
    return q.float() * by


_C = math.sqrt(2.0 / math.pi)


def _act(g, kind):
    if kind == "silu":
        return g / (1.0 + torch.exp(-g))
    if kind == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1.0 + torch.tanh(_C * (g + 0.044715 * g * g * g)))


def _slope(g, kind):
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return p * (1.0 + g * (1.0 - p))
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    t = torch.tanh(_C * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * _C * (1.0 + 3 * 0.044715 * g * g)


def _plain(s):
    op = s["op"]
    if op == "quantize":
        x = s["x"].float()
        q, scale = _encode(x, s["fmt"], s["tile"])
        if not s["both"]:
            return dict(q=q, scale=scale)
        qt, scale_t = _encode(x.t(), s["fmt"], s["tile"])
        return dict(q=q, scale=scale, qt=qt, scale_t=scale_t)
    if op == "product":
        a, b = _decoded(s["a"], s["scale_a"], False), _decoded(s["b"], s["scale_b"], s["tile"])
        return dict(c=torch.matmul(a, b.t()).to(TYPES[s["out"]]))
    t = s["x"].dtype
    x, wg, wu = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
    if op == "gated":
        g, u = torch.matmul(x, wg.t()), torch.matmul(x, wu.t())
        out = dict(h=(_act(g, s["act"]) * u).to(t))
        if s["save"]:
            out.update(gate=g.to(t), up=u.to(t))
        return out
    g, u, dh = s["gate"].float(), s["up"].float(), s["dh"].float()
    dg, du = dh * u * _slope(g, s["act"]), dh * _act(g, s["act"])
    dx = torch.matmul(dg, wg) + torch.matmul(du, wu)
    return dict(dx=dx.to(t), dw_gate=torch.matmul(dg.t(), x).to(t), dw_up=torch.matmul(du.t(), x).to(t))


def _own(s):
    from precision_optimizer_step_amd import opt8_products as ops
    op = s["op"]
    if op == "quantize":
        block = ops.OPT8_FP8_BLOCK_TILE if s["tile"] else ops.OPT8_FP8_BLOCK_ROW
        ops.opt8_fp8_quantize(ops.make_fp8_quant(s["x"], s["q"], s["scale"], s["qt"], s["scale_t"], block=block))
        if not s["both"]:
            return dict(q=s["q"], scale=s["scale"])
        return dict(q=s["q"], scale=s["scale"], qt=s["qt"], scale_t=s["scale_t"])
    if op == "product":
        block = ops.OPT8_FP8_BLOCK_TILE if s["tile"] else ops.OPT8_FP8_BLOCK_ROW
        ops.opt8_fp8_matmul(ops.make_fp8_product(s["a"], s["scale_a"], s["b"], s["scale_b"], s["c"], block_b=block))
        return dict(c=s["c"])
    act = {"silu": ops.OPT8_ACT_SILU, "gelu": ops.OPT8_ACT_GELU, "gelu_tanh": ops.OPT8_ACT_GELU_TANH}[s["act"]]
    if op == "gated":
        ops.opt8_gated_ffn_forward(ops.make_gated_ffn(s["x"], s["w_gate"], s["w_up"], s["h"], s["gate"], s["up"], act=act))
        if not s["save"]:
            return dict(h=s["h"])
        return dict(h=s["h"], gate=s["gate"], up=s["up"])
    ops.opt8_gated_ffn_backward(ops.make_gated_ffn_grad(s["dh"], s["x"], s["w_gate"], s["w_up"], s["gate"], s["up"],
                                                        s["dx"], s["dw_gate"], s["dw_up"], s["scratch"], act=act))
    return dict(dx=s["dx"], dw_gate=s["dw_gate"], dw_up=s["dw_up"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op == "quantize":
        r, c, ways = case["rows"], case["cols"], 2 if case["both"] else 1
        scales = 4 * blocks(c) * (blocks(r) if case["tile"] else r)
        if case["both"]:
            scales += 4 * blocks(r) * (blocks(c) if case["tile"] else c)
        return dict(bytes=r * c * (SIZE[case["x"]] + ways) + scales, flops=2 * ways * r * c)
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        scales = 4 * blocks(k) * (m + (blocks(n) if case["tile"] else n))
        return dict(bytes=m * k + n * k + scales + SIZE[case["out"]] * m * n, flops=2 * m * n * k)
    r, d, f = case["rows"], case["d"], case["f"]
    if op == "gated":
        return dict(bytes=2 * (r * d + 2 * f * d + r * f * (3 if case["save"] else 1)), flops=4 * r * d * f)
    return dict(bytes=2 * (3 * r * f + 2 * r * d + 4 * f * d), flops=8 * r * d * f)


# ---------------------------------------------------------------- in 64 bits, from the definitions
def _codes64(x, fmt, tile):
    """The code nearest to each value over its block's scale, and the scales."""
    rows, cols = x.shape
    row_block = torch.arange(rows, device=x.device) // (BLOCK if tile else 1)
    col_block = torch.arange(cols, device=x.device) // BLOCK
    nr, nc = int(row_block[-1]) + 1, int(col_block[-1]) + 1
    by_cols = torch.zeros(rows, nc, device=x.device, dtype=torch.float64)
    by_cols.scatter_reduce_(1, col_block.expand(rows, cols), x.abs(), "amax")
    top = torch.zeros(nr, nc, device=x.device, dtype=torch.float64)
    top.scatter_reduce_(0, row_block[:, None].expand(rows, nc), by_cols, "amax")
    scale = torch.maximum(top / FMAX[fmt], torch.full_like(top, 2.0 ** -126))
    return (x / scale[row_block][:, col_block]).to(F8[fmt]), scale.transpose(0, 1).contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].double()
        q, scale = _codes64(x, case["fmt"], case["tile"])
        if not case["both"]:
            return dict(q=q, scale=scale)
        qt, scale_t = _codes64(x.transpose(0, 1).contiguous(), case["fmt"], case["tile"])
        return dict(q=q, scale=scale, qt=qt, scale_t=scale_t)
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        block = torch.arange(k, device="cuda") // BLOCK
        a = s["a"].float().double() * s["scale_a"].double()[block].transpose(0, 1)
        sb = s["scale_b"].double()[block].transpose(0, 1)
        b = s["b"].float().double() * (sb[torch.arange(n, device="cuda") // BLOCK] if case["tile"] else sb)
        return dict(c=a @ b.transpose(0, 1))
    x, wg, wu = s["x"].double(), s["w_gate"].double(), s["w_up"].double()

    def value_and_slope(g):
        if case["act"] == "silu":
            p = torch.special.expit(g)
            return g * p, p + g * p * (1 - p)
        if case["act"] == "gelu":
            below = torch.special.ndtr(g)
            return g * below, below + g * torch.exp(-g * g / 2) / (2 * math.pi) ** 0.5
        c = (2 / math.pi) ** 0.5
        p = torch.special.expit(2 * c * (g + 0.044715 * g ** 3))
        return g * p, p + 2 * c * g * p * (1 - p) * (1 + 0.134145 * g ** 2)

    if op == "gated":
        g, u = x @ wg.transpose(0, 1), x @ wu.transpose(0, 1)
        h = value_and_slope(g)[0] * u
        return dict(h=h, gate=g, up=u) if case["save"] else dict(h=h)
    value, slope = value_and_slope(s["gate"].double())
    dh = s["dh"].double()
    dg, du = dh * s["up"].double() * slope, dh * value
    return dict(dx=dg @ wg + du @ wu, dw_gate=dg.transpose(0, 1) @ x, dw_up=du.transpose(0, 1) @ x)
