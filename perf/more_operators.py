"""The operators around a language model's matrix products, as cases to measure: token embeddings (lookup and gradient),
the root-mean-square norm (with the residual's addition and 8-bit codes, and its backward pass), and the global norm and
clipping of a list of gradients.

`run` computes each in elementary torch operations in 32 bits, or (`own`) through the package's entry points.
Widths and parameter lists are those of the workload lists (1024, 1600, 2560 and 4096 wide, 50257 tokens) and generic ones.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6          # of the norm, and of the clipping's division
WIDEST = 16384 * 4096


def listed():
    return [
        # one token of a running text and its place: latency
        dict(name="embed-one-token", op="embed", tokens=1, vocab=50257, d=4096, x="bf16", ids="int64", places=2048, pad=False),
        # a training batch, 8 texts of 2048 tokens
        dict(name="embed-batch", op="embed", tokens=16384, vocab=50257, d=4096, x="bf16", ids="int64", places=2048, pad=False),
        # a short batch's gradient added to that of the output head, which has the same table
        dict(name="embed-grad-tied", op="embed-grad", tokens=1001, vocab=50257, d=1600, x="bf16", dw="bf16", ids="int32",
             add=True, pad=False),
        # a padded training batch's gradient for the optimizer's step: every row of the table is written
        dict(name="embed-grad-batch", op="embed-grad", tokens=16384, vocab=50257, d=4096, x="bf16", dw="bf16", ids="int64",
             add=False, pad=True),
        # one token's activations with the residual, as codes for an 8-bit product: latency
        dict(name="norm-one-token", op="norm", rows=1, d=4096, x="bf16", w="bf16", residual=True, y=False, q="e4m3"),
        # every head's own norm in an odd batch: short rows
        dict(name="norm-heads", op="norm", rows=64032, d=128, x="fp16", w="fp32", residual=False, y=True, q=""),
        # a training batch with the residual: the norm for the backward pass, codes and scales for the 8-bit product
        dict(name="norm-batch", op="norm", rows=16384, d=4096, x="bf16", w="bf16", residual=True, y=True, q="e4m3"),
        # the backward pass of an odd batch, and of a training batch whose residual brings a gradient of its own
        dict(name="norm-grad-odd", op="norm-grad", rows=4001, d=1600, x="fp16", w="fp32", dw="fp32", residual=False),
        dict(name="norm-grad-batch", op="norm-grad", rows=16384, d=4096, x="bf16", w="bf16", dw="bf16", residual=True),
        # a small model's gradients, clipped in 32 bits and rounded for the step: latency
        dict(name="clip-small", op="clip", layers=2, d=256, ffn=1024, vocab=1000, places=128, g="fp32", to="bf16", apart=8, clips=True),
        # gradients gathered in 32 bits over several batches, clipped and rounded for the step
        dict(name="clip-gathered", op="clip", layers=24, d=1024, ffn=4096, vocab=50257, places=1024, g="fp32", to="bf16", apart=8, clips=True),
        # the gradients of a large list, in place and within the norm allowed (as most steps are)
        dict(name="clip-large", op="clip", layers=32, d=2560, ffn=10240, vocab=50257, places=2048, g="bf16", to="", apart=8, clips=False),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["embed", "embed-grad", "embed-grad", "norm", "norm", "norm-grad", "norm-grad", "clip"])
    x = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "clip":
        d = _spread(rng, 64, 1024)
        to = rng.choice(["", "bf16", "fp16" if x == "fp16" else "bf16", "fp32"])
        return dict(op=op, layers=_spread(rng, 1, 24), d=d, ffn=4 * d, vocab=_spread(rng, 1000, 50257), places=_spread(rng, 64, 2048),
                    g=x, to=to, apart=rng.choice([1, 8]), clips=bool(to) and rng.random() < 0.6)
    while True:
        if op in ("embed", "embed-grad"):
            c = dict(op=op, tokens=_spread(rng, 1, 32768), vocab=_spread(rng, 100, 131072), d=_spread(rng, 64, 8192), x=x)
            if op == "embed":
                c.update(ids=rng.choice(["int32", "int64"]), places=rng.choice([0, 512, 2048]), pad=rng.random() < 0.3)
            else:
                c.update(dw=rng.choice([x, "fp32"]), ids=rng.choice(["int32", "int64"]), add=rng.random() < 0.3, pad=rng.random() < 0.3)
            fits = c["tokens"] * c["d"] <= WIDEST and c["vocab"] * c["d"] <= 50257 * 4096
        else:
            c = dict(op=op, rows=_spread(rng, 1, 65536), d=_spread(rng, 64, 16384), x=x, w=rng.choice([x, "fp32"]))
            c["residual"] = rng.random() < 0.5
            if op == "norm":
                c["q"] = rng.choice(["", "e4m3", "e5m2"])
                c["y"] = not c["q"] or rng.random() < 0.5
            else:
                c["dw"] = rng.choice([x, "fp32"])
            fits = c["rows"] * c["d"] <= WIDEST
        if fits:
            return c


def _shapes(c):
    """Element counts of the tensors of a decoder's parameter list, in its order."""
    d, ffn = c["d"], c["ffn"]
    layer = [d, d, 3 * d * d, 3 * d, d * d, d, d, d, d * ffn, ffn, ffn * d, d]
    return [c["vocab"] * d, c["places"] * d] + layer * c["layers"] + [d, d]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(rows, cols, gen):
    """Normal values with some channels far larger than the others, as activations have."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    loud = torch.rand(cols, device="cuda", generator=gen) < 0.01
    return x * torch.where(loud, 20.0, 1.0)


def _ids(tokens, vocab, kind, pad, gen):
    """Token numbers, each id about as frequent as 1 / (id + 1); with pad, the end of every 512 tokens is -1 (no token)."""
    u = torch.rand(tokens, device="cuda", generator=gen, dtype=torch.float64)
    ids = (torch.exp(u * math.log(vocab + 1)).long() - 1).clamp(0, vocab - 1)
    if pad:
        ends = torch.randint(256, 513, (-(-tokens // 512),), device="cuda", generator=gen)
        place = torch.arange(tokens, device="cuda")
        ids = torch.where(place % 512 < ends[place // 512], ids, -1)
    return ids.to(torch.int32 if kind == "int32" else torch.int64)


def _blocks(n):
    return -(-n // BLOCK)


def prepare(case, seed):
    gen = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "embed":
        n, v, d, t = case["tokens"], case["vocab"], case["d"], TYPES[case["x"]]
        s["table"] = torch.randn(v, d, device="cuda", generator=gen).mul_(0.02).to(t)
        s["ids"] = _ids(n, v, case["ids"], case["pad"], gen)
        s["place_table"] = s["place_ids"] = None
        if case["places"]:
            s["place_table"] = torch.randn(case["places"], d, device="cuda", generator=gen).mul_(0.01).to(t)
            start = torch.randint(0, case["places"], (1,), device="cuda", generator=gen)
            s["place_ids"] = ((start + torch.arange(n, device="cuda")) % case["places"]).to(s["ids"].dtype)
        s["factor"] = math.sqrt(d)
        s["y"] = torch.empty(n, d, device="cuda", dtype=t)
    elif op == "embed-grad":
        n, v, d, t = case["tokens"], case["vocab"], case["d"], TYPES[case["x"]]
        small = 1.0 if case["x"] == "fp16" else 1e-3    # half precision trains with a scaled loss
        s["ids"] = _ids(n, v, case["ids"], case["pad"], gen)
        s["dy"] = torch.randn(n, d, device="cuda", generator=gen).mul_(small).to(t)
        s["dtable"] = torch.empty(v, d, device="cuda", dtype=TYPES[case["dw"]])
        if case["add"]:
            s["dtable"].copy_(torch.randn(v, d, device="cuda", generator=gen).mul_(small))
        s["factor"] = 0.5
        # scratch memory: the sorted tokens, and partial sums of tokens that many places share
        s["scratch"] = torch.empty(32 * n + 16 * v + n * d + 64 * d + (1 << 20), device="cuda", dtype=torch.uint8)
    elif op == "norm":
        r, d, t = case["rows"], case["d"], TYPES[case["x"]]
        s["x"] = _activations(r, d, gen).to(t)
        s["res"] = s["sum"] = None
        if case["residual"]:
            s["res"] = torch.randn(r, d, device="cuda", generator=gen).mul_(3.0).to(t)
            s["sum"] = torch.empty(r, d, device="cuda", dtype=t)
        s["weight"] = (1.0 + 0.1 * torch.randn(d, device="cuda", generator=gen)).to(TYPES[case["w"]])
        s["out"] = torch.empty(r, d, device="cuda", dtype=t) if case["y"] else None
        s["codes"] = s["scale"] = None
        if case["q"]:
            s["codes"] = torch.empty(r, -(-d // 16) * 16, device="cuda", dtype=F8[case["q"]])[:, :d]
            s["scale"] = torch.empty(_blocks(d), r, device="cuda")
        s["rstd"] = torch.empty(r, device="cuda")
    elif op == "norm-grad":
        r, d, t = case["rows"], case["d"], TYPES[case["x"]]
        s["x"] = _activations(r, d, gen).to(t)
        s["weight"] = (1.0 + 0.1 * torch.randn(d, device="cuda", generator=gen)).to(TYPES[case["w"]])
        small = 1.0 if case["x"] == "fp16" else 1e-3
        s["dy"] = torch.randn(r, d, device="cuda", generator=gen).mul_(small).to(t)
        s["dres"] = torch.randn(r, d, device="cuda", generator=gen).mul_(small).to(t) if case["residual"] else None
        s["rstd"] = 1.0 / torch.sqrt(s["x"].float().square().mean(1) + EPS)     # what the forward pass left
        s["dx"] = torch.empty(r, d, device="cuda", dtype=t)
        s["dweight"] = torch.empty(d, device="cuda", dtype=TYPES[case["dw"]])
        s["scratch"] = torch.empty(4096 * d + (1 << 20), device="cuda", dtype=torch.uint8)     # partial sums
    else:
        # the tensors of a list lie one after another in one store, as they do where ranks exchange them
        counts, apart = _shapes(case), case["apart"]
        begins, end = [], 0
        for n in counts:
            begins.append(end)
            end += -(-n // apart) * apart
        small = 0.1 if case["g"] == "fp16" else 1e-3
        s["store"] = torch.empty(end, device="cuda", dtype=TYPES[case["g"]])
        for at in range(0, end, 1 << 28):
            part = s["store"][at:at + (1 << 28)]
            part.copy_(torch.randn(part.numel(), device="cuda", generator=gen).mul_(small))
        s["grads"] = [s["store"][b:b + n] for b, n in zip(begins, counts)]
        s["store_to"] = s["to_list"] = None
        if case["to"]:
            s["store_to"] = torch.zeros(end, device="cuda", dtype=TYPES[case["to"]])
            s["to_list"] = [s["store_to"][b:b + n] for b, n in zip(begins, counts)]
        # a norm of about small * sqrt(elements)
        s["most"] = small * math.sqrt(sum(counts)) * (0.125 if case["clips"] else 8.0)
        s["squares"] = torch.empty(1, device="cuda", dtype=torch.float64)
        s["norm"] = torch.empty(1, device="cuda")
        s["scratch"] = torch.empty(1 << 16, device="cuda", dtype=torch.uint8)
    return s


def _rows_of(table, ids):
    """Rows of a table in 32 bits; zeros where there is no token."""
    there = ids >= 0
    return torch.where(there[:, None], table[torch.where(there, ids, 0).long()].float(), 0.0)


def _encode(y, fmt):
    """8-bit codes of y's rows and the scale of each 128 values, [blocks of columns, rows]."""
    rows, cols = y.shape
    p = torch.zeros(rows, _blocks(cols) * BLOCK, device=y.device)
    p[:, :cols] = y
    top = p.view(rows, -1, BLOCK).abs().amax(2)
    # tensors on both sides of each division: by a Python number torch multiplies by its rounded inverse
    scale = (top / torch.full_like(top, FMAX[fmt])).clamp_min(2.0 ** -126)
    by = (torch.ones_like(scale) / scale).repeat_interleave(BLOCK, 1)[:, :cols]
    return (y * by).to(F8[fmt]), scale.t().contiguous()


def _plain(s):
    op = s["op"]
    if op == "embed":
        y = _rows_of(s["table"], s["ids"]) * s["factor"]
        if s["place_ids"] is not None:
            y = y + _rows_of(s["place_table"], s["place_ids"])
        return dict(y=y.to(s["y"].dtype))
    if op == "embed-grad":
        there = s["ids"] >= 0
        dy = torch.where(there[:, None], s["dy"].float() * s["factor"], 0.0)
        dt = s["dtable"].float() if s["add"] else torch.zeros(s["vocab"], s["d"], device="cuda")
        dt.index_add_(0, torch.where(there, s["ids"], 0).long(), dy)
        s["dtable"].copy_(dt)
        return dict(dtable=s["dtable"])
    if op == "norm":
        x, t = s["x"].float(), s["x"].dtype
        out = {}
        if s["residual"]:
            x = x + s["res"].float()
            out["sum"] = x.to(t)
        rstd = 1.0 / torch.sqrt((x * x).mean(1) + EPS)
        y = x * rstd[:, None] * s["weight"].float()
        if s["out"] is not None:
            out["y"] = y.to(t)
        if s["q"]:
            out["q"], out["scale"] = _encode(y, s["q"])
        return dict(rstd=rstd, **out)
    if op == "norm-grad":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = s["x"].float() * rstd
        g = dy * s["weight"].float()
        dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
        if s["residual"]:
            dx = dx + s["dres"].float()
        return dict(dx=dx.to(s["x"].dtype), dweight=(dy * xhat).sum(0).to(s["dweight"].dtype))
    squares = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum()
    norm = torch.sqrt(squares)
    factor = (s["most"] / (norm + EPS)).clamp_max(1.0).float()
    to = s["to_list"] if s["to"] else s["grads"]
    for o, g in zip(to, s["grads"]):
        o.copy_(g.float() * factor)
    return dict(norm=norm.float().reshape(1), grads=s["store_to"] if s["to"] else s["store"])


def _own(s):
    from precision_optimizer_step_amd import opt8_layers as ops
    op = s["op"]
    if op == "embed":
        ops.opt8_embedding_forward(ops.make_embedding(s["ids"], s["table"], s["y"], scale=s["factor"], place_ids=s["place_ids"],
                                                      place_table=s["place_table"]))
        return dict(y=s["y"])
    if op == "embed-grad":
        ops.opt8_embedding_backward(ops.make_embedding_grad(s["ids"], s["dy"], s["dtable"], s["scratch"], scale=s["factor"],
                                                            accumulate=s["add"]))
        return dict(dtable=s["dtable"])
    if op == "norm":
        ops.opt8_rms_norm_forward(ops.make_rms_norm(s["x"], s["weight"], y=s["out"], q=s["codes"], scale=s["scale"], rstd=s["rstd"],
                                                    residual=s["res"], sum=s["sum"], eps=EPS))
        out = dict(sum=s["sum"], y=s["out"], q=s["codes"], scale=s["scale"], rstd=s["rstd"])
        return {k: v for k, v in out.items() if v is not None}
    if op == "norm-grad":
        ops.opt8_rms_norm_backward(ops.make_rms_norm_grad(s["dy"], s["x"], s["weight"], s["rstd"], s["dx"], s["dweight"], s["scratch"],
                                                          dsum=s["dres"]))
        return dict(dx=s["dx"], dweight=s["dweight"])
    if "list" not in s:
        # a training loop makes its list once, and keeps it while its gradients stay where they are
        s["list"] = ops.opt8_grad_table(s["grads"], s["to_list"])
    grads = ops.make_grads(s["list"], s["squares"], s["norm"], s["scratch"], max_norm=s["most"])
    ops.opt8_grad_norm(grads)
    ops.opt8_grad_clip(grads)
    return dict(norm=s["norm"], grads=s["store_to"] if s["to"] else s["store"])


def run(state):
    return _own(state) if own else _plain(state)


def _distinct(tokens, vocab):
    """How many different ids so many tokens have, in the mean."""
    p = np.diff(np.log(np.arange(1, vocab + 2))) / math.log(vocab + 1)
    return float((1.0 - np.exp(tokens * np.log1p(-np.minimum(p, 1 - 1e-9)))).sum())


def work(case):
    op = case["op"]
    if op in ("embed", "embed-grad"):
        n, v, d = case["tokens"], case["vocab"], case["d"]
        size, id_size = SIZE[case["x"]], 4 if case["ids"] == "int32" else 8
        there = n * 0.75 if case["pad"] else n
        rows = _distinct(there, v)
        if op == "embed":
            places = min(n, case["places"])
            return dict(bytes=(n + rows + places) * d * size + n * id_size * (2 if places else 1), flops=2 * n * d)
        written = d * SIZE[case["dw"]] * (2 * rows if case["add"] else v)
        return dict(bytes=there * d * size + n * id_size + written, flops=2 * n * d)
    if op in ("norm", "norm-grad"):
        r, d, size = case["rows"], case["d"], SIZE[case["x"]]
        more = 4 * r + SIZE[case["w"]] * d
        if op == "norm":
            each = size * (1 + (2 if case["residual"] else 0) + (1 if case["y"] else 0)) + (1 if case["q"] else 0)
            return dict(bytes=r * d * each + more + (4 * r * _blocks(d) if case["q"] else 0), flops=6 * r * d)
        each = size * (3 + (1 if case["residual"] else 0))
        return dict(bytes=r * d * each + more + SIZE[case["dw"]] * d, flops=10 * r * d)
    n = sum(_shapes(case))
    # within the norm allowed, gradients that stay in place are only read; otherwise read again (the norm is not known before) and written
    again = SIZE[case["g"]] + SIZE[case["to"]] if case["to"] else 0
    return dict(bytes=n * (SIZE[case["g"]] + again), flops=2 * n + (n if again else 0))


# ---------------------------------------------------------------- in 64 bits, from the definitions
def _placed(ids, rows):
    """(places of the tokens, their ids) without the padding."""
    at = torch.nonzero((ids >= 0) & (ids < rows)).flatten()
    return at, ids[at].long()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        y = torch.zeros(case["tokens"], case["d"], device="cuda", dtype=torch.float64)
        at, ids = _placed(s["ids"], case["vocab"])
        y[at] = s["table"][ids].double() * s["factor"]
        if case["places"]:
            at, ids = _placed(s["place_ids"], case["places"])
            y[at] += s["place_table"][ids].double()
        return dict(y=y)
    if op == "embed-grad":
        at, ids = _placed(s["ids"], case["vocab"])
        dt = s["dtable"].double() if case["add"] else torch.zeros(case["vocab"], case["d"], device="cuda", dtype=torch.float64)
        return dict(dtable=dt.index_put((ids,), s["dy"][at].double() * s["factor"], accumulate=True))
    if op == "norm":
        x = s["x"].double()
        out = {}
        if case["residual"]:
            x = x + s["res"].double()
            out["sum"] = x
        power = torch.linalg.vector_norm(x, dim=1) ** 2 / case["d"]
        rstd = (power + EPS) ** -0.5
        y = x * rstd.unsqueeze(1) * s["weight"].double()
        if case["y"]:
            out["y"] = y
        if case["q"]:
            block = torch.arange(case["d"], device="cuda") // BLOCK
            top = torch.zeros(case["rows"], _blocks(case["d"]), device="cuda", dtype=torch.float64)
            top.scatter_reduce_(1, block.expand(case["rows"], case["d"]), y.abs(), "amax")
            scale = torch.maximum(top / FMAX[case["q"]], torch.full_like(top, 2.0 ** -126))
            out["q"], out["scale"] = (y / scale[:, block]).to(F8[case["q"]]), scale.transpose(0, 1).contiguous()
        return dict(rstd=rstd, **out)
    if op == "norm-grad":
        dy, x, w, rstd = s["dy"].double(), s["x"].double(), s["weight"].double(), s["rstd"].double()
        # the derivative of x * rstd(x) * w: rstd changes with x by -rstd^3 x / d
        along = torch.linalg.vecdot(dy * w, x) * rstd ** 3 / case["d"]
        dx = dy * w * rstd.unsqueeze(1) - x * along.unsqueeze(1)
        if case["residual"]:
            dx = dx + s["dres"].double()
        return dict(dx=dx, dweight=torch.matmul(rstd, dy * x))
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g[a:a + (1 << 28)].double())) ** 2
                               for g in s["grads"] for a in range(0, g.numel(), 1 << 28)))
    store = s["store"].double() * min(1.0, s["most"] / (norm + EPS))
    if case["to"]:
        # what lies between the tensors is left as it was
        inside = torch.zeros(store.numel(), device="cuda", dtype=torch.bool)
        for g in s["grads"]:
            inside[g.storage_offset():g.storage_offset() + g.numel()] = True
        store = torch.where(inside, store, 0.0)
    return dict(norm=torch.tensor([norm], device="cuda", dtype=torch.float64), grads=store)
