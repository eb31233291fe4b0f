"""The longest sums of the operators in opt8_layers.h: whole numbers, whose sums are exact in any order,
and values of one sign, whose roundings would add up."""

import pytest
import torch

import layers_reference as lref
from precision_optimizer_step_amd import opt8_layers as ops

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible AMD GPU")
    torch.cuda.set_device(0)


def embedding_gradient(ids, dy, vocab, scale=1.0, old=None):
    """The fp32 gradient of dy, all on the GPU."""
    tokens, d = dy.shape
    out = torch.full((vocab, d), 77.0, device="cuda") if old is None else old
    work = torch.full((ops.opt8_embedding_workspace(tokens, vocab, d),), 255, dtype=torch.uint8, device="cuda")
    ops.opt8_embedding_backward(ops.make_embedding_grad(ids, dy, out, work, scale=scale, accumulate=old is not None))
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("tokens,d", [(1 << 22, 5), (300000, 130), (20000, 1025)])
def test_a_sum_of_one_sign_does_not_drift(tokens, d):
    """One id's tokens with the same dy, as a placeholder's or a small table's can be: at most 31 additions of
    32 bits in a chunk, the rounding of what the chunks give in 64 bits, and scale's."""
    row = 0.1 + torch.arange(d, device="cuda") * 0.37 % 0.8
    got = embedding_gradient(torch.full((tokens,), 2, device="cuda"), row.expand(tokens, d).contiguous(), 4, 0.7)
    scale = float(torch.tensor(0.7, dtype=F32))
    want = row.cpu().double() * tokens * scale
    lref.check("dtable", got[2], want, (31 + 2 + 1e-3) * lref.U * want)
    assert bool((got[[0, 1, 3]] == 0).all())


def whole(rows, cols, dtype, most, seed, extra=0, head=0):
    """Whole numbers of at most `most`, `extra` columns of NaN behind each row and `head` values of it before the first."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    store = torch.full((rows * (cols + extra) + head,), float("nan"), dtype=dtype, device="cuda")
    t = store[head:].view(rows, cols + extra)[:, :cols]
    t.copy_(torch.randint(-most, most + 1, (rows, cols), device="cuda", generator=g, dtype=torch.int8))
    return t


def ids_of(n, vocab, kind, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "one":
        return torch.full((n,), vocab // 2, device="cuda")
    u = torch.rand(n, device="cuda", generator=g, dtype=torch.float64)
    ids = ((vocab + 1.0) ** u).long().sub(1).clamp(0, vocab - 1) if kind == "frequent" else (u * vocab).long().clamp(0, vocab - 1)
    return torch.where(torch.rand(n, device="cuda", generator=g) < 0.2, -1, ids) if kind == "padded" else ids


def exact_gradient(ids, dy, vocab, old=None):
    """In 64 bits, id by id where they are few, else a million tokens at a time."""
    want = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device="cuda") if old is None else old.double()
    if vocab <= 8:
        for v in range(vocab):
            want[v] += dy[ids == v].sum(0, dtype=torch.float64)
        return want
    for a in range(0, len(ids), 1 << 20):
        i, d = ids[a:a + (1 << 20)], dy[a:a + (1 << 20)]
        there = (i >= 0) & (i < vocab)
        want.index_add_(0, i[there], d[there].double())
    return want


@pytest.mark.parametrize("tokens,vocab,d,kind", [
    (1 << 22, 3, 8, "one"), (1 << 22, 1 << 22, 2, "frequent"), (1 << 22, 7, 3, "padded"), (200000, 5, 8, "one"), (70000, 90, 513, "frequent"),
    (20000, 300000, 24, "even"), (33000, 50257, 1030, "frequent"), (129, 4, 70, "one"), (1000, 50257, 64, "padded")])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_of_whole_numbers_are_exact(tokens, vocab, d, kind, dtype):
    """No sum passes 3 * 2^22 < 2^24: every token's row counts, once."""
    ids, dy = ids_of(tokens, vocab, kind, 1), whole(tokens, d, dtype, 3, 2, extra=3, head=1)
    dy[ids < 0] = float("nan")
    want = exact_gradient(ids, dy, vocab)
    assert float(want.abs().sum()) > 0
    assert torch.equal(embedding_gradient(ids, dy, vocab).double(), want)
    old = whole(vocab, d, F32, 3, 3).contiguous()
    want = exact_gradient(ids, dy, vocab, old)
    assert torch.equal(embedding_gradient(ids.int(), dy, vocab, old=old).double(), want)


@pytest.mark.parametrize("rows,d", [(1 << 22, 3), (1 << 19, 200), (1 << 17, 700), (60000, 1600), (20000, 4096), (5000, 8192), (3000, 9000), (1 << 14, 17000)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_dweight_of_whole_numbers_is_exact(rows, d, dtype):
    """With rstd of one and values of at most 3 and 1 no sum passes 3 * 2^22: every row counts, once."""
    dy, x = whole(rows, d, dtype, 3, 4, extra=1, head=1), whole(rows, d, dtype, 1, 5)
    w, rstd = torch.ones(d, dtype=dtype, device="cuda"), torch.ones(rows, device="cuda")
    work = torch.full((ops.opt8_rms_norm_workspace(rows, d),), 255, dtype=torch.uint8, device="cuda")
    want = torch.zeros(d, dtype=torch.float64, device="cuda")
    for a in range(0, rows, 4096):
        want += (dy[a:a + 4096].double() * x[a:a + 4096].double()).sum(0)
    assert float(want.abs().sum()) > 0
    for dx in (None, torch.empty(rows, d, dtype=dtype, device="cuda")):
        dw = torch.full((d,), 77.0, device="cuda")
        ops.opt8_rms_norm_backward(ops.make_rms_norm_grad(dy, x, w, rstd, dx, dw, work))
        torch.cuda.synchronize()
        assert torch.equal(dw.double(), want)


def test_an_id_s_tokens_are_added_in_their_order():
    """The bits of a sequential sum in 32 bits, by the sort: every id has the 8 tokens that a chunk of a short batch holds."""
    g = torch.Generator().manual_seed(8)
    ids, dy = torch.arange(50).repeat(8)[torch.randperm(400, generator=g)] * 7, torch.randn(400, 33, generator=g)
    want = torch.zeros(400, 33)
    for i, v in enumerate(ids.tolist()):
        want[v] += dy[i]
    assert torch.equal(embedding_gradient(ids.cuda(), dy.cuda(), 400).cpu(), want)


@pytest.mark.parametrize("tokens", [129, 1000, 5003])
def test_a_shared_id_s_chunks_are_joined_exactly(tokens):
    """One id: sequential sums in 32 bits of 8 tokens each, added up in 64 bits (exactly: all are multiples of
    2^-32 below 2^14) and rounded once."""
    dy = torch.randn(tokens, 19, generator=torch.Generator().manual_seed(9))
    dy[dy.abs() < 2.0 ** -8] = 0
    parts = []
    for a in range(0, tokens, 8):
        s = torch.zeros(19)
        for row in dy[a:a + 8]:
            s = s + row
        parts.append(s.double())
    want = torch.stack(parts).sum(0).float()
    got = embedding_gradient(torch.zeros(tokens, dtype=torch.int64, device="cuda"), dy.cuda(), 1)
    assert torch.equal(got[0].cpu(), want)


def test_the_sorted_gradient_past_32_bits():
    """Rows of dtable, and of dy, more than 2^32 bytes from the first, by the sort."""
    vocab, d, tokens = (1 << 20) + 5, 2100, 300
    g = torch.Generator().manual_seed(10)
    ids = torch.full((tokens,), -1)
    some = torch.randperm(tokens, generator=g)[:60]
    ids[some] = vocab - 1 - torch.randint(0, 3, (60,), generator=g)
    ids[some[:5]] = 0
    dy = whole(tokens, d, BF, 3, 11)
    want = exact_gradient((vocab - 1 - ids).cuda().where(ids.cuda() >= 0, -1), dy, 3), exact_gradient(ids.cuda(), dy, 1)
    work = torch.empty(ops.opt8_embedding_workspace(tokens, vocab, d), dtype=torch.uint8, device="cuda")
    table = torch.full((vocab, d), 9.0, dtype=BF, device="cuda")
    for accumulate in (False, True):
        if accumulate:
            table[:1], table[-3:] = 1, 1
        ops.opt8_embedding_backward(ops.make_embedding_grad(ids.cuda(), dy, table, work, accumulate=accumulate))
        assert torch.equal(table[-3:].flip(0).double(), want[0] + accumulate) and torch.equal(table[:1].double(), want[1] + accumulate)
        assert int(table[1:-3].count_nonzero()) == 0
    del table
    ld = (1 << 23) + 8
    far = torch.empty(tokens * ld, dtype=BF, device="cuda").view(tokens, ld)[:, :70]
    far.copy_(dy[:, :70])
    ids = torch.arange(tokens, device="cuda") % 7
    assert torch.equal(embedding_gradient(ids, far, 7).double(), exact_gradient(ids, far, 7))
