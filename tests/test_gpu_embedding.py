"""Token embeddings and their gradient against 64-bit forms."""

import pytest
import torch

import layers_reference as lref
from precision_optimizer_step_amd import opt8_layers as ops

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
I32, I64 = torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible AMD GPU")
    torch.cuda.set_device(0)


def values(rows, cols, dtype, g, extra=0, head=0, scale=1.0):
    store, t = lref.room(rows, cols, dtype, extra, fill=float("nan"), head=head)   # what lies between rows is never used
    t.copy_((torch.randn(rows, cols, generator=g) * scale).to(dtype))
    return t


def some_ids(n, vocab, g, kind="even"):
    if kind == "one":
        return torch.full((n,), vocab // 2, dtype=I64)
    if kind == "multiples":    # of the number of the sort's workgroups
        return torch.randint(0, vocab // 256, (n,), generator=g) * 256
    if kind == "frequent":
        return (torch.exp(torch.rand(n, generator=g, dtype=torch.float64) * torch.log(torch.tensor(vocab + 1.0))).long() - 1).clamp(0, vocab - 1)
    ids = torch.randint(0, vocab, (n,), generator=g)
    if kind == "outside":      # paddings and other numbers that are no rows
        ids = torch.where(torch.rand(n, generator=g) < 0.4, torch.tensor([-1, vocab, -5, 2 ** 31 - 1])[torch.randint(0, 4, (n,), generator=g)], ids)
    return ids


def lookup(tokens, vocab, d, dtype=BF, id_type=I64, places=0, scale=1.0, extra=0, head=0, kind="even", seed=0):
    g = torch.Generator().manual_seed(seed)
    table = values(vocab, d, dtype, g, extra, head)
    ids = some_ids(tokens, vocab, g, kind)
    store, y = lref.room(tokens, d, dtype, extra, head=head)
    kw, where = {}, None
    if places:
        where = some_ids(tokens, places, g, "outside" if kind == "outside" else "even")
        kw = dict(place_ids=where.to(id_type).cuda(), place_table=values(places, d, dtype, g, extra, head))
    ops.opt8_embedding_forward(ops.make_embedding(ids.to(id_type).cuda(), table, y, scale=scale, **kw))
    torch.cuda.synchronize()
    scale = float(torch.tensor(scale, dtype=F32))
    want, err = lref.embedding(ids, table.cpu(), scale, where, kw["place_table"].cpu() if places else None)
    lref.check("y", y, want, err)
    assert lref.untouched(store, y)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("tokens,vocab,d", [(1, 1, 1), (1, 100, 4096), (3, 7, 513), (130, 1000, 96), (65, 50, 1030), (1000, 333, 7)])
def test_lookup(tokens, vocab, d, dtype):
    lookup(tokens, vocab, d, dtype, scale=d ** 0.5)
    lookup(tokens, vocab, d, dtype, I32, places=5, extra=3, head=1, kind="outside", seed=1)


def test_lookup_without_a_vocabulary_gives_zeros_and_places():
    ids, p = torch.zeros(5, dtype=I64, device="cuda"), torch.randn(3, 40).cuda()
    y = torch.full((5, 40), 3.0, device="cuda")
    ops.opt8_embedding_forward(ops.make_embedding(ids, torch.empty(0, 40, device="cuda"), y))
    assert bool((y == 0).all())
    ops.opt8_embedding_forward(ops.make_embedding(ids, torch.empty(0, 40, device="cuda"), y, place_ids=ids + 2, place_table=p))
    assert torch.equal(y, p[2].expand(5, 40))
    ops.opt8_embedding_forward(ops.make_embedding(ids + 1, p, y, place_ids=ids, place_table=torch.empty(0, 40, device="cuda")))
    assert torch.equal(y, p[1].expand(5, 40))


def test_rows_beside_the_tokens_do_not_count():
    """NaN and infinities in rows that no token names."""
    table = torch.full((50, 64), float("nan"), dtype=BF, device="cuda")
    table[7] = 2.0
    y = torch.empty(9, 64, dtype=BF, device="cuda")
    ids = torch.tensor([7, -1, 7, 50, 7, 7, 1 << 40, -(1 << 40), 7], device="cuda")
    ops.opt8_embedding_forward(ops.make_embedding(ids, table, y, scale=0.5))
    assert y[:, 0].tolist() == [1, 0, 1, 0, 1, 1, 0, 0, 1] and bool((y == y[:, :1]).all())


def gradient(tokens, vocab, d, dtype=BF, out=None, id_type=I64, accumulate=False, scale=1.0, extra=0, head=0, kind="even", seed=0, spare=0):
    g = torch.Generator().manual_seed(seed)
    out = out or dtype
    dy = values(tokens, d, dtype, g, extra, head)
    ids = some_ids(tokens, vocab, g, kind)
    dy[(ids < 0).to("cuda")] = float("nan")         # a padding's gradient is left out, whatever it is
    store, dtable = lref.room(vocab, d, out, extra, head=head)
    old = torch.randn(vocab, d, generator=g).to(out)
    if accumulate:
        dtable.copy_(old)
    work = torch.full((ops.opt8_embedding_workspace(tokens, vocab, d) + spare,), 255, dtype=torch.uint8, device="cuda")
    call = ops.make_embedding_grad(ids.to(id_type).cuda(), dy, dtable, work, scale=scale, accumulate=accumulate)
    ops.opt8_embedding_backward(call)
    torch.cuda.synchronize()
    want, err = lref.embedding_grad(ids, dy.cpu(), vocab, scale, old if accumulate else None)
    lref.check("dtable", dtable, want, err)
    assert lref.untouched(store, dtable)
    assert not spare or bool((work[-spare:] == 255).all())
    if accumulate:
        without = torch.bincount(ids[(ids >= 0) & (ids < vocab)], minlength=vocab) == 0
        assert torch.equal(dtable.cpu()[without], old[without])
    return dtable


@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, HF), (F32, F32), (BF, F32), (HF, F32)])
@pytest.mark.parametrize("tokens,vocab,d,kind", [(1, 1, 1, "one"), (1, 600, 512, "even"), (40, 7, 33, "even"), (700, 300, 65, "frequent"),
                                                 (2100, 1030, 520, "outside"), (999, 3, 1025, "one")])
def test_gradient(tokens, vocab, d, kind, dtype, out):
    gradient(tokens, vocab, d, dtype, out, kind=kind, scale=0.75, spare=64)
    gradient(tokens, vocab, d, dtype, out, I32, True, kind=kind, extra=5, head=3, seed=1)


@pytest.mark.parametrize("tokens", [2, 63, 64, 65, 127, 128, 129, 130])
@pytest.mark.parametrize("kind", ["one", "frequent", "outside"])
def test_gradient_of_few_tokens(tokens, kind):
    """Around the number that a wave holds, where the sort begins."""
    for accumulate in (False, True):
        gradient(tokens, 11, 530, BF, F32, accumulate=accumulate, kind=kind)
        gradient(tokens, 70, 20, HF, id_type=I32, accumulate=accumulate, kind=kind, extra=1, seed=1)


@pytest.mark.parametrize("tokens,vocab,d,kind", [
    (8191, 50257, 64, "frequent"), (20000, 1000, 40, "frequent"),   # chunks of 8 tokens, and ids over several of them
    (32768, 300, 1024, "even"), (70000, 90, 513, "frequent"),       # chunks of 16 and of 32
    (20000, 300000, 24, "even"),                                    # more ids than 256 workgroups count
    (9000, 50257, 16, "multiples"), (9000, 300000, 16, "multiples"),
    (9000, 4, 16, "one"), (200000, 5, 8, "one")])                   # more of one id than a wave notes
def test_gradient_of_many_tokens(tokens, vocab, d, kind):
    gradient(tokens, vocab, d, F32, kind=kind)


@pytest.mark.parametrize("vocab,d,kind", [(1 << 22, 2, "frequent"), (1 << 22, 1, "even"), (3, 8, "one")])
def test_the_most_tokens(vocab, d, kind):
    """2^22 of them, into as many rows or into one."""
    gradient(1 << 22, vocab, d, BF, F32, kind=kind)
    lookup(1 << 22, vocab, d, BF, kind=kind)


def test_the_widest_rows():
    lookup(3, 5, 1 << 20, BF, places=2)
    gradient(11, 5, 1 << 20, BF, kind="outside")


def test_gradient_without_tokens_is_zero_or_what_it_was():
    ids, dy = torch.empty(0, dtype=I64, device="cuda"), torch.empty(0, 70, dtype=BF, device="cuda")
    work = torch.empty(ops.opt8_embedding_workspace(0, 33, 70), dtype=torch.uint8, device="cuda")
    dt = torch.ones(33, 70, dtype=BF, device="cuda")
    ops.opt8_embedding_backward(ops.make_embedding_grad(ids, dy, dt, work, accumulate=True))
    assert bool((dt == 1).all())
    ops.opt8_embedding_backward(ops.make_embedding_grad(ids, dy, dt, work))
    assert bool((dt == 0).all())


def test_gradient_gives_the_same_bits_and_sums_in_the_tokens_order():
    """Twice the same bits, and those of a sequential fp32 sum where an id's tokens lie in one chunk."""
    a = gradient(3000, 40, 100, F32, kind="frequent")
    assert torch.equal(a, gradient(3000, 40, 100, F32, kind="frequent"))
    g = torch.Generator().manual_seed(3)
    dy, ids = torch.randn(8, 24, generator=g), torch.tensor([4, 2, 4, 4, 2, 0, 4, 2])
    dt, work = torch.empty(6, 24, device="cuda"), torch.empty(ops.opt8_embedding_workspace(8, 6, 24), dtype=torch.uint8, device="cuda")
    ops.opt8_embedding_backward(ops.make_embedding_grad(ids.cuda(), dy.cuda(), dt, work))
    want = torch.zeros(6, 24)
    for i, v in enumerate(ids.tolist()):
        want[v] += dy[i]
    assert torch.equal(dt.cpu(), want)


def test_gradient_is_the_lookup_s_derivative():
    """The lookup is linear: <dy, lookup(table)> changes with the table by its gradient, here in numbers
    that fp32 holds exactly."""
    g = torch.Generator().manual_seed(0)
    vocab, d, tokens = 20, 32, 90
    ids = torch.randint(-1, vocab, (tokens,), generator=g)
    dy = torch.randint(-8, 9, (tokens, d), generator=g).float()
    dt, work = torch.empty(vocab, d, device="cuda"), torch.empty(ops.opt8_embedding_workspace(tokens, vocab, d), dtype=torch.uint8, device="cuda")
    ops.opt8_embedding_backward(ops.make_embedding_grad(ids.cuda(), dy.cuda(), dt, work, scale=0.5))
    for row, col in [(0, 0), (7, 31), (19, 5)]:
        ends = []
        for step in (1.0, -1.0):
            table, y = torch.zeros(vocab, d, device="cuda"), torch.empty(tokens, d, device="cuda")
            table[row, col] = step
            ops.opt8_embedding_forward(ops.make_embedding(ids.cuda(), table, y, scale=0.5))
            ends.append(float((y.cpu().double() * dy.double()).sum()))
        assert float(dt[row, col]) == (ends[0] - ends[1]) / 2


def test_offsets_past_32_bits():
    """Tables whose last rows lie more than 2^32 bytes from the first."""
    vocab, d = (1 << 20) + 5, 2100
    table = torch.zeros(vocab, d, dtype=BF, device="cuda")
    table[-3:] = torch.arange(1, 4, dtype=BF, device="cuda")[:, None]
    ids = torch.tensor([vocab - 1, 0, vocab - 3, vocab - 2, vocab - 1], device="cuda")
    y = torch.empty(5, d, dtype=BF, device="cuda")
    ops.opt8_embedding_forward(ops.make_embedding(ids, table, y))
    assert y[:, 0].tolist() == [3, 0, 1, 2, 3] and bool((y == y[:, :1]).all())
    work = torch.empty(ops.opt8_embedding_workspace(5, vocab, d), dtype=torch.uint8, device="cuda")
    ops.opt8_embedding_backward(ops.make_embedding_grad(ids, y, table, work, accumulate=True))
    assert table[-4:, 5].tolist() == [0, 2, 4, 9] and bool((table[:-3] == 0).all())
    table.fill_(1)
    ops.opt8_embedding_backward(ops.make_embedding_grad(ids, y, table, work))
    assert table[-4:, 2099].tolist() == [0, 1, 2, 6] and float(table.float().sum()) == 9 * d
