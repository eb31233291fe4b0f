"""64-bit forms of the operators in opt8_layers.h, and the error bounds their tests hold the
kernels to (before the last rounding; products_reference.rounded adds that one).

U = 2^-24 is half a step of fp32.  Each fp32 operation is off by at most U of its result; a sum of
terms along a path of k additions by at most k * U of the sum of the magnitudes.
"""

import torch

import products_reference as ref

U = 2.0 ** -24


def embedding(ids, table, scale, place_ids=None, place_table=None):
    """y and its bound: one rounding of the product, one of the sum."""
    def rows(i, t):
        there = (i >= 0) & (i < t.shape[0])
        out = torch.zeros(len(i), t.shape[1], dtype=torch.float64)
        out[there] = t.double()[i[there].long()]
        return out
    y = rows(ids, table) * scale
    err = U * y.abs()
    if place_ids is not None:
        y = y + rows(place_ids, place_table)
        err = err + U * (y.abs() + err)
    return y, err


def embedding_grad(ids, dy, vocab, scale, old=None):
    """The table's gradient and its bound: a sum of n terms in any order (n - 1 additions), the
    product with scale, and the addition to what was there."""
    there = (ids >= 0) & (ids < vocab)
    at = ids[there].long()
    d = dy.double()[there]
    total = torch.zeros(vocab, dy.shape[1], dtype=torch.float64).index_add_(0, at, d)
    size = torch.zeros_like(total).index_add_(0, at, d.abs())
    n = torch.bincount(at, minlength=vocab)[:, None]
    want, err = total * scale, (n + 1) * U * size * abs(scale)
    if old is not None:
        want = want + old.double()
        err = torch.where(n > 0, err + U * (want.abs() + err), torch.zeros_like(err))
    return want, err


def depth(d):
    """Additions on the longest path of a sum over a row: at most 64 in a lane that holds its share
    (8 for each 8192 columns where rows are read twice), then 4 among 16 lanes, 2 among four such
    groups and 15 among the waves."""
    return 96 + d // 1024


def norm(x, weight, eps, residual=None):
    """dict of (value, bound) for sum, n, rstd.

    t is off by U of itself; the sum of squares by 2U + depth U (all terms are positive), its product
    with the rounded 1/d and the addition of eps by 3U more; the root halves that and adds U, the
    division U; n takes t's, rstd's and two products' errors.  1.01 covers the terms of second order."""
    t = x.double() + (residual.double() if residual is not None else 0.0)
    d = x.shape[1]
    rstd = (t.square().mean(1) + eps) ** -0.5
    er = 1.01 * U * ((depth(d) + 5) / 2 + 2)
    n = t * rstd[:, None] * weight.double()
    return dict(sum=(t, U * t.abs()), rstd=(rstd, er * rstd), n=(n, (er + 3 * U) * 1.01 * n.abs()))


def norm_grad(dy, x, weight, rstd, dsum=None):
    """dx and dweight with their bounds.  h and g are off by U of themselves, so the mean of their
    products by depth + 2 of them and two roundings more; then one operation after the other.
    dweight: a term is off by U, a column's path has at most rows additions, and no more than
    rows / 64 in a workgroup (rows / 8 of few long rows), 16 among its groups of rows, 4 and 7 in the second kernel."""
    dy, x, w, r = dy.double(), x.double(), weight.double(), rstd.double()[:, None]
    rows, d = x.shape
    h, g = x * r, dy * w
    c = (g * h).mean(1, keepdim=True)
    ec = (depth(d) + 5) * U * (g * h).abs().mean(1, keepdim=True)
    inner = g - c * h
    err = r * (U * g.abs() + ec * h.abs() + 2 * U * (c * h).abs() + U * inner.abs() + U * inner.abs())
    dx = r * inner
    if dsum is not None:
        dx = dx + dsum.double()
        err = err + U * dx.abs()
    path = min(rows, rows // 8 + 1 if rows <= 512 else rows // 64 + 1) + 32
    dw = (dy * h).sum(0)
    return (dx, 1.01 * err), (dw, (path + 2) * U * (dy * h).abs().sum(0))


def check(name, got, want, err, dtype=None):
    dtype = dtype or got.dtype
    worst = ref.worst(got, want.cpu(), ref.rounded(want, err, dtype).cpu())
    assert worst <= 1.0, f"{name}: error is {worst} times its bound"


def room(rows, cols, dtype, extra=0, fill=77.0, head=0):
    """[rows, cols] on the GPU with `extra` elements between rows, a row behind, `head` elements
    before it, and `fill` wherever nothing belongs to it."""
    ld = cols + extra
    store = torch.full(((rows + 1) * ld + head,), fill, dtype=dtype, device="cuda")
    return store, store[head:head + rows * ld].view(rows, ld)[:, :cols] if rows else store[:0].view(0, cols)


def untouched(store, view, fill=77.0):
    """Whether all of the store but the view still holds `fill`."""
    if view.numel() == 0:
        return bool((store == fill).all())
    mask = torch.ones_like(store, dtype=torch.bool)
    torch.as_strided(mask, view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool((store[mask] == fill).all())
