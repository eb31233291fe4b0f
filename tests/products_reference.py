"""Plain 64-bit forms of the operators in opt8_products.h, and the error bounds the
tests hold the kernels to.

Bounds.  u(t) = finfo(t).eps / 2 is half a step of a type relative to the value.
A sum of n products in fp32 is off by at most n * 2^-24 * sum|terms| in any order
(each product is exact or rounded once, each addition once); with the products'
own rounding, gamma(n) = (n + 2) * 2^-24.  The matrix cores add in fp32 too.
"""

import numpy as np
import torch

BLOCK = 128
FMAX = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}


def half_step(t):
    return torch.finfo(t).eps / 2


def gamma(n):
    return (n + 2) * 2.0 ** -24


def ceil128(n):
    return -(-n // BLOCK)


def quantize(x, kind, tile):
    """Scales as float32 and codes by the definition, on the CPU: s = max(max|x|/fmax, 2^-126),
    code = nearest(x * (1/s)); every operation is one fp32 rounding (numpy float32)."""
    x = x.detach().cpu().float().numpy()
    rows, cols = x.shape
    nr = ceil128(rows) if tile else rows
    scale = np.zeros((ceil128(cols), nr), np.float32)
    codes = torch.zeros(rows, cols, dtype=torch.uint8)
    with np.errstate(all="ignore"):
        for b in range(ceil128(cols)):
            for i in range(nr):
                rs = slice(BLOCK * i, BLOCK * i + BLOCK) if tile else slice(i, i + 1)
                part = x[rs, BLOCK * b:BLOCK * b + BLOCK]
                mags = np.abs(part[~np.isnan(part)])
                top = np.float32(mags.max()) if mags.size else np.float32(0)
                s = max(np.float32(top / np.float32(FMAX[kind])), np.float32(2.0 ** -126))
                scale[b, i] = s
                q = torch.from_numpy((part * np.float32(np.float32(1) / s)).astype(np.float32)).to(kind)
                codes[rs, BLOCK * b:BLOCK * b + BLOCK] = q.view(torch.uint8)
    return codes, torch.from_numpy(scale)


def decode(codes, scale, tile):
    """float64 values; scale [blocks, rows or row blocks]."""
    rows, cols = codes.shape
    s = scale.double().cpu()[torch.arange(cols) // BLOCK]
    s = s[:, torch.arange(rows) // BLOCK] if tile else s
    return codes.cpu().float().double() * s.t()


def product(a, sa, b, sb, tile):
    """The product in 64 bits, and the bound of the kernels' form before the final rounding.

    Within a block the 8-bit matrix instruction cuts each of 8 products (8 consecutive k) to a
    grid of 2^-13 of the largest one's power of two: at most 7 terms lose less than 2^-13 of
    max|term| each (the largest itself has 8 bits).  The rest is fp32: sums of n terms, the
    scales' product, and its product with a block's sum, one rounding each."""
    k = a.shape[1]
    x, y = decode(a, sa, False), decode(b, sb, tile)
    pad = -k % 8
    ax = torch.nn.functional.pad(x.abs(), (0, pad)).view(x.shape[0], -1, 8)
    ay = torch.nn.functional.pad(y.abs(), (0, pad)).view(y.shape[0], -1, 8)
    cut = torch.zeros(x.shape[0], y.shape[0], dtype=torch.float64)
    for g in range(ax.shape[1]):
        top = ax[:, g, 0, None] * ay[None, :, g, 0]
        for j in range(1, 8):
            top = torch.maximum(top, ax[:, g, j, None] * ay[None, :, g, j])
        cut += top
    return x @ y.t(), cut * 7 * 2.0 ** -13 + (x.abs() @ y.abs().t()) * (gamma(k) + 4 * 2.0 ** -24)


def act(g, kind):
    """Value and slope in 64 bits."""
    if kind == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    if kind == "gelu":
        p = torch.special.erfc(-g * np.sqrt(0.5)) / 2     # (1 + erf)/2 cancels far below zero
        return g * p, p + g * torch.exp(-g * g / 2) / np.sqrt(2 * np.pi)
    # (1 + tanh y)/2 = sigmoid(2y), which does not cancel far below zero
    c = np.sqrt(2 / np.pi)
    p = torch.sigmoid(2 * c * (g + 0.044715 * g ** 3))
    return g * p, p + 2 * g * p * (1 - p) * c * (1 + 3 * 0.044715 * g * g)


def rounded(want, bound, kind):
    """Bound after one rounding to `kind`: half a step of the value (with the error before it),
    or half the type's smallest number where it is subnormal."""
    return bound + half_step(kind) * (want.abs() + bound) + torch.finfo(kind).smallest_normal * half_step(kind)


def worst(got, want, bound):
    """The largest error in units of its bound; NaN anywhere counts as infinite.  Where the bound
    reaches the value that rounds to infinity (the largest number and half a step of it), an
    infinity of that sign is the result too."""
    if got.numel() == 0:
        return 0.0
    g = got.double().cpu()
    top = torch.finfo(got.dtype).max * (1 + torch.finfo(got.dtype).eps / 4)
    over = torch.isinf(g) & (g.sign() == want.sign()) & (want.abs() + bound >= top)
    d = (g - want).abs() / bound.clamp_min(1e-300)
    d = torch.where((g == want) | over, torch.zeros_like(d), d)
    return float("inf") if bool(torch.isnan(d).any()) else float(d.max())
