"""The 64-bit forms of products_reference on the tensors' own device, for sizes that are too long
for the CPU: the same formulas and bounds (torch's double precision, no kernel of this package)."""

import torch

import products_reference as ref


def worst(got, want, bound, kind):
    """The largest error in units of the bound that includes the rounding to `kind`."""
    b = ref.rounded(want, bound, kind)
    d = (got.double() - want).abs() / b
    return float("inf") if bool(torch.isnan(d).any()) else float(d.max())


def decode(codes, scale, tile):
    rows, cols = codes.shape
    s = scale.double()[torch.arange(cols, device=codes.device) // ref.BLOCK]
    s = s[:, torch.arange(rows, device=codes.device) // ref.BLOCK] if tile else s
    return codes.float().double() * s.t()


def product(a, sa, b, sb, tile):
    """The product and its bound, as products_reference.product derives it."""
    k = a.shape[1]
    x, y = decode(a, sa, False), decode(b, sb, tile)
    pad = -k % 8
    ax = torch.nn.functional.pad(x.abs(), (0, pad)).view(x.shape[0], -1, 8)
    ay = torch.nn.functional.pad(y.abs(), (0, pad)).view(y.shape[0], -1, 8)
    cut = torch.zeros(x.shape[0], y.shape[0], dtype=torch.float64, device=a.device)
    for g in range(ax.shape[1]):
        top = ax[:, g, 0, None] * ay[None, :, g, 0]
        for j in range(1, 8):
            top = torch.maximum(top, ax[:, g, j, None] * ay[None, :, g, j])
        cut += top
    return x @ y.t(), cut * 7 * 2.0 ** -13 + (x.abs() @ y.abs().t()) * (ref.gamma(k) + 4 * 2.0 ** -24)


ACT_ERR = 2.0 ** -20      # the activation's value, relative: fast exponential and reciprocal


def gated(x, wg, wu, act):
    """h, g, u and bounds of their fp32 forms (slopes are at most 1.13 in magnitude)."""
    X, G, U = (t.double() for t in (x, wg, wu))
    g, u = X @ G.t(), X @ U.t()
    eg, eu = ((X.abs() @ t.abs().t()) * ref.gamma(x.shape[1]) for t in (G, U))
    v, _ = ref.act(g, act)
    ev = 1.13 * eg + ACT_ERR * (v.abs() + 2.0 ** -20 * g.abs())
    return (v * u, g, u), (ev * (u.abs() + eu) + v.abs() * eu + 2.0 ** -24 * (v * u).abs(), eg, eu)


def gated_grad(dh, x, wg, wu, g, u, act, dtype):
    """dx, dw_gate, dw_up and bounds of their fp32 forms from dg, du rounded once to `dtype`: slopes
    within 2^-18, values within 2^-18 of themselves, sums within gamma of the magnitudes."""
    H, X, G, U, g, u = (t.double() for t in (dh, x, wg, wu, g, u))
    v, s = ref.act(g, act)
    dg, du = H * u * s, H * v
    eg = ref.rounded(dg, (H * u).abs() * 2.0 ** -18 + 4 * 2.0 ** -24 * dg.abs(), dtype)
    eu = ref.rounded(du, H.abs() * (v.abs() * 2.0 ** -18 + g.abs() * 2.0 ** -30) + 4 * 2.0 ** -24 * du.abs(), dtype)
    ag, au = dg.abs() + eg, du.abs() + eu
    n, f = H.shape
    aG, aU, aX = G.abs(), U.abs(), X.abs()
    ex = eg @ aG + eu @ aU + (ag @ aG + au @ aU) * ref.gamma(2 * f + 128)
    ewg, ewu = (e.t() @ aX + (m.t() @ aX) * ref.gamma(n) for e, m in ((eg, ag), (eu, au)))
    return (dg @ G + du @ U, dg.t() @ X, du.t() @ X), (ex, ewg, ewu)
