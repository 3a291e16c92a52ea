"""Plain 64-bit forms of the training operators, and the error bounds their fp32 kernels
are held to.

u is fp32's unit roundoff.  A sum of n terms in any order is off by at most (n - 1) u times
the sum of the terms' magnitudes; the norm kernels' sums over a row are trees over at most
64 terms per lane, so 80 u covers them at any width.  Every bound ends with the one rounding
of the output: the unit roundoff of bf16 (8 significant bits: 2^-8 of the value) or fp32 (u).
"""
import math

import torch

u = 2.0 ** -24
ROW = 80 * u          # relative error of a sum over a row (of its terms' magnitudes)
HALF = {torch.float32: u, torch.bfloat16: 2.0 ** -8}
TINY = 2.0 ** -126    # what underflow may lose (below fp32's normal range)
F8 = torch.float64


def close(got, want, tol, what=""):
    """|got - want| <= tol, element by element, and NaN exactly where want has it."""
    got, want = got.to(F8), want.to(F8)
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}, not {tuple(want.shape)}"
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    fine = ~(nan | inf)
    over = ((got - want).abs() - tol.expand_as(want))[fine]
    assert not (over > 0).any(), f"{what}: off by {float(over.max()):.3e} more than allowed"


def lookup(table, tokens, scale):
    ok = (tokens >= 0) & (tokens < table.shape[0])
    out = torch.zeros(*tokens.shape, table.shape[1], dtype=F8, device=table.device)
    out[ok] = table.to(F8)[tokens[ok].long()] * scale
    return out, out.abs() * (HALF[table.dtype] + 2 * u) + TINY


def table_gradient(dy, tokens, rows, scale, offsets, padding_idx, old, dtype):
    """[(gradient, bound)] per worker; `old`: what it is added to, or None."""
    dy, tokens = dy.reshape(-1, dy.shape[-1]).to(F8), tokens.reshape(-1).long()
    out = []
    for k in range(len(offsets) - 1):
        t, g = tokens[offsets[k]:offsets[k + 1]], dy[offsets[k]:offsets[k + 1]]
        ok = (t >= 0) & (t < rows)
        if padding_idx is not None:
            ok &= t != padding_idx
        total = torch.zeros(rows, dy.shape[1], dtype=F8, device=dy.device)
        size, count = torch.zeros_like(total), torch.zeros(rows, 1, dtype=F8, device=dy.device)
        total.index_put_((t[ok],), scale * g[ok], accumulate=True)
        size.index_put_((t[ok],), abs(scale) * g[ok].abs(), accumulate=True)
        count.index_put_((t[ok],), torch.ones(int(ok.sum()), 1, dtype=F8, device=dy.device), accumulate=True)
        tol = (count + 3) * u * size
        if old is not None:
            total = total + old[k].reshape(rows, -1).to(F8)
            tol = tol + u * total.abs()
        out.append((total, tol + HALF[dtype] * (total.abs() + tol) + TINY))
    return out


def norm(x, weight, bias, eps):
    """(y, bound), (mean, bound), (rstd, bound), (h, bound), over the last dimension of a matrix."""
    x8 = x.to(F8)
    n = x.shape[1]
    w = torch.ones(n, dtype=F8, device=x.device) if weight is None else weight.to(F8)
    b = torch.zeros(n, dtype=F8, device=x.device) if bias is None else bias.to(F8)
    mean = x8.mean(1, keepdim=True)
    var = (x8 - mean).square().mean(1, keepdim=True)
    r = 1 / torch.sqrt(var + eps)
    h = (x8 - mean) * r
    mean_tol = (ROW + 2 * u) * x8.abs().mean(1, keepdim=True)
    # the variance: each difference off by the mean's error and u (|x| + |mean|), the sum by ROW
    d_tol = mean_tol + u * (x8.abs() + mean.abs())
    var_tol = (ROW + 4 * u) * var + (2 * (x8 - mean).abs() * d_tol + d_tol ** 2).mean(1, keepdim=True)
    r_tol = r * (0.75 * var_tol * r ** 2 + 6 * u)
    h_tol = d_tol * r + (x8 - mean).abs() * r_tol + 2 * u * h.abs()
    y = h * w + b
    y_tol = h_tol * w.abs() + 2 * u * ((h * w).abs() + b.abs())
    return ((y, y_tol + HALF[x.dtype] * (y.abs() + y_tol) + TINY), (mean[:, 0], mean_tol[:, 0] + TINY),
            (r[:, 0], r_tol[:, 0]), (h, h_tol))


def norm_gradient(dy, h, h_tol, rstd, weight, offsets, old_w, old_b, dtype):
    """(dx, bound), [(dw, bound)], [(db, bound)] for h known to h_tol and rstd given."""
    g8, r = dy.to(F8), rstd.to(F8)[:, None]
    n = dy.shape[1]
    w = torch.ones(n, dtype=F8, device=dy.device) if weight is None else weight.to(F8)
    g = g8 * w
    mg, mgh = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    dx = r * (g - mg - h * mgh)
    mg_tol = (ROW + 4 * u) * g.abs().mean(1, keepdim=True)
    mgh_tol = (ROW + 4 * u) * (g * h).abs().mean(1, keepdim=True) + (g.abs() * h_tol).mean(1, keepdim=True)
    dx_tol = r * (mg_tol + (h.abs() + h_tol) * mgh_tol + h_tol * mgh.abs() + 4 * u * (g.abs() + mg.abs() + (h * mgh).abs()))
    dw, db = [], []
    for k in range(len(offsets) - 1):
        part = slice(offsets[k], offsets[k + 1])
        rows = offsets[k + 1] - offsets[k]
        for out, old, terms, extra in ((dw, old_w, g8[part] * h[part], g8[part].abs() * h_tol[part]),
                                       (db, old_b, g8[part], torch.zeros_like(g8[part]))):
            total, tol = terms.sum(0), (rows + 4) * u * terms.abs().sum(0) + extra.sum(0)
            if old is not None:
                total = total + old[k].to(F8)
                tol = tol + u * total.abs()
            out.append((total, tol + HALF[dtype] * (total.abs() + tol) + TINY))
    return (dx, dx_tol + HALF[dy.dtype] * (dx.abs() + dx_tol) + TINY), dw, db


def pack(x):
    """(codes, scales) of a float32 or bfloat16 matrix, bit for bit: fp32 arithmetic on the
    host, where torch's divisions are correctly rounded."""
    x = x.float().cpu()
    rows, cols = x.shape
    nb = -(-cols // 128)
    b = torch.nn.functional.pad(x, (0, nb * 128 - cols)).view(rows, nb, 128)
    top = b.abs().amax(2)
    bad = ~torch.isfinite(b).all(2)
    top = torch.where(bad | (top < 2.0 ** -119), torch.zeros_like(top), top)
    limit = torch.full_like(top, 127.0)
    inv = torch.where(top > 0, limit / top, torch.zeros_like(top))
    codes = torch.round(torch.nan_to_num(b, 0.0, 0.0, 0.0) * inv[:, :, None])
    scales = torch.where(bad, torch.full_like(top, math.nan), top / limit)
    return codes.view(rows, nb * 128)[:, :cols].to(torch.int8), scales


def unpacked(codes, scales, cols):
    """What codes stand for, in 64 bits."""
    wide = scales.to(F8).repeat_interleave(128, 1)[:, :cols]
    return codes[:, :cols].to(F8) * wide


def gelu(x, tanh):
    """(value, slope) in 64 bits."""
    if tanh:
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x ** 3))
        # 1 + t without cancellation where t is near -1
        q = 1 / (1 + torch.exp(-2 * c * (x + 0.044715 * x ** 3)))
        return x * q, q + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)
    q = 0.5 * torch.special.erfc(-x / math.sqrt(2))
    return x * q, q + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)


#: Error of the fp32 normal distribution function (or its tanh form): an erf good to 1.5e-7
#: (Abramowitz and Stegun 7.1.26's bound), halved, and a dozen roundings of values up to 1/2.
PHI = 0.75e-7 + 6 * u
#: The same of the slope: that, and x times the density, below 0.25, to 24 roundings.
SLOPE = PHI + 6 * u
