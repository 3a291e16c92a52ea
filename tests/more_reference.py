"""Plain 64-bit forms of the root-mean-square norm and the relative position bias, and the
error bounds their fp32 kernels are held to (training_reference.py has the conventions)."""
import math

import torch

from training_reference import F8, HALF, ROW, TINY, u


def rms(x, weight, eps, residual=None):
    """(total, bound), (y, bound), (rstd, bound), (h, bound); the last three of the rounded total."""
    x8 = x.to(F8) if residual is None else x.to(F8) + residual.to(F8)
    # the sum in fp32, then rounded to the type: bf16 twice
    total = (x8, x8.abs() * (HALF[x.dtype] + u) + TINY)
    t = x8.float().to(x.dtype).to(F8)
    w = torch.ones(x.shape[1], dtype=F8, device=x.device) if weight is None else weight.to(F8)
    sq = t.square().mean(1, keepdim=True)
    r = 1 / torch.sqrt(sq + eps)
    # the squares' sum off by ROW, the mean and eps by 2 u; half of that in the root; 4 u for the
    # root and the quotient
    r_tol = r * (0.5 * (ROW + 2 * u) + 4 * u)
    h = t * r
    h_tol = t.abs() * r_tol + u * h.abs()
    y = h * w
    y_tol = h_tol * w.abs() + u * y.abs()
    return total, (y, y_tol + HALF[x.dtype] * (y.abs() + y_tol) + TINY), (r[:, 0], r_tol[:, 0]), (h, h_tol)


def rms_gradient(dy, h, h_tol, rstd, weight, past, offsets, old, dtype):
    """(dx, bound), [(dw, bound)] for h known to h_tol and rstd given."""
    g8, r = dy.to(F8), rstd.to(F8)[:, None]
    w = torch.ones(dy.shape[1], dtype=F8, device=dy.device) if weight is None else weight.to(F8)
    g = g8 * w
    mgh = (g * h).mean(1, keepdim=True)
    dx = r * (g - h * mgh)
    mgh_tol = (ROW + 4 * u) * (g * h).abs().mean(1, keepdim=True) + (g.abs() * h_tol).mean(1, keepdim=True)
    tol = r * ((h.abs() + h_tol) * mgh_tol + h_tol * mgh.abs() + 4 * u * (g.abs() + (h * mgh).abs()))
    if past is not None:
        dx = dx + past.to(F8)
        tol = tol + u * (dx.abs() + past.to(F8).abs())
    dw = []
    for k in range(len(offsets) - 1):
        part = slice(offsets[k], offsets[k + 1])
        terms, rows = g8[part] * h[part], offsets[k + 1] - offsets[k]
        total = terms.sum(0)
        t = (rows + 4) * u * terms.abs().sum(0) + (g8[part].abs() * h_tol[part]).sum(0)
        if old is not None:
            total = total + old[k].to(F8)
            t = t + u * total.abs()
        dw.append((total, t + HALF[dtype] * (total.abs() + t) + TINY))
    return (dx, tol + HALF[dy.dtype] * (dx.abs() + tol) + TINY), dw


def bucket(rel, buckets, both, distance):
    """The bucket of one relative position, in whole numbers."""
    n = buckets // 2 if both else buckets
    d = abs(rel) if both else max(0, -rel)
    e = n // 2
    if d < e:
        j = d
    else:
        j = e
        # ((n - e) ln(d / e) >= i ln(distance / e)) as powers of whole numbers
        while j < n - 1 and d ** (n - e) * e ** (j + 1 - e) >= distance ** (j + 1 - e) * e ** (n - e):
            j += 1
    return j + (n if both and rel > 0 else 0)


def bucket_matrix(queries, keys, offset, buckets, both, distance, device):
    """Buckets of (query, key)."""
    lo = -(queries - 1) - offset
    of = torch.tensor([bucket(lo + i, buckets, both, distance) for i in range(queries + keys - 1)], dtype=torch.int64, device=device)
    return of[torch.arange(keys, device=device)[None, :] - torch.arange(queries, device=device)[:, None] + queries - 1]


def bias_gradient(d, index, buckets, offsets, old, dtype):
    """[(gradient, bound)] per worker, each buckets x heads.  A value is added once in a sum of at
    most as many terms as its bucket has; the additions of partial sums are among them."""
    out = []
    heads = d.shape[1]
    flat = index.flatten()
    for k in range(len(offsets) - 1):
        x = d[offsets[k]:offsets[k + 1]].to(F8)
        rows = x.transpose(0, 1).reshape(heads, x.shape[0], d.shape[2] * d.shape[3])
        total = torch.zeros(buckets, heads, dtype=F8, device=d.device)
        size = torch.zeros_like(total)
        total.index_add_(0, flat, rows.sum(1).t())
        size.index_add_(0, flat, rows.abs().sum(1).t())
        count = torch.bincount(flat, minlength=buckets)[:, None] * x.shape[0]
        # a unit's running sum has at most 256 * 16 terms, 16 of them short sums, then 512 slots,
        # then partial sums: never more additions than terms, nor than 2^13 and the units
        adds = torch.minimum(count, torch.full_like(count, 1 << 13) + count // 4096)
        tol = (adds + 8) * u * size
        if old is not None:
            total = total + old[k].view(buckets, heads).to(F8)
            tol = tol + u * total.abs()
        out.append((total, tol + HALF[dtype] * (total.abs() + tol) + TINY))
    return out
