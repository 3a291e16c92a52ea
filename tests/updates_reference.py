"""The orthogonalised update in 64 bits, and how far the kernels' results may be from it."""
import math

import torch

F8 = torch.float64
QUINTIC = (3.4445, -4.7750, 2.0315)


def orthogonal(x, steps=5, coefficients=QUINTIC, eps=1e-7):
    """The iteration on the matrices of x; coefficients: a triple, or one a step."""
    x = x.to(F8)
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    for a, b, c in ([coefficients] * steps if isinstance(coefficients[0], float) else coefficients):
        p = x @ x.mT
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.mT if tall else x


def bound(x, dtype, steps=5, slope=3.4445):
    """Relative error (of the norm) allowed for a result of `dtype`.

    What a step adds.  fp32: every operand is kept to 2^-22 of its largest values' size (two
    fp16 of 11 bits each), products lose 2^-22 by the term left out, and sums of 512 along the
    depth are cut off 32 times, each by up to 2^-23 of the sum: 2^-18 of a product A; a step
    adds |a| + 3 |b| + 5 |c| (at most 28) such errors weighted by the values' sizes, all at
    most about 1, so 28 * 2^-18 if every one had its largest size and the same sign.  They
    are cut-offs of half that on average, of sums half as large on average, and of the
    terms of one sign only on the diagonal of A: an eighth.  Errors that point into directions
    of small singular values grow by the slope a of every later step, but were small by the
    same factor: directions of the input below 2^-22 of its norm, scaled by sqrt(m) for
    roundings spread over m directions, count as lost.
    bf16: fp16 operands, 2^-12 per rounding (half a step): A, B and the X they multiply give
    three such errors a step, of which the last three steps' remain (earlier ones are
    brought together by the polynomial's flat part): 9 * 2^-12 spread as a root of squares,
    and the result's rounding, 2^-9 on average of at most 2^-8.
    """
    if dtype == torch.float32:
        step = 28 * 2.0 ** -18 / 8
        m = min(x.shape[-2:])
        lost = 2.0 ** -22 * slope ** (steps - 1) / math.sqrt(m)
        return step + lost
    return math.sqrt(9) * 2.0 ** -12 * 3 + 2.0 ** -8


def updates(*shape, gen, strong=0.5, device="cuda:0"):
    """Matrices of a few strong directions over noise, as gradients have."""
    rows, cols = shape[-2:]
    r = max(1, min(rows, cols) // 16)
    left = torch.randn(*shape[:-1], r, generator=gen, device=device) / math.sqrt(r)
    right = torch.randn(*shape[:-2], r, cols, generator=gen, device=device)
    return left @ right + strong * torch.randn(*shape, generator=gen, device=device)
