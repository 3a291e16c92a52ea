"""How near bf16 results come, besides the rounding of their elements: 2^-9 of the norm, as
include/adasum.h says.  The two errors are independent, so that they add as a root of squares.

What there is to be off by, in parts of the norm: a step's product has X rounded to 11 bits, on
average by 2^-11 / sqrt(12) = 1.4e-4, B's elements off the diagonal likewise and, by X's products,
A's; these meet B off the diagonal, of a norm of about 1 at most where singular values lie between
0.7 and 1.2 (b s^2 + c s^4 between -1.8 and -2.8, less its mean on the diagonal), slopes of A of
|b + 2 c s^2| up to 3.8: some 4e-4 a step, whose five add up to about 9e-4 if none is brought together, and
the linear term's rounding in the last two steps, 3.4 * 1.4e-4 = 4.8e-4 each: 1.1e-3 in all.  With A's and B's
diagonals in 11 bits too, a step has |b s^2 + c s^4| * 1.4e-4 more of each: results off by up to 2.8e-3."""
import math

import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
from test_gpu_update_tiles import in_fp32, matrices, off, tile  # noqa: F401 (a fixture)
from updates_reference import orthogonal

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("rows,cols", [(64, 64), (24, 4099), (129, 300), (300, 700), (700, 300), (517, 1000), (1111, 777), (1024, 4096)])
@pytest.mark.parametrize("kind", ["random", "loud", "power", "flat"])
def test_bf16_results(native, tile, kind, rows, cols):
    x = matrices(kind, 2, rows, cols).to(BF16)
    for steps in (1, 3, 5):
        want = orthogonal(x, steps)
        rounding = off(want.to(BF16), want)
        errors = off(ags.orthogonalize(x, steps=steps), want)
        assert all(e <= math.hypot(2.0 ** -9, r) for e, r in zip(errors, rounding)), f"steps {steps}: {errors}, rounding {rounding}"


def test_the_product_as_it_is(native):
    """The tiles that it takes by itself, of a large batch and of a single large matrix."""
    for batch, rows, cols in ((16, 300, 700), (12, 1024, 512), (1, 3000, 2500)):
        x = matrices("random", batch, rows, cols).to(BF16)
        want = orthogonal(x)
        assert all(e <= math.hypot(2.0 ** -9, r) for e, r in zip(off(ags.orthogonalize(x), want), off(want.to(BF16), want)))


@pytest.mark.parametrize("batch,rows,cols", [(11, 2, 1), (10, 2, 3), (10, 4, 7), (10, 9, 3), (6, 8, 8), (4, 16, 16), (4, 31, 31), (2, 59, 17), (3, 5, 200)])
def test_few_elements(native, tile, batch, rows, cols):
    """Whose errors do not average: computed as fp32 results are, by at most twice fp32's error and
    2^-22, which the rounding may add twice where it moves a value over a rounding's border."""
    x = matrices("random", batch, rows, cols).to(BF16)
    for steps in (1, 3, 5, 7):
        want = orthogonal(x, steps)
        rounding, plain = off(want.to(BF16), want), off(in_fp32(x.float(), steps), want)
        errors = off(ags.orthogonalize(x, steps=steps), want)
        assert all(e <= r + 2 * (2 * p + 2.0 ** -22) for e, r, p in zip(errors, rounding, plain)), f"steps {steps}"
