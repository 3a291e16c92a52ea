"""Orthogonalised updates with steep coefficients: B = b A + c A A leaves what fp16 holds at the
usual scale (16) where singular values stay below 2.8 all the same."""
import math

import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
from updates_reference import F8, orthogonal

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32


def tolerance(dtype, triples):
    """Of a matrix all of whose singular values are 0 or about 1, so that X, A and X's products
    are at most about 1 in norm.  A step rounds X (three times a product b A X, five times c A A X),
    A and B; in bf16 form each to one fp16 number, 2^-11, in fp32 form to two, 2^-22, where each
    of the three products also leaves out 2^-22 and cuts off few (at most 8) sums by 2^-23.  What a
    step gets wrong is multiplied by the next steps' slopes: a in new directions, |a + 3 b + 5 c| in
    the old one."""
    r = 2.0 ** -11 if dtype == BF16 else 2.0 ** -22
    more = 0 if dtype == BF16 else 5
    total = 0.0
    for a, b, c in triples:
        total = total * max(abs(a), abs(a + 3 * b + 5 * c)) + r * (abs(a) + (5 + 2 * more) * abs(b) + (8 + 3 * more) * abs(c))
    return total + (2.0 ** -8 if dtype == BF16 else 2.0 ** -23)


def check(x, triples):
    for dtype in (BF16, FP32):
        y = x.to(dtype)
        want = orthogonal(y, len(triples), triples, 0.0)
        got = ags.orthogonalize(y, steps=len(triples), coefficients=triples, eps=0.0)
        assert torch.isfinite(got).all()
        assert float((got.to(F8) - want).norm()) <= tolerance(dtype, triples) * max(1.0, float(want.norm()))
    assert ags.get_last_error() == 0


STEEP = [(20.0, -19.0, 0.0), (50.0, -49.0, 0.0), (16.0, -60.0, 45.0), (-400.0, 0.0, 401.0), (1.0, 2000.0, -2000.0)]


@pytest.mark.parametrize("triple", STEEP)
@pytest.mark.parametrize("rows,cols", [(1, 16), (2, 24), (24, 2), (3, 200)])
def test_one_direction(native, rows, cols, triple):
    """Equal rows: one singular value, of 1, and elements of B of b + c over the number of rows."""
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    small, large = min(rows, cols), max(rows, cols)
    x = torch.randn(1, large, generator=g, device=DEV).expand(small, large)
    check((x if rows <= cols else x.t()).contiguous(), [triple])


@pytest.mark.parametrize("triple", STEEP)
def test_one_element(native, triple):
    x = torch.zeros(5, 70, device=DEV)
    x[3, 68] = -0.01
    check(x, [triple])


@pytest.mark.parametrize("triples", [[(1.5, -0.5, 0.0), (20.0, -19.0, 0.0), (1.5, -0.5, 0.0)],
                                     [(20.0, -19.0, 0.0), (50.0, -49.0, 0.0), (1.5, -0.5, 0.0), (1.5, -0.5, 0.0)]])
def test_steep_steps_among_others(native, triples):
    x = torch.zeros(5, 70, device=DEV)
    x[1, 30] = 7.0
    check(x, triples)
    check(torch.ones(2, 64, device=DEV), triples)


def test_steps_of_weights(native):
    """The same through the step: a matrix whose update has one direction."""
    g = torch.ones(2 * 64, device=DEV)
    w, v = torch.zeros(128, device=DEV), torch.zeros(128, device=DEV)
    ags.muon_step(g, [0, 128], [(2, 64)], w, v, lr=1.0, mu=0.0, steps=1, coefficients=(50.0, -49.0, 0.0), eps=0.0, scale=None)
    want = -1 / math.sqrt(128)
    assert float((w.double() - want).norm()) <= tolerance(FP32, [(50.0, -49.0, 0.0)])
