"""Orthogonalised updates of matrices whose norm is far below eps: X starts far below 1, where fp16
holds few of its bits, and grows by the slope of every step."""
import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
from test_gpu_update_tiles import check, gen, in_fp32, matrices, off, tile  # noqa: F401 (a fixture)
from updates_reference import F8, orthogonal, updates

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
TYPES = [BF16, FP32]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(200, 300), (513, 260)])
def test_norms_below_eps(native, tile, rows, cols, dtype):
    """eps is 1e-7, about 2^-23; the matrices' norms are about 2^7 times the power."""
    x = matrices("loud", 1, rows, cols)
    for power in (-24, -28, -30, -31, -32, -34, -37, -40, -43, -47, -50, -60, -80, -100, -110):
        y = (x * 2.0 ** power).to(dtype)
        for steps in (1, 2, 5):
            check(y, steps)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_batch_of_many_norms(native, tile, dtype):
    """Each matrix by its own norm, zeros and NaN among them."""
    x = matrices("random", 24, 65, 130)
    x *= 2.0 ** -(5.0 * torch.arange(24, device=DEV))[:, None, None]
    x = x.to(dtype)
    x[7] = 0
    x[11, 3, 4] = float("nan")
    got = ags.orthogonalize(x)
    assert not got[7].any() and torch.isnan(got[11]).all()
    keep = [i for i in range(24) if i not in (7, 11)]
    check(x[keep], got=got[keep])


def test_far_more_steps_than_it_takes(native, tile):
    """From far below 1 up to it, and on."""
    x = matrices("random", 1, 100, 260) * 2.0 ** -60
    triples = [(3.4445, -4.7750, 2.0315)] * 30 + [(1.875, -1.25, 0.375)] * 8
    got = ags.orthogonalize(x, steps=38, coefficients=triples)
    assert off(got, orthogonal(x, 38, triples))[0] < 1e-4
    assert float((torch.linalg.svdvals(got.double()) - 1).abs().max()) < 1e-4


@pytest.mark.parametrize("triples", [[(0.25, 0.0, 0.0)] * 3, [(100.0, -99.0, 0.0), (2.0, -1.0, 0.0)], [(0.0, 3.0, -2.0)] * 2, [(-5.0, 4.0, 0.0)] * 4])
def test_other_slopes(native, tile, triples):
    """Steps that shrink X, that make it grow much, or that have no linear term, as long as its singular
    values stay below 2.8, as they have to."""
    x = matrices("random", 2, 70, 90)
    tried = 0
    for power in (0, -30, -36, -45):
        y = x * 2.0 ** power
        if any(float(torch.linalg.svdvals(orthogonal(y, k, triples[:k])).max()) >= 2.8 for k in range(1, len(triples))):
            continue
        tried += 1
        want = orthogonal(y, len(triples), triples)
        got = ags.orthogonalize(y, steps=len(triples), coefficients=triples)
        # a step's roundings, 2^-22 of its terms each, and 8 cut-offs of 2^-23 a sum, times later slopes
        r, total = 2.0 ** -22, 0.0
        for a, b, c in triples:
            total = total * max(1.0, abs(a)) + r * (abs(a) + 15 * abs(b) + 23 * abs(c))
        # of no linear term: cubes, whose norm may be far below what is held of A and X
        floor = 0.0 if all(a != 0 for a, _, _ in triples) else 2.0 ** -24
        assert float((got.double() - want).norm()) <= total * max(1.0, 1.0 / abs(triples[0][0] or 1.0)) * float(want.norm()) + floor
    assert tried >= 2


@pytest.mark.parametrize("power", [-100, -126, -130, -140])
def test_the_smallest_numbers(native, power):
    """Without eps their scale does not matter, down to fp32's subnormal numbers."""
    x = (updates(40, 72, gen=gen(5)) * 2.0 ** power)
    assert x.any()
    usual = x.double().mul(2.0 ** -power)[None]  # (exact; fp32 throughout is measured there, where an eps of 1e-7 is nothing)
    plain = off(in_fp32(usual.float(), 5), orthogonal(usual))[0]
    assert off(ags.orthogonalize(x, eps=0.0)[None], orthogonal(x, eps=0.0)[None])[0] <= 2 * plain + 2.0 ** -22


def test_weights_of_a_vanishing_gradient(native):
    """A step whose matrix has all but no gradient moves its weights by that little."""
    shapes, offs = [(64, 96), (96, 64)], [0, 6144, 12288]
    g = torch.randn(12288, generator=gen(1), device=DEV)
    g[6144:] *= 1e-14
    w, v = torch.zeros(12288, device=DEV), torch.zeros(12288, device=DEV)
    ags.muon_step(g, offs, shapes, w, v, lr=1.0, mu=0.0, scale=None)
    for s, shape in enumerate(shapes):
        part = slice(offs[s], offs[s + 1])
        want = -orthogonal(g[part].view(1, *shape))
        plain = off(-in_fp32(g[part].view(1, *shape), 5), want)[0]
        assert off(w[part].view(1, *shape), want)[0] <= 2 * plain + 2.0 ** -22
