"""GELU's erf form for fp32 activations: as accurate as fp32 arithmetic allows.

With q = 1/2 erfc(|x| / sqrt 2), gelu = max(x, 0) - |x| q.  The bound on q counts what an fp32
evaluation of exp(-x^2 / 2) times a slowly varying factor H cannot avoid: the exponent's
argument x^2 / 2 after two products and a rounded constant is off by 3 u of itself, 1.5 x^2 u
of the exponential, 2^-22 = 4 u of that the exponential's own; a quotient z = c b / (1 + c b)
is off by 5 u (three roundings and an approximate reciprocal, 2^-23), which H's slope passes
on with a factor of at most 1 + x^2 / 8, and a polynomial of z adds its own roundings, at most
12 u up to |x| = 5 and growing slower than x^2 / 2 from there.  Together (22 + 2 x^2) u."""
import math

import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
import training_reference as ref
from test_gpu_training import DEV, gen, randn
from training_reference import F8, TINY, close, u

pytestmark = pytest.mark.gpu


def tail(x):
    """(q, its bound) in 64 bits."""
    q = 0.5 * torch.special.erfc(x.abs() / math.sqrt(2))
    return q, q * (22 + 2 * x * x) * u * (1 + 2.0 ** -10)


def value(x):
    want, (_, tol) = ref.gelu(x, False)[0], tail(x)
    return want, x.abs() * tol + u * want.abs() * (1 + 2.0 ** -10) + (1 + x.abs()) * TINY


def slope(x):
    """Phi, one rounding of it; x times the density: its constant, two products and the
    exponential; one rounding of their sum."""
    want, (_, tol) = ref.gelu(x, False)[1], tail(x)
    phi = 0.5 * torch.special.erfc(-x / math.sqrt(2))
    rest = x.abs() * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    return want, tol + u * (phi + (7 + 1.5 * x * x) * rest + want.abs()) * (1 + 2.0 ** -10) + (1 + x.abs()) * TINY


@pytest.mark.parametrize("cols", [1024, 1001])
def test_value_and_slope(native, cols):
    x = torch.linspace(-13.5, 13.5, 512 * cols, device=DEV).view(512, cols)
    x[0, :8] = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 3e4, -3e4], device=DEV)
    y, kept = ags.gelu_checkpointed(x)
    close(y, *value(x.to(F8)), "gelu")
    v = ags.checkpoint_unpack(kept)
    dx, again = ags.gelu_checkpointed_backward(torch.ones_like(x), kept, with_output=True)
    close(again, *value(v.to(F8)), "gelu again")
    want, tol = slope(v.to(F8))
    close(dx, want, tol + u * want.abs(), "slope")


def test_small_steps_and_zeros(native):
    """Blocks of one size, so that the values the slope is taken at reach from 0 to each size."""
    top = torch.logspace(-6, 1.1, 4096, device=DEV)[:, None]
    x = top * (2 * torch.rand(4096, 128, generator=gen(1), device=DEV) - 1)
    x[:, 0], x[:, 1] = top[:, 0], 0.0
    _, kept = ags.gelu_checkpointed(x)
    v = ags.checkpoint_unpack(kept)
    dx = ags.gelu_checkpointed_backward(torch.ones_like(x), kept)
    want, tol = slope(v.to(F8))
    close(dx, want, tol + u * want.abs(), "slope")
    assert (dx[v == 0] == 0.5).all()


def test_no_worse_than_elementary_operations(native):
    """On normal activations, the norm of the error against that of the formula in fp32
    operations (an erf good to 2 ulp): about as many roundings, so at most half as much again."""
    x = randn(2048, 1024, seed=5)
    y, kept = ags.gelu_checkpointed(x)
    v = ags.checkpoint_unpack(kept)
    dx = ags.gelu_checkpointed_backward(torch.ones_like(x), kept)
    cdf = lambda t: 0.5 * (1 + torch.erf(t * math.sqrt(0.5)))  # noqa: E731
    for got, plain, want in ((y, x * cdf(x), ref.gelu(x.to(F8), False)[0]),
                             (dx, cdf(v) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi), ref.gelu(v.to(F8), False)[1])):
        assert float((got.to(F8) - want).norm()) <= 1.5 * float((plain.to(F8) - want).norm())
