"""Waits of the iteration that run out: the call ends with a status, and the next one is right."""
import time

import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
from updates_reference import bound, orthogonal, updates

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


@pytest.mark.parametrize("steps", [1, 3])
@pytest.mark.parametrize("tile", ["0", "1", "2"])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_a_product_that_is_never_ready(native, hooks, monkeypatch, dtype, tile, steps):
    """From the second step on (of one: from the first) no tile finds its matrix's last product
    written (injected on the host), by which time earlier ones have been copied and multiplied.  All
    waits end after their clock budget, the status says so once, and the context stays usable."""
    monkeypatch.setenv("ADASUM_UPDATE_TILE", tile)
    x = updates(5, 600, 900, gen=gen(1)).to(dtype)
    want = ags.orthogonalize(x, steps=steps)
    torch.cuda.synchronize()
    assert ags.get_last_error() == ags.Status.OK
    monkeypatch.setenv("ADASUM_FAULT_INJECT", "timeout")
    began = time.monotonic()
    ags.orthogonalize(x, steps=steps)
    torch.cuda.synchronize()
    assert time.monotonic() - began < 1.0  # (some milliseconds, were the machine idle)
    monkeypatch.delenv("ADASUM_FAULT_INJECT")
    assert ags.get_last_error() == ags.Status.ERR_TIMEOUT
    assert ags.get_last_error() == ags.Status.OK
    got = ags.orthogonalize(x, steps=steps)
    torch.cuda.synchronize()
    assert ags.get_last_error() == ags.Status.OK
    assert torch.equal(got, want)
    off = float((got.double() - orthogonal(x, steps)).norm() / orthogonal(x, steps).norm())
    assert off <= bound(x, dtype, steps)


def test_a_step_that_is_never_ready(native, hooks, monkeypatch):
    shapes = [(300, 200), (64, 500)]
    offs = [0, 60000, 92000]
    g = torch.randn(offs[-1], generator=gen(2), device=DEV)
    w, v = torch.zeros_like(g), torch.zeros_like(g)
    monkeypatch.setenv("ADASUM_FAULT_INJECT", "timeout")
    ags.muon_step(g, offs, shapes, w.clone(), v.clone(), lr=0.1)
    torch.cuda.synchronize()
    assert ags.get_last_error() == ags.Status.ERR_TIMEOUT
    monkeypatch.delenv("ADASUM_FAULT_INJECT")
    a = ags.muon_step(g, offs, shapes, w.clone(), v.clone(), lr=0.1)
    b = ags.muon_step(g, offs, shapes, w.clone(), v.clone(), lr=0.1)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[0].isfinite().all() and a[0].any()
    assert ags.get_last_error() == ags.Status.OK
