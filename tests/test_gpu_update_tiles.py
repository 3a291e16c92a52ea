"""Each of the iteration's six kernels (three tile sizes for each type of result) against the
iteration in 64 bits.  Which one a call takes follows from its sizes, so the test build is made to
take each of them for every size here.

What a result may be off by is what include/adasum.h promises.  fp32: twice what the same iteration
in fp32 throughout is off by, and 2^-22, to which operands are kept.  bf16: 2^-8 of the norm
(the most that the rounding of its elements can be), besides that rounding itself, whose error is
added as a root of squares, being independent of the other."""
import math

import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
from updates_reference import F8, QUINTIC, orthogonal, updates

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
TYPES = [BF16, FP32]


@pytest.fixture(params=[0, 1, 2], ids=["pairs", "128", "64"])
def tile(request, hooks, monkeypatch):
    """0: pairs of CTAs, 256 x 256 (bf16) or 256 x 128 tiles; 1: 128 x 128; 2: 128 x 64."""
    monkeypatch.setenv("ADASUM_UPDATE_TILE", str(request.param))
    return request.param


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def in_fp32(x, steps):
    """The same iteration in fp32 throughout."""
    assert not torch.backends.cuda.matmul.allow_tf32
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + 1e-7)
    a, b, c = QUINTIC
    for _ in range(steps):
        p = x @ x.mT
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.mT if tall else x


def off(got, want):
    assert got.shape == want.shape
    assert torch.isfinite(got).all()
    return [float((g.to(F8) - w).norm() / w.norm()) for g, w in zip(got.view(-1, *got.shape[-2:]), want.view(-1, *want.shape[-2:]))]


def check(x, steps=5, got=None):
    """Every matrix of the batch by itself."""
    want = orthogonal(x, steps)
    got = ags.orthogonalize(x, steps=steps) if got is None else got
    errors = off(got, want)
    if x.dtype == BF16:
        allowed = [math.hypot(2.0 ** -8, r) for r in off(want.to(BF16), want)]
    else:
        allowed = [2 * e + 2.0 ** -22 for e in off(in_fp32(x, steps), want)]
    assert all(e <= t for e, t in zip(errors, allowed)), f"{errors} of {allowed}"
    torch.cuda.synchronize()
    assert ags.get_last_error() == ags.Status.OK


def matrices(kind, batch, rows, cols):
    g = gen(rows + cols)
    if kind == "loud":
        return updates(batch, rows, cols, gen=g)
    x = torch.randn(batch, rows, cols, generator=g, device=DEV)
    if kind == "random":
        return x
    small, large = min(rows, cols), max(rows, cols)
    q = torch.linalg.qr(torch.randn(batch, large, small, generator=g, device=DEV, dtype=F8))[0]
    if kind == "power":
        other = torch.linalg.qr(torch.randn(batch, small, small, generator=g, device=DEV, dtype=F8))[0]
        q = (q / torch.arange(1, small + 1, device=DEV, dtype=F8)) @ other
    return (q if rows >= cols else q.mT).float().contiguous()


# Remainders of rows and columns in tiles of 64, 128 and 256, on both sides of a boundary; wide and
# tall; depths of less than one stage, of one run of sums (512 for A, 1024 for the others) and of several; batches
SIZES = [(1, 5, 7), (2, 63, 129), (1, 129, 65), (3, 127, 300), (2, 255, 257), (1, 513, 300), (2, 257, 513), (3, 300, 700),
         (2, 1000, 517), (1, 777, 1111), (1, 1111, 777), (1, 24, 4099), (1, 200, 5000), (1, 1100, 2050), (1, 2050, 1100), (1, 1025, 1090)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,rows,cols", SIZES)
def test_sizes(native, tile, batch, rows, cols, dtype):
    x = matrices("loud", batch, rows, cols).to(dtype)
    check(x)
    check(x, steps=1)
    check(x, steps=2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(300, 129), (517, 1000), (1111, 777), (1024, 4096)])
@pytest.mark.parametrize("kind", ["random", "power", "flat"])
def test_spectra(native, tile, kind, rows, cols, dtype):
    """Singular values of one size (flat), of which the diagonals dominate, and falling ones."""
    check(matrices(kind, 2, rows, cols).to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_values_strides_and_padding(native, tile, dtype):
    """NaN and infinities stay in their matrix; strided matrices (whose norm is added up in another
    order) and a shifted output."""
    x = matrices("loud", 6, 301, 203).to(dtype)
    want = ags.orthogonalize(x)
    check(x, got=want)
    bad = x.clone()
    bad[1, 300, 202] = math.nan
    bad[4, 0, 7] = -math.inf
    bad[2] = 0
    got = ags.orthogonalize(bad)
    assert torch.isnan(got[1]).all() and torch.isnan(got[4]).all() and not got[2].any()
    for i in (0, 3, 5):
        assert torch.equal(got[i], want[i])
    wide = torch.full((6, 310, 211), math.nan, dtype=dtype, device=DEV)
    view = wide[:, 4:305, 3:206]
    view.copy_(x)
    room = torch.full((x.numel() + 33,), 7.0, dtype=dtype, device=DEV)
    out = room[1:1 + x.numel()].view_as(x)
    check(x, got=ags.orthogonalize(view, out=out))
    assert room[0] == 7 and (room[1 + x.numel():] == 7).all()
    assert torch.isnan(wide[:, :4]).all() and torch.isnan(wide[:, :, :3]).all()


def step_in(dtype, g, offs, shapes, w, v, lr, mu, decay):
    """The step in 64 bits, or in fp32 throughout."""
    w, v = w.to(dtype).clone(), v.to(dtype).clone()
    moved = torch.zeros_like(w)
    for s, shape in enumerate(shapes):
        part = slice(offs[s], offs[s + 1])
        v[part] = mu * v[part] + g[part].to(dtype)
        y = (g[part].to(dtype) + mu * v[part]).view(shape)
        x = orthogonal(y) if dtype == F8 else in_fp32(y, 5)
        moved[part] = lr * math.sqrt(max(1.0, shape[0] / shape[1])) * x.reshape(-1)
        w[part] = (1 - lr * decay) * w[part] - moved[part]
    return w, v, moved


@pytest.mark.parametrize("dtype", TYPES)
def test_step_of_many_shapes(native, tile, dtype):
    """Matrices of five shapes, tall and wide of the same size among them, in launches of up to four."""
    shapes = [(300, 517), (517, 300), (1025, 260), (300, 517), (129, 64), (700, 700), (64, 129), (1, 9), (260, 1025)]
    offs = [0]
    for r, c in shapes:
        offs.append(offs[-1] + r * c)
    n = offs[-1]
    g, w, v = (k * torch.randn(n, generator=gen(i), device=DEV) for i, k in enumerate((1e-3, 0.02, 5e-3)))
    g = g.to(dtype)
    w0, v0 = w.clone(), v.clone()
    ags.muon_step(g, offs, shapes, w, v, lr=0.05, mu=0.9, weight_decay=0.1)
    want_w, want_v, moved = step_in(F8, g, offs, shapes, w0, v0, 0.05, 0.9, 0.1)
    plain = step_in(FP32, g, offs, shapes, w0, v0, 0.05, 0.9, 0.1)[2]
    u = 2.0 ** -24
    assert float((v.to(F8) - want_v).abs().max()) <= 3 * u * float(v0.abs().max() + g.abs().max())
    for s in range(len(shapes)):
        part = slice(offs[s], offs[s + 1])
        size = float(moved[part].norm())
        tol = 2 * float((plain[part].to(F8) - moved[part]).norm()) + 2.0 ** -22 * size + 4 * u * (float(w0[part].norm()) + size)
        assert float((w[part].to(F8) - want_w[part]).norm()) <= tol, f"segment {s}"
    torch.cuda.synchronize()
    assert ags.get_last_error() == ags.Status.OK


def test_step_of_a_large_layer(native):
    """Sizes for which the product takes its large tiles, in several launches (of 1 GB of scratch memory)."""
    shapes = [(2048, 2048)] * 3 + [(2048, 5461)] * 4 + [(5461, 2048)] * 2 + [(1024, 4096)] * 2
    offs = [0]
    for r, c in shapes:
        offs.append(offs[-1] + r * c)
    n = offs[-1]
    g, w, v = (torch.randn(n, generator=gen(i), device=DEV) for i in range(3))
    g = g.to(BF16)
    w0, v0 = w.clone(), v.clone()
    ags.muon_step(g, offs, shapes, w, v, lr=0.5, mu=0.9, weight_decay=0.1)
    for s in (0, 2, 3, 6, 7, 8, 9, 10):
        part = slice(offs[s], offs[s + 1])
        at, one = [0, offs[s + 1] - offs[s]], [shapes[s]]
        want_w, want_v, moved = step_in(F8, g[part], at, one, w0[part], v0[part], 0.5, 0.9, 0.1)
        plain = step_in(FP32, g[part], at, one, w0[part], v0[part], 0.5, 0.9, 0.1)[2]
        size, u = float(moved.norm()), 2.0 ** -24
        tol = 2 * float((plain.to(F8) - moved).norm()) + 2.0 ** -22 * size + 4 * u * (float(w0[part].norm()) + size)
        assert float((w[part].to(F8) - want_w).norm()) <= tol, f"segment {s}"
        assert float((v[part].to(F8) - want_v).abs().max()) <= 3 * u * float(v0[part].abs().max() + g[part].abs().max())
    assert ags.get_last_error() == ags.Status.OK
