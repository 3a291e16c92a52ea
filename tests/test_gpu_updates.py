"""The orthogonalised updates on the GPU against the iteration in 64 bits."""
import math

import numpy as np
import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
from updates_reference import F8, QUINTIC, bound, orthogonal, updates

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
TYPES = [BF16, FP32]
u = 2.0 ** -24
HALF = {FP32: u, BF16: 2.0 ** -8}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def off(got, want):
    assert got.shape == want.shape
    assert torch.isfinite(got).all()
    return float((got.to(F8) - want).norm() / want.norm())


def check_status():
    torch.cuda.synchronize()
    assert ags.get_last_error() == 0


# One row or column, sizes around the tiles' (64, 128, 256), odd ones, both orientations,
# depths beyond one run of the accumulators (512), batches beyond the SMs.
SIZES = [(1, 1, 1), (1, 1, 9), (2, 9, 1), (1, 5, 7), (3, 17, 33), (1, 64, 64), (1, 63, 129), (2, 128, 128), (1, 129, 127),
         (1, 65, 520), (5, 300, 129), (2, 256, 256), (1, 257, 511), (1, 517, 1000), (3, 1000, 517), (1, 24, 4099), (1, 4099, 24),
         (2, 1024, 1024), (1, 1100, 2050), (200, 48, 80), (300, 8, 8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,rows,cols", SIZES)
def test_orthogonalize(native, batch, rows, cols, dtype):
    x = updates(batch, rows, cols, gen=gen(rows + cols)).to(dtype)
    for steps in (1, 2, 3, 5):
        got = ags.orthogonalize(x, steps=steps)
        assert got.dtype == dtype
        assert off(got, orthogonal(x, steps)) <= bound(x, dtype, steps), f"steps {steps}"
    check_status()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(128, 512), (700, 650)])
@pytest.mark.parametrize("spectrum", ["random", "power", "one", "flat"])
def test_spectra(native, rows, cols, dtype, spectrum):
    g = gen(3)
    x = torch.randn(rows, cols, generator=g, device=DEV)
    if spectrum != "random":
        left = torch.linalg.qr(torch.randn(rows, min(rows, cols), generator=g, device=DEV, dtype=F8))[0]
        right = torch.linalg.qr(torch.randn(cols, min(rows, cols), generator=g, device=DEV, dtype=F8))[0]
        s = torch.arange(1, min(rows, cols) + 1, device=DEV, dtype=F8)
        s = {"power": 1 / s, "one": (s == 1).to(F8), "flat": torch.ones_like(s)}[spectrum]
        x = ((left * s) @ right.mT).float()
    x = x.to(dtype)
    if spectrum == "one":
        # (what rounding the input left around the one direction is part of the input)
        got, want = ags.orthogonalize(x, steps=2), orthogonal(x, 2)
        assert off(got, want) <= bound(x, dtype, 2)
    else:
        assert off(ags.orthogonalize(x), orthogonal(x)) <= bound(x, dtype)
    check_status()


def test_singular_values_approach_one(native):
    x = torch.randn(3, 256, 700, generator=gen(1), device=DEV)
    s = torch.linalg.svdvals(ags.orthogonalize(x).double())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.25
    # a converging iteration, from one triple a step
    triples = [QUINTIC] * 4 + [(1.875, -1.25, 0.375)] * 6
    got = ags.orthogonalize(x, steps=10, coefficients=triples)
    assert off(got, orthogonal(x, 10, triples)) <= bound(x, FP32, 5)
    assert float((torch.linalg.svdvals(got.double()) - 1).abs().max()) < 1e-4


@pytest.mark.parametrize("dtype", TYPES)
def test_scale_does_not_matter(native, dtype):
    """Magnitudes whose squares leave fp32's range."""
    x = updates(40, 72, gen=gen(5))
    want = orthogonal(x.to(dtype), eps=0.0)
    for power in (-100, -70, -50, -20, 0, 30, 60, 90, 110):
        got = ags.orthogonalize((x * 2.0 ** power).to(dtype), eps=0.0)
        assert off(got, want) <= bound(x, dtype), f"2^{power}"


@pytest.mark.parametrize("dtype", TYPES)
def test_values(native, dtype):
    x = updates(4, 33, 50, gen=gen(6)).to(dtype)
    alone = ags.orthogonalize(x[3])
    x[0] = 0
    x[1, 4, 5] = math.nan
    x[2, 32, 49] = math.inf
    got = ags.orthogonalize(x)
    assert not got[0].any()
    assert torch.isnan(got[1]).all() and torch.isnan(got[2]).all()
    assert torch.equal(got[3], alone)  # the others of a batch do not matter
    check_status()


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_outputs(native, dtype):
    base = updates(2, 3, 40, 70, gen=gen(7)).to(dtype)
    want = ags.orthogonalize(base)
    wide = torch.full((2, 3, 45, 77), math.nan, dtype=dtype, device=DEV)
    view = wide[:, :, 2:42, 3:73]
    view.copy_(base)
    assert torch.equal(ags.orthogonalize(view[0]), want[0])
    assert torch.equal(ags.orthogonalize(wide.view(6, 45, 77)[:, 2:42, 3:73]).view_as(want), want)
    assert torch.equal(ags.orthogonalize(view[1, 2]), want[1, 2])
    out = torch.full_like(base, math.nan)
    assert ags.orthogonalize(base, out=out) is out and torch.equal(out, want)
    shifted = torch.full((base.numel() + 1,), math.nan, dtype=dtype, device=DEV)[1:].view_as(base)
    shifted.copy_(base)
    assert torch.equal(ags.orthogonalize(shifted), want)
    assert ags.orthogonalize(base[:0]).shape == (0, 3, 40, 70)
    assert ags.orthogonalize(base[..., :0]).shape == (2, 3, 40, 0)
    with torch.no_grad():
        p = torch.nn.Parameter(base.float()[0, 0].clone())
    assert not ags.orthogonalize(p).requires_grad


def test_equal_bits_and_inputs_kept(native):
    x = updates(2, 300, 500, gen=gen(8))
    kept = x.clone()
    first = ags.orthogonalize(x)
    for _ in range(5):
        assert torch.equal(ags.orthogonalize(x), first)
    assert torch.equal(x, kept)


# --------------------------------------------------------------------------------- step

SHAPES = [(64, 96), None, (96, 64), (7, 130), None, (130, 7), (1, 5), (200, 200), None, (64, 96)]


def layout(shapes, lengths=(11, 0, 300)):
    it = iter(lengths)
    offs = [0]
    for s in shapes:
        offs.append(offs[-1] + (next(it) if s is None else s[0] * s[1]))
    return offs


def step_reference(g, offs, shapes, w, v, lr, mu, nesterov, decay, scale, steps=5):
    w, v = w.to(F8).clone(), v.to(F8).clone()
    moved = torch.zeros_like(w)
    for s, shape in enumerate(shapes):
        if shape is None:
            continue
        part = slice(offs[s], offs[s + 1])
        gs = g[part].to(F8)
        v[part] = mu * v[part] + gs
        x = orthogonal((gs + mu * v[part] if nesterov else v[part]).view(shape), steps).reshape(-1)
        k = {None: 1.0, "spectral": math.sqrt(max(1.0, shape[0] / shape[1])), "rms": 0.2 * math.sqrt(max(shape))}[scale]
        moved[part] = lr * k * x
        w[part] = (1 - lr * decay) * w[part] - lr * k * x
    return w, v, moved


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale,nesterov,decay", [("spectral", True, 0.0), ("rms", False, 0.1), (None, True, 0.3)])
def test_step(native, dtype, scale, nesterov, decay):
    offs = layout(SHAPES)
    n = offs[-1]
    g, w, v = (k * torch.randn(n, generator=gen(i), device=DEV) for i, k in enumerate((1e-3, 0.02, 5e-3)))
    g = g.to(dtype)
    w0, v0 = w.clone(), v.clone()
    got = ags.muon_step(g, offs, SHAPES, w, v, lr=0.05, mu=0.9, nesterov=nesterov, weight_decay=decay, scale=scale)
    assert got[0] is w and got[1] is v
    want_w, want_v, moved = step_reference(g, offs, SHAPES, w0, v0, 0.05, 0.9, nesterov, decay, scale)
    assert float((v.to(F8) - want_v).abs().max()) <= 3 * u * float(v0.abs().max() + g.abs().max())
    for s, shape in enumerate(SHAPES):
        part = slice(offs[s], offs[s + 1])
        if shape is None:  # not touched
            assert torch.equal(w[part], w0[part]) and torch.equal(v[part], v0[part])
            continue
        x = want_w[part].view(shape)
        tol = bound(x, FP32) * float(moved[part].norm()) + 4 * u * float(w0[part].norm() + moved[part].norm())
        assert float((w[part].to(F8) - want_w[part]).norm()) <= tol
    check_status()


def test_steps_of_many_shapes_and_chunks(native):
    """More matrices of one shape than one launch takes, beside single ones."""
    shapes = [(8, 16)] * 150 + [(16, 8)] * 150 + [(40, 40), None, (12, 300)]
    offs = layout(shapes, (5,))
    g, w, v = (torch.randn(offs[-1], generator=gen(i), device=DEV) for i in range(3))
    w0, v0 = w.clone(), v.clone()
    ags.muon_step(g, np.array(offs), shapes, w, v, lr=0.1)
    want_w, want_v, moved = step_reference(g, offs, shapes, w0, v0, 0.1, 0.95, True, 0.0, "spectral")
    assert float((w.to(F8) - want_w).norm()) <= bound(torch.empty(8, 16), FP32) * float(moved.norm()) + 4 * u * float(want_w.norm())
    assert float((v.to(F8) - want_v).norm()) <= 3 * u * float(want_v.norm())


def test_step_after_the_combine(native):
    """Two workers' gradients combined, then stepped; the norm's segment by momentum."""
    shapes = [(48, 64), None, (64, 32)]
    offs = layout(shapes, (64,))
    grads = [torch.randn(offs[-1], generator=gen(i), device=DEV).to(BF16) for i in (1, 2)]
    w, v = torch.randn(offs[-1], generator=gen(3), device=DEV), torch.zeros(offs[-1], device=DEV)
    w0 = w.clone()
    g = ags.reduce(grads, offs)
    ags.muon_step(g, offs, shapes, w, v, lr=0.02)
    want_w, _, moved = step_reference(g, offs, shapes, w0, torch.zeros_like(v), 0.02, 0.95, True, 0.0, "spectral")
    assert float((w.to(F8) - want_w).norm()) <= bound(torch.empty(48, 64), FP32) * float(moved.norm()) + 4 * u * float(w0.norm())
    part = slice(offs[1], offs[2])
    ags.reduce_momentum_sgd([x[part] for x in grads], None, w[part], v[part], lr=0.02, mu=0.95)
    assert not torch.equal(w[part], w0[part])


# -------------------------------------------------------------------- streams and graphs


def test_streams_overlap(native):
    xs = [updates(2, 300, 400, gen=gen(i)) for i in range(4)]
    want = [ags.orthogonalize(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = [ags.orthogonalize(x, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    check_status()


def test_capture(native):
    shapes = [(96, 160), (160, 96)]
    offs = layout(shapes)
    g = torch.randn(offs[-1], generator=gen(1), device=DEV).to(BF16)
    w, v = torch.randn(offs[-1], generator=gen(2), device=DEV), torch.randn(offs[-1], generator=gen(3), device=DEV)
    w1, v1 = w.clone(), v.clone()
    for _ in range(3):
        ags.muon_step(g, offs, shapes, w1, v1, lr=0.02)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ags.muon_step(g, offs, shapes, w, v, lr=0.02)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, w1) and torch.equal(v, v1)
    check_status()


def test_two_captured_graphs(native):
    """Their scratch memory is each graph's own."""
    xs = [updates(300, 200, gen=gen(i)) for i in range(2)]
    want = [ags.orthogonalize(x) for x in xs]
    graphs, outs = [], []
    for x in xs:
        out = torch.empty_like(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ags.orthogonalize(x, out=out)
        graphs.append(graph)
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


def test_launches_are_the_librarys(native):
    x = updates(64, 64, gen=gen(1))
    before = ags.launch_count()
    ags.orthogonalize(x)
    assert ags.launch_count() > before


# ------------------------------------------------------------------------------ refusals


def test_refusals(native):
    x = torch.randn(4, 6, device=DEV)
    for bad in (x.double(), x.int(), "x"):
        with pytest.raises(TypeError):
            ags.orthogonalize(bad)
    for bad in (x[0], x.t(), x.expand(3, 4, 6), x[:, ::2]):
        with pytest.raises(ValueError):
            ags.orthogonalize(bad)
    for more in (dict(steps=0), dict(coefficients=(1.0, 2.0)), dict(coefficients=[(1.0, 2.0, 3.0)] * 4), dict(out=x.bfloat16()),
                 dict(out=torch.empty(6, 4, device=DEV))):
        with pytest.raises(ValueError):
            ags.orthogonalize(x, **more)
    for more in (dict(eps=-1.0), dict(eps=math.nan), dict(coefficients=(math.nan, 1.0, 1.0)), dict(out=x)):
        with pytest.raises(ags.AdasumError):
            ags.orthogonalize(x, **more)
    with pytest.raises(ags.AdasumError):
        ags.orthogonalize(x, steps=65)
    n = 24
    g, w, v = (torch.randn(n, device=DEV) for _ in range(3))
    good = (g, [0, n], [(4, 6)], w, v)
    ags.muon_step(*good, lr=0.1)
    for i, bad in ((0, g.view(4, 6)), (1, [0, 20]), (1, [0, 12, n]), (2, [(4, 6), None]), (3, w[:20]), (3, w.bfloat16()), (4, v.cpu())):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            ags.muon_step(*args, lr=0.1)
    for more in (dict(scale="frobenius"), dict(steps=-1)):
        with pytest.raises(ValueError):
            ags.muon_step(*good, lr=0.1, **more)
    for args in ((g, [0, n], [(4, 5)], w, v), (g, [0, n], [(-4, -6)], w, v), (g, [0, n], [(4, 6)], w, w), (g, [0, n], [(4, 6)], g, v)):
        with pytest.raises(ags.AdasumError):
            ags.muon_step(*args, lr=0.1)
    ags.muon_step(g[:0], [0], [], w[:0], v[:0], lr=0.1)
    kept = w.clone()
    ags.muon_step(g, [0, n], [None], w, v, lr=0.1)
    assert torch.equal(w, kept)


def test_scratch_is_checked(native):
    import ctypes
    lib = ags.load_library()
    x, out = torch.randn(4, 6, device=DEV), torch.empty(4, 6, device=DEV)
    need = lib.adasum_orthogonalize_scratch_bytes(1, 4, 6, 0)
    assert need > 0
    scratch = torch.empty(need + 256, dtype=torch.uint8, device=DEV)
    co = (ctypes.c_float * 3)(*QUINTIC)
    call = lambda p, nbytes: lib.adasum_orthogonalize(x.data_ptr(), 1, 4, 6, 24, 6, 0, 1, ctypes.addressof(co), 1e-7, out.data_ptr(), p, nbytes, 0)
    assert call(scratch.data_ptr(), need) == 0
    assert call(None, need) == 1 and call(scratch.data_ptr(), need - 1) == 1 and call(scratch.data_ptr() + 128, need) == 1
    assert call(x.data_ptr(), need) in (1, 3)
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows,cols", [(5, 7), (130, 257), (300, 60)])
def test_guards(native, monkeypatch, rows, cols):
    """Bytes behind the scratch memory and the output stay as they were."""
    from adaptive_gradient_summation_gb300 import updates as module
    guards = []

    def guarded(nbytes, index):
        t = torch.full((nbytes + 512,), 171, dtype=torch.uint8, device=DEV)
        guards.append(t[nbytes:])
        return t[:nbytes]

    monkeypatch.setattr(module, "_scratch", guarded)
    for dtype in TYPES:
        x = updates(2, rows, cols, gen=gen(1)).to(dtype)
        buf = torch.full((x.numel() + 64,), 7.0, dtype=dtype, device=DEV)
        ags.orthogonalize(x, out=buf[:x.numel()].view_as(x))
        assert (buf[x.numel():] == 7).all()
    torch.cuda.synchronize()
    assert len(guards) == 2 and all((g == 171).all() for g in guards)


def test_full_grids_on_two_streams(native):
    """Calls whose CTAs fill the GPU each, at once: CTAs of one wait for each other."""
    xs = [updates(16, 512, 640, gen=gen(i)).to(BF16) for i in range(3)]
    want = [ags.orthogonalize(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [ags.orthogonalize(x, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    check_status()
