"""The root-mean-square norm with the residual's addition, its gradient and its 8-bit form on
the GPU against plain 64-bit forms."""
import math

import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
import more_reference as more
import training_reference as ref
from training_reference import F8, HALF, TINY, close, u

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
TYPES = [BF16, FP32]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(*shape, seed=0, dtype=FP32, std=1.0):
    return (std * torch.randn(*shape, generator=gen(seed), device=DEV)).to(dtype)


def strided(t, extra, shift=0):
    rows, cols = t.shape
    buf = torch.full((rows * (cols + extra) + shift,), math.nan, dtype=t.dtype, device=t.device)
    view = buf[shift:].view(rows, cols + extra)[:, :cols]
    view.copy_(t)
    return view


# every width of a team (256 * 2^i columns), its neighbours, odd ones, many narrow rows
SHAPES = [(1, 1), (3, 7), (5, 128), (700, 129), (9, 255), (2500, 256), (17, 257), (33, 500), (3000, 512), (65, 1000), (40, 1024),
          (21, 1025), (700, 2048), (13, 2049), (6, 4096), (11, 4100), (8, 8192), (5, 8200), (3, 16384), (4, 16383)]


def check(total, y, rstd, x, residual, weight, eps):
    want = more.rms(x, weight, eps, residual)
    if residual is not None:
        close(total, *want[0], "total")
        # exactly the fp32 sum rounded
        assert torch.equal(total, (x.float() + residual.float()).to(x.dtype))
    close(y, *want[1], "y")
    close(rstd, *want[2], "rstd")
    return want


@pytest.mark.parametrize("wdtype", [None, BF16, FP32])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm(native, rows, cols, dtype, wdtype):
    x, r = randn(rows, cols, seed=1, dtype=dtype, std=2.0), randn(rows, cols, seed=2, dtype=dtype)
    w = None if wdtype is None else (1 + randn(cols, seed=3, std=0.2)).to(wdtype)
    y, rstd = ags.rms_norm(x, w, eps=1e-5)
    check(None, y, rstd, x, None, w, 1e-5)
    y, total, rstd = ags.rms_norm(x, w, residual=r)
    check(total, y, rstd, x, r, w, 1e-6)
    again = ags.rms_norm(total, w)  # the same from the sum, bit for bit
    assert torch.equal(again[0], y) and torch.equal(again[1], rstd)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_checkpointed(native, rows, cols, dtype):
    x, r, w = randn(rows, cols, seed=1, dtype=dtype), randn(rows, cols, seed=2, dtype=dtype, std=3.0), randn(cols, seed=3)
    y0, total0, rstd0 = ags.rms_norm(x, w, residual=r)
    y, total, kept, rstd = ags.rms_norm_checkpointed(x, w, residual=r)
    assert torch.equal(y, y0) and torch.equal(total, total0) and torch.equal(rstd, rstd0)
    want = more.rms(x, w, 1e-6, r)
    h, h_tol = want[3]
    codes, scales = kept.codes[:, :cols], kept.scales
    wide = scales.to(F8).repeat_interleave(128, 1)[:, :cols]
    # half a code, and what h itself may be off (by which the largest of the block too)
    top = wide * 127
    off = (ref.unpacked(codes, scales, cols) - h).abs()
    assert not (off > wide * 0.5 + 2 * h_tol.amax(1, keepdim=True) + 4 * u * top + TINY).any()
    y1, kept1, rstd1 = ags.rms_norm_checkpointed(total, w)
    assert torch.equal(y1, y) and torch.equal(kept1.codes[:, :cols], codes) and torch.equal(kept1.scales, scales)


GRADS = [(1, 1, [0, 1]), (7, 5, [0, 3, 3, 7]), (130, 129, [0, 1, 130]), (70, 256, [0, 70]), (2100, 257, [0, 2000, 2100]),
         (600, 512, [0, 200, 400, 600]), (65, 1000, [0, 0, 65]), (300, 1024, [0, 100, 150, 300]), (90, 2048, [0, 90]),
         (33, 2500, [0, 11, 33]), (40, 4096, [0, 40]), (15, 8192, [0, 7, 15]), (9, 8200, [0, 4, 9]), (12, 16384, [0, 5, 12])]


@pytest.mark.parametrize("past", [False, True])
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,offs", GRADS)
def test_gradient(native, rows, cols, offs, dtype, kept, past):
    x, dy = randn(rows, cols, seed=1, dtype=dtype, std=2.0), randn(rows, cols, seed=2, dtype=dtype)
    w = (1 + randn(cols, seed=3, std=0.2)).to(FP32 if dtype == BF16 else BF16)
    d = randn(rows, cols, seed=4, dtype=dtype) if past else None
    workers = len(offs) - 1
    for gdtype, accumulate in ((FP32, False), (BF16, True)):
        old = [randn(cols, seed=5 + k, dtype=gdtype) for k in range(workers)]
        grads = [g.clone() for g in old]
        more_args = dict(grad_residual=d, worker_offsets=offs, grad_weights=grads, accumulate=accumulate)
        if kept:
            y, keep, rstd = ags.rms_norm_checkpointed(x, w)
            h = ref.unpacked(keep.codes, keep.scales, cols)
            h_tol = u * h.abs()
            dx, dw, again = ags.rms_norm_checkpointed_backward(dy, keep, rstd, w, with_output=True, **more_args)
            y8 = h * w.to(F8)
            close(again, y8, 2 * u * y8.abs() + HALF[dtype] * y8.abs() * (1 + 2 * u) + TINY, "again")
        else:
            y, rstd = ags.rms_norm(x, w)
            h = x.to(F8) * rstd.to(F8)[:, None]
            h_tol = u * h.abs()
            dx, dw = ags.rms_norm_backward(dy, x, rstd, w, **more_args)
        assert all(a is b for a, b in zip(dw, grads))
        want, dws = more.rms_gradient(dy, h, h_tol, rstd, w, d, offs, old if accumulate else None, gdtype)
        close(dx, *want, "dx")
        for k in range(workers):
            close(dw[k], *dws[k], f"dw of worker {k}")
    # without the weights' gradients, and with ones allocated here
    if not kept:
        only, none = ags.rms_norm_backward(dy, x, rstd, w, grad_residual=d, parameter_grads=False)
        assert none is None and torch.equal(only, dx)
        _, fresh = ags.rms_norm_backward(dy, x, rstd, w, grad_residual=d, worker_offsets=offs)
        assert len(fresh) == workers and fresh[0].dtype == w.dtype and fresh[0].shape == (cols,)


@pytest.mark.parametrize("kept", [False, True])
def test_gradient_of_many_rows(native, kept):
    """Several CTAs a worker, an empty worker, partial sums of thousands of rows."""
    rows, cols, offs = 20000, 384, [0, 9000, 9000, 9001, 20000]
    x, dy, d = randn(rows, cols, seed=1, dtype=BF16), randn(rows, cols, seed=2, dtype=BF16), randn(rows, cols, seed=3, dtype=BF16)
    if kept:
        _, keep, rstd = ags.rms_norm_checkpointed(x)
        h = ref.unpacked(keep.codes, keep.scales, cols)
        dx, dw = ags.rms_norm_checkpointed_backward(dy, keep, rstd, grad_residual=d, worker_offsets=offs)
    else:
        _, rstd = ags.rms_norm(x)
        h = x.to(F8) * rstd.to(F8)[:, None]
        dx, dw = ags.rms_norm_backward(dy, x, rstd, grad_residual=d, worker_offsets=offs)
    want, dws = more.rms_gradient(dy, h, u * h.abs(), rstd, None, d, offs, None, FP32)
    close(dx, *want, "dx")
    for k in range(4):
        close(dw[k], *dws[k], f"dw of worker {k}")
    assert not dw[1].any()


def test_difference(native):
    """The gradient against differences of the forward pass in fp32."""
    rows, cols = 4, 96
    x, r, w, dy, ds = (randn(rows if i != 2 else 1, cols, seed=i) for i in range(5))
    w = w[0]

    def loss(x, w):
        y, total, _ = ags.rms_norm(x, w, residual=r)
        return float((y.double() * dy.double()).sum() + (total.double() * ds.double()).sum())

    _, total, rstd = ags.rms_norm(x, w, residual=r)
    dx, dw = ags.rms_norm_backward(dy, total, rstd, w, grad_residual=ds)
    step = 1e-2
    for i in range(6):
        t, c = i % rows, 17 * i % cols
        e = torch.zeros_like(x)
        e[t, c] = step
        diff = (loss(x + e, w) - loss(x - e, w)) / (2 * step)
        # third derivatives of order 1 times step^2, and rounding over step
        assert abs(diff - float(dx[t, c])) < 2e-3 + 1e-3 * abs(diff)
        f = torch.zeros_like(w)
        f[c] = step
        diff = (loss(x, w + f) - loss(x, w - f)) / (2 * step)
        assert abs(diff - float(dw[0][c])) < 1e-3 + 1e-3 * abs(diff)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("extra,shift", [(0, 1), (3, 0), (8, 8), (16, 0), (1, 3)])
def test_strides(native, dtype, extra, shift):
    rows, cols = 37, 520
    x, r, dy, d = (randn(rows, cols, seed=i, dtype=dtype) for i in range(4))
    w = randn(cols, seed=5)
    y, total, kept, rstd = ags.rms_norm_checkpointed(x, w, residual=r)
    xs, rs, dys, ds = (strided(t, extra, shift) for t in (x, r, dy, d))
    for a, b in ((xs, r), (x, rs), (xs, rs)):
        got = ags.rms_norm_checkpointed(a, w, residual=b)
        close(got[0], y.to(F8), more.rms(x, w, 1e-6, r)[1][1] * 2, "y")
        assert torch.equal(got[1], total)
    want = ags.rms_norm_backward(dy, total, rstd, w, grad_residual=d)
    tol = more.rms_gradient(dy, total.to(F8) * rstd.to(F8)[:, None], u * total.to(F8).abs() * rstd.to(F8)[:, None], rstd, w, d, [0, rows], None, FP32)
    for g, t, p in ((dys, total, d), (dy, strided(total, extra, shift), d), (dy, total, ds)):
        got = ags.rms_norm_backward(g, t, rstd, w, grad_residual=p)
        close(got[0], want[0].to(F8), 2 * tol[0][1], "dx")
        close(got[1][0], want[1][0].to(F8), 2 * tol[1][0][1], "dw")
    got = ags.rms_norm_checkpointed_backward(dys, kept, rstd, w, grad_residual=ds)
    base = ags.rms_norm_checkpointed_backward(dy, kept, rstd, w, grad_residual=d)
    close(got[0], base[0].to(F8), 2 * tol[0][1] + 2.0 ** -7 * base[0].to(F8).abs() * (dtype == BF16), "dx")


@pytest.mark.parametrize("dtype", TYPES)
def test_values(native, dtype):
    x = randn(6, 300, seed=1, dtype=dtype)
    x[1] = 0
    x[2, 7] = math.nan
    x[3, 299] = math.inf
    x[4] *= 1e-30
    y, rstd = ags.rms_norm(x, eps=1e-6)
    assert not y[1].any() and float(rstd[1]) == pytest.approx(1e3, rel=1e-6)
    assert torch.isnan(y[2]).all() and float(rstd[3]) == 0 and torch.isnan(y[3, 299]) and not y[3, :299].any()
    assert torch.isfinite(y[4]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[5]).all()
    # eps of zero on a row of zeros: 0 / 0
    assert torch.isnan(ags.rms_norm(x, eps=0.0)[0][1]).all()
    _, kept, _ = ags.rms_norm_checkpointed(x)
    assert torch.isnan(kept.scales[2]).all() and not kept.scales[1].any()


def test_empty(native):
    x = torch.empty(0, 64, device=DEV)
    y, total, rstd = ags.rms_norm(x, residual=x)
    assert y.shape == total.shape == (0, 64) and rstd.shape == (0,)
    dx, dw = ags.rms_norm_backward(x, x, rstd, worker_offsets=[0, 0, 0])
    assert dx.shape == (0, 64) and len(dw) == 2 and not dw[0].any() and not dw[1].any()
    y, kept, rstd = ags.rms_norm_checkpointed(x)
    ags.rms_norm_checkpointed_backward(x, kept, rstd)
    x3 = randn(2, 3, 64)
    y, total, rstd = ags.rms_norm(x3, residual=x3)
    assert y.shape == x3.shape and rstd.shape == (2, 3)


def test_streams_and_capture(native):
    x, r, dy, w = (randn(300, 1000, seed=i, dtype=BF16) for i in range(4))
    w = w[0].contiguous()
    want = ags.rms_norm(x, w, residual=r)
    back = ags.rms_norm_backward(dy, want[1], want[2], w, grad_residual=dy, worker_offsets=[0, 100, 300])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = ags.rms_norm(x, w, residual=r, stream=s)
    got_back = ags.rms_norm_backward(dy, got[1], got[2], w, grad_residual=dy, worker_offsets=[0, 100, 300], stream=s)
    torch.cuda.synchronize()
    for a, b in zip((*got, got_back[0], *got_back[1]), (*want, back[0], *back[1])):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, total, kept, rstd = ags.rms_norm_checkpointed(x, w, residual=r)
        dx, dw = ags.rms_norm_checkpointed_backward(dy, kept, rstd, w)
    x.copy_(dy)  # other inputs for the replay
    graph.replay()
    torch.cuda.synchronize()
    y2, total2, kept2, rstd2 = ags.rms_norm_checkpointed(x, w, residual=r)
    dx2, dw2 = ags.rms_norm_checkpointed_backward(dy, kept2, rstd2, w)
    assert torch.equal(y, y2) and torch.equal(total, total2) and torch.equal(dx, dx2) and torch.equal(dw[0], dw2[0])


def test_guards(native):
    """Outputs between guard elements."""
    for dtype in TYPES:
        x, r = randn(5, 1003, seed=1, dtype=dtype), randn(5, 1003, seed=2, dtype=dtype)
        buf = torch.full((5 * 1003 + 64,), 7.0, dtype=dtype, device=DEV)
        out = buf[32:32 + 5 * 1003].view(5, 1003)
        ags.rms_norm(x, residual=r, out=out)
        assert (buf[:32] == 7).all() and (buf[-32:] == 7).all()


def test_refusals(native):
    x, w = randn(4, 8), randn(8)
    rstd = torch.ones(4, device=DEV)
    for call in (lambda: ags.rms_norm(x.double()), lambda: ags.rms_norm(x, residual=x.int()), lambda: ags.rms_norm(x, w.half())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: ags.rms_norm(x, w[:4]), lambda: ags.rms_norm(x, residual=x[:2]), lambda: ags.rms_norm(x, residual=x.bfloat16()),
                 lambda: ags.rms_norm(x.t()), lambda: ags.rms_norm(x, out=x.bfloat16()),
                 lambda: ags.rms_norm_backward(x[:2], x, rstd), lambda: ags.rms_norm_backward(x, x, rstd[:2]),
                 lambda: ags.rms_norm_backward(x, x, rstd, grad_residual=x[:, :4]), lambda: ags.rms_norm_backward(x, x, rstd, accumulate=True),
                 lambda: ags.rms_norm_backward(x, x, rstd, worker_offsets=[0, 3]),
                 lambda: ags.rms_norm_backward(x, x, rstd, grad_weights=[w], parameter_grads=False),
                 lambda: ags.rms_norm_backward(x, x, rstd, grad_weights=[w, w])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ags.rms_norm(x, out=x), lambda: ags.rms_norm(x, residual=w.expand(4, 8).contiguous(), eps=-1.0),
                 lambda: ags.rms_norm(torch.zeros(2, 16385, device=DEV)),
                 lambda: ags.rms_norm_backward(x, x, rstd, grad_weights=[x[0]], worker_offsets=[0, 4])):
        with pytest.raises(ags.AdasumError):
            call()
    with pytest.raises(TypeError):
        ags.rms_norm_checkpointed_backward(x, (x, x), rstd)
    lib = ags.load_library()
    # a residual without a place for the sum, and the reverse
    y = torch.empty_like(x)
    assert lib.adasum_rms_norm(x.data_ptr(), 4, 8, 8, 0, rstd.data_ptr(), 8, None, None, 0, 1e-6, y.data_ptr(), None, None, None, 0) == 1
    assert lib.adasum_rms_norm(x.data_ptr(), 4, 8, 8, 0, None, 0, y.data_ptr(), None, 0, 1e-6, y.data_ptr(), None, None, None, 0) == 1
