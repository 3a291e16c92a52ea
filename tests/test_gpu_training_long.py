"""The training operators where their kernels loop: many rows a warp, and many tokens a part.

The norm kernels' grids hold 304 CTAs on 152 SMs, a CTA's teams and a team's rows (up to four
at a time) lying a grid apart, so it takes thousands of narrow rows to come to a second pass;
row counts here are past one pass and no multiple of one."""
import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
import training_reference as ref
from test_gpu_training import BF16, DEV, FP32, TYPES, activations, check_table_gradient, params, randn, skewed_tokens
from training_reference import F8, TINY, close, u

pytestmark = pytest.mark.gpu

LONG = [(10_007, 64), (10_007, 128), (10_007, 250), (6001, 512), (4001, 1000), (4001, 1024), (2003, 2048), (1501, 4096),
        (1301, 4100), (911, 8192), (701, 16_384), (703, 16_383)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", LONG)
def test_norm_of_many_rows(native, rows, cols, dtype):
    x, (w, b) = activations(rows, cols, dtype, seed=cols), params(cols, FP32, seed=7)
    (want_y, y_tol), want_mean, want_rstd, (h, h_tol) = ref.norm(x, w, b, 1e-5)
    y, mean, rstd = ags.layer_norm(x, w, b, eps=1e-5)
    close(y, want_y, y_tol, "y")
    close(mean, *want_mean, "mean")
    close(rstd, *want_rstd, "rstd")
    del want_y, y_tol
    y_kept, kept, rstd_kept = ags.layer_norm_checkpointed(x, w, b, eps=1e-5)
    assert torch.equal(y_kept, y) and torch.equal(rstd_kept, rstd)
    top = torch.nn.functional.pad(h.abs() + h_tol, (0, -cols % 128)).view(rows, -1, 128).amax(2)
    step = (top / 254 * (1 + 200 * u)).repeat_interleave(128, 1)[:, :cols]
    close(ref.unpacked(kept.codes, kept.scales, cols), h, step + 2 * h_tol + TINY, "h in 8 bits")


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(10_007, 128), (4001, 1001), (2003, 2048), (1501, 4104), (1301, 8192), (1301, 16_384), (1303, 16_383)])
def test_norm_gradient_of_many_rows(native, rows, cols, dtype, accumulate, kept):
    """Three or more rows for every team of every CTA, workers of unequal size, h from the
    reference's statistics."""
    x, dy, (w, b) = activations(rows, cols, dtype, 5), randn(rows, cols, seed=3, dtype=dtype), params(cols, FP32, 9)
    offs = [0, rows // 3, rows // 3, rows // 3 + 1, rows]
    K = len(offs) - 1
    old = randn(2, K, cols, seed=11)
    dw, db = list(old[0].clone().unbind(0)), list(old[1].clone().unbind(0))
    more = dict(worker_offsets=offs, grad_weights=dw, grad_biases=db, accumulate=accumulate)
    x8 = x.to(F8)
    mean = x8.mean(1).float()
    rstd = (1 / torch.sqrt((x8 - mean.to(F8)[:, None]).square().mean(1) + 1e-5)).float()
    if kept:
        _, ckpt, rstd = ags.layer_norm_checkpointed(x, w, b)
        h = ref.unpacked(ckpt.codes, ckpt.scales, cols)
        h_tol = u * h.abs()
        dx, _, _, again = ags.layer_norm_checkpointed_backward(dy, ckpt, rstd, w, b, with_output=True, **more)
        y = h * w.to(F8) + b.to(F8)
        close(again, y, 4 * u * ((h * w.to(F8)).abs() + b.to(F8).abs()) + ref.HALF[dtype] * y.abs() + TINY, "y again")
    else:
        h = (x8 - mean.to(F8)[:, None]) * rstd.to(F8)[:, None]
        h_tol = 3 * u * (x8.abs() + mean.to(F8).abs()[:, None]) * rstd.to(F8)[:, None] + 2 * u * h.abs()
        dx = ags.layer_norm_backward(dy, x, mean, rstd, w, **more)[0]
    want_x, want_w, want_b = ref.norm_gradient(dy, h, h_tol, rstd, w, offs, old[0] if accumulate else None,
                                               old[1] if accumulate else None, FP32)
    close(dx, *want_x, "dx")
    for k in range(K):
        close(dw[k], *want_w[k], f"dw of worker {k}")
        close(db[k], *want_b[k], f"db of worker {k}")


def kinds(kind, n, rows):
    at = torch.arange(n, device=DEV)
    return {"same": torch.full_like(at, rows // 2), "all different": rows - 1 - at % rows,
            "two": 7 + (at * 7919 % 97 < 40).long(), "first and last": at % 2 * (rows - 1),
            "skewed": skewed_tokens(n, rows, seed=n)}[kind]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["same", "all different", "two", "first and last", "skewed"])
@pytest.mark.parametrize("n,cols", [(60_000, 256), (20_000, 1024), (65_536, 769), (40_000, 1024)])
def test_table_gradient_of_many_tokens(native, n, cols, kind, accumulate):
    """16 tokens a warp (60000 x 256, 20000 x 1024) and 32 (the others), on vectors and (769
    columns) off them: runs within a part, over warps, over chunks, over all of a worker."""
    rows = n // 2
    offs = [0, n // 3, n // 3, n // 3 + 700, n]
    for dtype, gdtype in ((BF16, FP32), (BF16, BF16)) if accumulate else ((BF16, FP32), (FP32, BF16)):
        check_table_gradient(rows, cols, offs, dtype, gdtype, accumulate, kinds(kind, n, rows), scale=0.75)
