"""The training operators (embeddings, layer norm, 8-bit checkpoints, GELU from them) on the
GPU against plain 64-bit forms, at the sizes and values where they can go wrong."""
import math

import numpy as np
import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
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
    """The same matrix with rows `extra` elements further apart, starting `shift` elements in."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + extra) + shift,), math.nan, dtype=t.dtype, device=t.device)
    view = buf[shift:].view(rows, cols + extra)[:, :cols]
    view.copy_(t)
    return view


def skewed_tokens(n, rows, seed, dtype=torch.int64, drop=0.1):
    """Frequencies falling off as 1 / rank, some tokens outside the table on both sides."""
    x = torch.rand(n, generator=gen(seed), device=DEV, dtype=F8)
    t = (torch.exp(x * math.log(rows + 1.0)) - 1).long().clamp_(0, rows - 1)
    t = torch.randperm(rows, generator=gen(seed + 1), device=DEV)[t]
    y = torch.rand(n, generator=gen(seed + 2), device=DEV)
    t = torch.where(y < drop / 2, torch.full_like(t, -1), t)
    t = torch.where((y >= drop / 2) & (y < drop), torch.full_like(t, rows), t)
    return t.to(dtype)


# ------------------------------------------------------------------------------ embeddings

LOOKUPS = [(1, 1, 1), (3, 5, 7), (17, 100, 8), (128, 1000, 1024), (65, 50, 1000), (33, 77, 129), (5, 9, 4100),
           (2, 3, 20000)]


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,rows,cols", LOOKUPS)
def test_lookup(native, n, rows, cols, dtype, ids):
    table = randn(rows, cols, seed=n, dtype=dtype)
    tokens = skewed_tokens(n, rows, seed=cols, dtype=ids, drop=0.3)
    for scale in (1.0, math.sqrt(cols)):
        got = ags.embedding(table, tokens, scale=scale)
        assert got.dtype == dtype
        want, tol = ref.lookup(table, tokens, np.float32(scale).item())
        close(got, want, tol, "lookup")
    assert torch.equal(ags.embedding(table, tokens)[tokens < 0], torch.zeros(int((tokens < 0).sum()), cols, dtype=dtype, device=DEV))


def test_lookup_shapes_and_extremes(native):
    table = randn(40, 24, seed=1, dtype=BF16)
    tokens = torch.randint(0, 40, (3, 5), generator=gen(2), device=DEV)
    assert torch.equal(ags.embedding(table, tokens), table[tokens])           # exact with scale 1
    assert ags.embedding(table, tokens[:0]).shape == (0, 5, 24)
    assert torch.equal(ags.embedding(table, tokens[0, 0]), table[tokens[0, 0]])
    far = torch.tensor([0, 39, 40, -1, 2 ** 62, -2 ** 62, 2 ** 32 + 1, 2 ** 31], device=DEV)
    got = ags.embedding(table, far)
    assert torch.equal(got[:2], table[[0, 39]]) and not got[2:].any()
    # NaN and infinity pass through; a scale does not touch the zeros of a missing token
    table[3, :] = math.nan
    table[4, :] = math.inf
    got = ags.embedding(table, torch.tensor([3, 4, -1], device=DEV), scale=2.0)
    assert got[0].isnan().all() and got[1].isinf().all() and not got[2].any()
    assert torch.equal(ags.embedding(torch.empty(0, 8, device=DEV), torch.tensor([0, 1], device=DEV)),
                       torch.zeros(2, 8, device=DEV))
    out = torch.empty(8, 24, dtype=BF16, device=DEV)
    assert ags.embedding(table, far, out=out) is out


@pytest.mark.parametrize("shift", [0, 1, 4])
@pytest.mark.parametrize("dtype", TYPES)
def test_lookup_unaligned(native, dtype, shift):
    n, rows, cols = 37, 50, 96
    table = randn(rows * cols + shift, seed=3, dtype=dtype)[shift:].view(rows, cols)
    tokens = skewed_tokens(n, rows, seed=5)
    buf = torch.full((n * cols + 2 * 64 + shift,), 7.0, dtype=dtype, device=DEV)
    out = buf[64 + shift:64 + shift + n * cols].view(n, cols)
    ags.embedding(table, tokens, out=out)
    close(out, *ref.lookup(table, tokens, 1.0), "lookup")
    assert (buf[:64 + shift] == 7).all() and (buf[64 + shift + n * cols:] == 7).all()


# (rows of the table, columns, worker offsets)
TABLES = [(1, 1, [0, 1]), (7, 3, [0, 0]), (50, 8, [0, 200]), (1000, 129, [0, 700]), (313, 256, [0, 0, 5, 5, 1000]),
          (5000, 96, [0, 4099]), (77, 1000, [0, 33, 64, 65, 300]), (40, 40, [0, 31, 32, 64]), (9, 4100, [0, 65]),
          (70_000, 8, [0, 3000])]


def check_table_gradient(n_rows, cols, offs, dtype, gdtype, accumulate, tokens, padding_idx=None, scale=1.0, seed=9,
                         dy=None):
    n, K = offs[-1], len(offs) - 1
    dy = randn(n, cols, seed=seed, dtype=dtype) if dy is None else dy
    old = randn(K, n_rows * cols, seed=seed + 1, dtype=gdtype)
    guard = 64
    bufs = torch.full((K, n_rows * cols + 2 * guard), 5.0, dtype=gdtype, device=DEV)
    grads = [b[guard:guard + n_rows * cols] for b in bufs]
    for g, o in zip(grads, old):
        g.copy_(o)
    got = ags.embedding_backward(dy, tokens, n_rows, scale=scale, worker_offsets=offs, padding_idx=padding_idx,
                                 grads=grads, accumulate=accumulate)
    wants = ref.table_gradient(dy, tokens, n_rows, np.float32(scale).item(), offs, padding_idx,
                               list(old) if accumulate else None, gdtype)
    for k, (want, tol) in enumerate(wants):
        assert got[k].data_ptr() == grads[k].data_ptr()
        close(got[k].view(n_rows, cols), want, tol, f"worker {k}")
    assert (bufs[:, :guard] == 5).all() and (bufs[:, guard + n_rows * cols:] == 5).all()
    return got


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("gdtype", TYPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n_rows,cols,offs", TABLES)
def test_table_gradient(native, n_rows, cols, offs, dtype, gdtype, accumulate):
    tokens = skewed_tokens(offs[-1], n_rows, seed=cols, dtype=torch.int32 if cols % 2 else torch.int64)
    check_table_gradient(n_rows, cols, offs, dtype, gdtype, accumulate, tokens, scale=1.0 if cols > 100 else 2.5)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 64, 1000, 4096, 4097, 20_000])
@pytest.mark.parametrize("kind", ["same", "all different", "two", "first and last", "none"])
def test_table_gradient_runs(native, kind, n):
    """Runs of one token of every length: within a chunk, over its ends, over all of it."""
    rows, cols = 20_000, 16
    at = torch.arange(n, device=DEV)
    tokens = {"same": torch.full_like(at, 12345), "all different": rows - 1 - at, "two": 7 + (at * 7919 % 97 < 40).long(),
              "first and last": (at % 2) * (rows - 1), "none": torch.full_like(at, -1)}[kind]
    offs = [0, n // 3, n] if n > 3 else [0, n]
    check_table_gradient(rows, cols, offs, BF16, FP32, False, tokens, seed=n)


@pytest.mark.parametrize("n", [50, 300, 5000, 9000])
@pytest.mark.parametrize("rows,cols", [(1 << 23, 2), ((1 << 24) + 5, 1)])
def test_table_gradient_many_rows(native, rows, cols, n):
    """Tokens of 24 and 25 bits: more digits to sort by, and no 32-bit word for a token and its
    place."""
    tokens = skewed_tokens(n, rows, seed=n)
    dy = randn(n, cols, seed=1)
    for accumulate in (False, True):
        grad = torch.zeros(rows * cols, device=DEV)
        ags.embedding_backward(dy, tokens, rows, grads=grad, accumulate=accumulate)
        want, tol = ref.table_gradient(dy, tokens, rows, 1.0, [0, n], None, None, FP32)[0]
        close(grad.view(rows, cols), want, tol, "gradient")


def test_table_gradient_most_workers(native):
    """256 workers of 0 to 70 tokens each, a few hundred, and one of thousands."""
    rows, cols = 37, 40
    for sizes in ([k % 71 for k in range(256)], [k % 3 * 130 for k in range(256)], [k % 71 for k in range(255)] + [9000]):
        offs = [0]
        for s in sizes:
            offs.append(offs[-1] + s)
        tokens = skewed_tokens(offs[-1], rows, seed=len(set(sizes)))
        check_table_gradient(rows, cols, offs, BF16, FP32, True, tokens)


def test_table_gradient_order_of_tokens(native):
    """Sorting is stable and sums are fixed: equal calls give equal bits, and tokens permuted
    within a worker change the sums by roundings only."""
    n, rows, cols = 6000, 300, 72
    tokens, dy = skewed_tokens(n, rows, seed=4), randn(n, cols, seed=5, dtype=FP32)
    first = ags.embedding_backward(dy, tokens, rows)[0]
    for _ in range(3):
        assert torch.equal(ags.embedding_backward(dy, tokens, rows)[0], first)
    perm = torch.randperm(n, generator=gen(6), device=DEV)
    check_table_gradient(rows, cols, [0, n], FP32, FP32, False, tokens[perm], dy=dy[perm])


def test_table_gradient_padding_and_absent(native):
    n, rows, cols = 500, 60, 40
    tokens = skewed_tokens(n, rows, seed=8)
    for pad in (0, int(tokens[tokens >= 0][0]), rows - 1, rows + 5, -7):
        check_table_gradient(rows, cols, [0, n], BF16, BF16, True, tokens, padding_idx=pad)
    # a token with a NaN row of gradient poisons its row only, or none when it is padding
    dy = randn(n, cols, seed=9)
    dy[17] = math.nan
    tokens[17] = 3
    got = ags.embedding_backward(dy, tokens, rows)[0]
    assert got[3].isnan().all() and not got[:3].isnan().any() and not got[4:].isnan().any()
    assert not ags.embedding_backward(dy, tokens, rows, padding_idx=3)[0].isnan().any()
    assert torch.equal(ags.embedding_backward(dy, tokens, rows, padding_idx=3)[0][3], torch.zeros(cols, device=DEV))


def test_table_gradient_rows_that_are_not_touched_keep_their_bits(native):
    n, rows, cols = 64, 1000, 33
    tokens, dy = torch.randint(0, 500, (n,), generator=gen(1), device=DEV), randn(n, cols, seed=2)
    grad = torch.full((rows * cols,), math.nan, device=DEV)
    ags.embedding_backward(dy, tokens, rows, grads=grad, accumulate=True)
    touched = torch.zeros(rows, dtype=torch.bool, device=DEV)
    touched[tokens] = True
    assert grad.isnan().all()
    grad = torch.full((rows * cols,), -0.0, device=DEV)  # (-0 + 0 would be 0)
    ags.embedding_backward(dy, tokens, rows, grads=grad, accumulate=True)
    assert torch.signbit(grad.view(rows, cols)[~touched]).all()
    assert not ags.embedding_backward(dy, tokens, rows)[0][~touched].any()


@pytest.mark.parametrize("extra,shift", [(0, 1), (8, 0), (3, 0), (24, 5)])
@pytest.mark.parametrize("dtype", TYPES)
def test_table_gradient_strided(native, dtype, extra, shift):
    n, rows, cols = 300, 50, 136
    tokens = skewed_tokens(n, rows, seed=3)
    dy = strided(randn(n, cols, seed=4, dtype=dtype), extra, shift)
    check_table_gradient(rows, cols, [0, 100, n], dtype, FP32, False, tokens, dy=dy)


def test_table_gradient_unaligned_gradients(native):
    n, rows, cols = 200, 30, 64
    tokens, dy = skewed_tokens(n, rows, seed=3), randn(n, cols, seed=4, dtype=BF16)
    want, tol = ref.table_gradient(dy, tokens, rows, 1.0, [0, n], None, None, BF16)[0]
    for shift in (1, 2, 4):
        buf = torch.full((rows * cols + 64,), 5.0, dtype=BF16, device=DEV)
        view = buf[shift:shift + rows * cols]
        ags.embedding_backward(dy, tokens, rows, grads=view)
        close(view.view(rows, cols), want, tol, "gradient")
        assert (buf[:shift] == 5).all() and (buf[shift + rows * cols:] == 5).all()


def test_embedding_difference(native):
    """The lookup is linear in the table, so a difference of its outputs along a direction is
    the gradient's product with it, up to the roundings of both."""
    n, rows, cols = 64, 20, 48
    table, way = randn(rows, cols, seed=1), randn(rows, cols, seed=2)
    tokens, dy = skewed_tokens(n, rows, seed=3), randn(n, cols, seed=4)
    grad = ags.embedding_backward(dy, tokens, rows, scale=3.0)[0]
    up, down = ags.embedding(table + way, tokens, scale=3.0), ags.embedding(table - way, tokens, scale=3.0)
    diff = float(((up.to(F8) - down.to(F8)) * dy.to(F8)).sum()) / 2
    want = float((grad.to(F8) * way.to(F8)).sum())
    tol = (n + 8) * u * float((up.to(F8).abs() + down.to(F8).abs()).mul(dy.to(F8).abs()).sum())
    assert abs(diff - want) <= tol


# ------------------------------------------------------------------------------ layer norm

NORMS = [(1, 1), (2, 2), (3, 7), (5, 64), (33, 100), (9, 128), (7, 129), (40, 256), (11, 1000), (129, 1024), (8, 1001),
         (6, 2048), (5, 2056), (3, 4096), (4, 4104), (2, 8192), (3, 16384), (2, 16383)]


def activations(rows, cols, dtype, seed):
    """Rows of unequal size and mean."""
    x = randn(rows, cols, seed=seed) * (0.5 + 2 * torch.rand(rows, 1, generator=gen(seed + 1), device=DEV))
    return (x + randn(rows, 1, seed=seed + 2)).to(dtype)


def params(cols, wdtype, seed):
    if wdtype is None:
        return None, None
    return 1 + 0.2 * randn(cols, seed=seed).to(wdtype), randn(cols, seed=seed + 1, dtype=wdtype)


@pytest.mark.parametrize("wdtype", [BF16, FP32, None])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", NORMS)
def test_norm(native, rows, cols, dtype, wdtype):
    x, (w, b) = activations(rows, cols, dtype, seed=cols), params(cols, wdtype, seed=7)
    y, mean, rstd = ags.layer_norm(x, w, b, eps=1e-5)
    want_y, want_mean, want_rstd, _ = ref.norm(x, w, b, 1e-5)
    close(y, *want_y, "y")
    close(mean, *want_mean, "mean")
    close(rstd, *want_rstd, "rstd")
    for only in ((w, None), (None, b)):
        close(ags.layer_norm(x, *only)[0], *ref.norm(x, *only, 1e-5)[0], "y, one parameter")


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", NORMS)
def test_norm_gradient(native, rows, cols, dtype, kept):
    x, dy = activations(rows, cols, dtype, seed=cols), randn(rows, cols, seed=3, dtype=dtype)
    for wdtype, gdtype, accumulate, offs in ((dtype, FP32, False, [0, rows]), (FP32, BF16, True, [0, 0, rows // 2, rows]),
                                             (None, dtype, False, [0, rows - 1, rows, rows])):
        w, b = params(cols, wdtype, seed=9)
        K = len(offs) - 1
        old = randn(2, K, cols, seed=11, dtype=gdtype)
        dw, db = list(old[0].clone().unbind(0)), list(old[1].clone().unbind(0))
        more = dict(worker_offsets=offs, grad_weights=dw, grad_biases=db, accumulate=accumulate)
        if kept:
            _, ckpt, rstd = ags.layer_norm_checkpointed(x, w, b)
            h = ref.unpacked(ckpt.codes, ckpt.scales, cols)
            h_tol = u * h.abs()
            dx, rw, rb, again = ags.layer_norm_checkpointed_backward(dy, ckpt, rstd, w, b, with_output=True, **more)
            w8 = 1.0 if w is None else w.to(F8)
            b8 = 0.0 if b is None else b.to(F8)
            y = h * w8 + b8
            close(again, y, 4 * u * ((h * w8).abs() + (abs(b8) if b is not None else 0.0)) + HALF[dtype] * y.abs() + TINY, "y again")
        else:
            _, mean, rstd = ags.layer_norm(x, w, b)
            h = (x.to(F8) - mean.to(F8)[:, None]) * rstd.to(F8)[:, None]
            h_tol = 3 * u * (x.to(F8).abs() + mean.to(F8).abs()[:, None]) * rstd.to(F8)[:, None] + 2 * u * h.abs()
            dx, rw, rb = ags.layer_norm_backward(dy, x, mean, rstd, w, **more)
        assert [t.data_ptr() for t in rw + rb] == [t.data_ptr() for t in dw + db]
        want_x, want_w, want_b = ref.norm_gradient(dy, h, h_tol, rstd, w, offs, old[0] if accumulate else None,
                                                   old[1] if accumulate else None, gdtype)
        close(dx, *want_x, "dx")
        for k in range(K):
            close(dw[k], *want_w[k], f"dw of worker {k}")
            close(db[k], *want_b[k], f"db of worker {k}")


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("offs", [[0, 3000], [0, 1, 2, 1500, 1500, 2999, 3000], list(range(0, 257))])
def test_norm_gradient_many_rows(native, offs, kept):
    rows, cols = offs[-1], 264
    x, dy, (w, b) = activations(rows, cols, BF16, 5), randn(rows, cols, seed=3, dtype=BF16), params(cols, FP32, 9)
    if kept:
        _, ckpt, rstd = ags.layer_norm_checkpointed(x, w, b)
        h = ref.unpacked(ckpt.codes, ckpt.scales, cols)
        got = [ags.layer_norm_checkpointed_backward(dy, ckpt, rstd, w, worker_offsets=offs) for _ in range(2)]
    else:
        _, mean, rstd = ags.layer_norm(x, w, b)
        h = (x.to(F8) - mean.to(F8)[:, None]) * rstd.to(F8)[:, None]
        got = [ags.layer_norm_backward(dy, x, mean, rstd, w, worker_offsets=offs) for _ in range(2)]
    h_tol = 4 * u * (x.to(F8).abs() * rstd.to(F8)[:, None] + h.abs() + 1)
    want_x, want_w, want_b = ref.norm_gradient(dy, h, h_tol, rstd, w, offs, None, None, FP32)
    dx, dw, db = got[0]
    close(dx, *want_x, "dx")
    for k in range(len(offs) - 1):
        close(dw[k], *want_w[k], f"dw of worker {k}")
        close(db[k], *want_b[k], f"db of worker {k}")
    assert all(torch.equal(p, q) for p, q in zip([got[0][0]] + got[0][1] + got[0][2], [got[1][0]] + got[1][1] + got[1][2]))


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(2100, 100), (2100, 512), (1100, 1000), (1100, 1001), (600, 2056), (300, 4104),
                                       (270, 8192), (265, 16383)])
def test_norm_gradient_long(native, rows, cols, dtype, kept):
    """Enough rows for the sums to be joined by a second kernel, at every width of team, two of
    the three workers' parts beginning inside a CTA's rows."""
    x, dy, (w, b) = activations(rows, cols, dtype, 5), randn(rows, cols, seed=3, dtype=dtype), params(cols, FP32, 9)
    offs = [0, rows // 3, rows // 3 + 1, rows]
    old = randn(2, 3, cols, seed=11)
    dw, db = list(old[0].clone().unbind(0)), list(old[1].clone().unbind(0))
    more = dict(worker_offsets=offs, grad_weights=dw, grad_biases=db, accumulate=True)
    if kept:
        _, ckpt, rstd = ags.layer_norm_checkpointed(x, w, b)
        h = ref.unpacked(ckpt.codes, ckpt.scales, cols)
        h_tol = u * h.abs()
        dx = ags.layer_norm_checkpointed_backward(dy, ckpt, rstd, w, **more)[0]
    else:
        _, mean, rstd = ags.layer_norm(x, w, b)
        h = (x.to(F8) - mean.to(F8)[:, None]) * rstd.to(F8)[:, None]
        h_tol = 3 * u * (x.to(F8).abs() + mean.to(F8).abs()[:, None]) * rstd.to(F8)[:, None] + 2 * u * h.abs()
        dx = ags.layer_norm_backward(dy, x, mean, rstd, w, **more)[0]
    want_x, want_w, want_b = ref.norm_gradient(dy, h, h_tol, rstd, w, offs, old[0], old[1], FP32)
    close(dx, *want_x, "dx")
    for k in range(3):
        close(dw[k], *want_w[k], f"dw of worker {k}")
        close(db[k], *want_b[k], f"db of worker {k}")


def test_scratch_is_checked(native):
    """Scratch memory that is missing, too small, not aligned or part of an input."""
    import ctypes
    lib, rows, cols = ags.load_library(), 3000, 64
    x, stat, out = randn(rows, cols, seed=1), torch.ones(rows, device=DEV), torch.empty(rows, cols, device=DEV)
    g = torch.empty(cols, device=DEV)
    offs, grads = (ctypes.c_int64 * 2)(0, rows), (ctypes.c_void_p * 1)(g.data_ptr())
    need = lib.adasum_layer_norm_backward_scratch_bytes(offs, 1, cols)
    scratch = torch.empty(need + 256, dtype=torch.uint8, device=DEV)
    call = lambda s, n: lib.adasum_layer_norm_backward(  # noqa: E731
        x.data_ptr(), cols, x.data_ptr(), cols, stat.data_ptr(), stat.data_ptr(), cols, 0, None, 0, offs, 1, out.data_ptr(),
        grads, None, 0, 0, s, n, None)
    before = ags.launch_count()
    assert need > 0 and call(None, need) == 1 and call(scratch.data_ptr(), need - 1) == 1
    assert call(scratch.data_ptr() + 8, need) == 1 and call(x.data_ptr(), need) == 3
    assert ags.launch_count() == before
    assert call(scratch.data_ptr(), need) == 0
    torch.cuda.synchronize()
    tokens = torch.zeros(rows, dtype=torch.int32, device=DEV)
    need = lib.adasum_embedding_backward_scratch_bytes(offs, 1, 1, cols)
    scratch = torch.empty(need + 256, dtype=torch.uint8, device=DEV)
    call = lambda s, n: lib.adasum_embedding_backward(  # noqa: E731
        x.data_ptr(), cols, cols, 0, tokens.data_ptr(), 4, offs, 1, 1, 1.0, -1, grads, 0, 0, s, n, None)
    before = ags.launch_count()
    assert need > 0 and call(None, need) == 1 and call(scratch.data_ptr(), need - 1) == 1
    assert call(scratch.data_ptr() + 8, need) == 1 and call(x.data_ptr(), need) == 3
    assert ags.launch_count() == before
    assert call(scratch.data_ptr(), need) == 0
    torch.cuda.synchronize()


def test_norm_without_rows(native):
    x = torch.empty(0, 40, device=DEV)
    w, b = params(40, FP32, 1)
    y, mean, rstd = ags.layer_norm(x, w, b)
    assert y.shape == (0, 40) and mean.shape == (0,)
    dx, dw, db = ags.layer_norm_backward(x, x, mean, rstd, w, worker_offsets=[0, 0, 0])
    assert dx.shape == (0, 40) and not any(t.any() for t in dw + db)
    old = randn(2, 40, seed=2)
    g = old.clone()
    ags.layer_norm_backward(x, x, mean, rstd, w, grad_weights=g[0], grad_biases=g[1], accumulate=True)
    assert torch.equal(g, old)
    _, kept, rstd = ags.layer_norm_checkpointed(x, w, b)
    assert ags.layer_norm_checkpointed_backward(x, kept, rstd, w)[0].shape == (0, 40)


@pytest.mark.parametrize("extra,shift", [(0, 1), (8, 0), (5, 0), (16, 3)])
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_strided(native, dtype, extra, shift):
    rows, cols = 21, 264
    x, dy, (w, b) = activations(rows, cols, dtype, 5), randn(rows, cols, seed=3, dtype=dtype), params(cols, dtype, 9)
    xs, dys = strided(x, extra, shift), strided(dy, extra, shift)
    y, mean, rstd = ags.layer_norm(xs, w, b)
    close(y, *ref.norm(x, w, b, 1e-5)[0], "y")
    h = (x.to(F8) - mean.to(F8)[:, None]) * rstd.to(F8)[:, None]
    h_tol = 3 * u * (x.to(F8).abs() + mean.to(F8).abs()[:, None]) * rstd.to(F8)[:, None] + 2 * u * h.abs()
    want = ref.norm_gradient(dy, h, h_tol, rstd, w, [0, rows], None, None, FP32)[0]
    close(ags.layer_norm_backward(dys, xs, mean, rstd, w)[0], *want, "dx")
    _, kept, rstd2 = ags.layer_norm_checkpointed(xs, w, b)
    full = ags.layer_norm_checkpointed_backward(dy, kept, rstd2, w)[0]
    h = ref.unpacked(kept.codes, kept.scales, cols)
    want = ref.norm_gradient(dy, h, u * h.abs(), rstd2, w, [0, rows], None, None, FP32)[0]
    close(full, *want, "dx from 8 bits")
    close(ags.layer_norm_checkpointed_backward(dys, kept, rstd2, w)[0], *want, "dx from 8 bits, strided")


def test_norm_leading_dimensions(native):
    x, (w, b) = activations(24, 48, BF16, 1), params(48, BF16, 2)
    flat = ags.layer_norm(x, w, b)
    shaped = ags.layer_norm(x.view(2, 3, 4, 48), w, b)
    assert shaped[0].shape == (2, 3, 4, 48) and shaped[1].shape == (2, 3, 4)
    assert all(torch.equal(p.reshape(-1), q.reshape(-1)) for p, q in zip(flat, shaped))
    row = ags.layer_norm(x[5], w, b)
    assert torch.equal(row[0], flat[0][5]) and row[1].shape == ()
    # every second row; not rows that do not flatten
    assert torch.equal(ags.layer_norm(x[::2], w, b)[0], flat[0][::2])
    with pytest.raises(ValueError):
        ags.layer_norm(x.view(4, 6, 48).transpose(0, 1), w, b)


@pytest.mark.parametrize("dtype", TYPES)
def test_norm_values(native, dtype):
    """Constant rows, rows whose mean is far larger than their spread, NaN and infinity."""
    cols = 1024
    x = activations(8, cols, dtype, 3)
    x[0] = 0
    x[1] = 3.0
    x[2] = (1e4 + randn(cols, seed=1)).to(dtype)
    x[3, 17] = math.nan
    x[4, 5] = math.inf
    x[5] = (1e-20 * randn(cols, seed=2)).to(dtype)
    w, b = params(cols, FP32, 4)
    y, mean, rstd = ags.layer_norm(x, w, b)
    fine = [0, 1, 2, 5, 6, 7]
    want_y, want_mean, want_rstd, _ = ref.norm(x[fine], w, b, 1e-5)
    close(y[fine], *want_y, "y")
    close(rstd[fine], *want_rstd, "rstd")
    assert y[3].isnan().all() and y[4].isnan().all()
    close(y[0], b.to(F8), HALF[dtype] * b.to(F8).abs() + TINY, "a constant row is the bias")
    dy = randn(8, cols, seed=6, dtype=dtype)
    dx, dw, db = ags.layer_norm_backward(dy, x, mean, rstd, w)
    assert dx[3].isnan().all() and not dx[fine].isnan().any()
    assert dw[0].isnan().all() and not db[0].isnan().any()
    _, kept, r2 = ags.layer_norm_checkpointed(x, w, b)
    dx, dw, db = ags.layer_norm_checkpointed_backward(dy, kept, r2, w)
    assert dx[3].isnan().all() and dx[4].isnan().all() and not dx[fine].isnan().any()


def test_norm_difference(native):
    """<dx, v> against the central difference of <dy, y> along v; the difference's own error is
    that of the same difference in 64 bits, and the roundings of y over the step."""
    rows, cols, step = 6, 192, 2.0 ** -6
    x, way, dy = activations(rows, cols, FP32, 1), randn(rows, cols, seed=2), randn(rows, cols, seed=3)
    w, b = params(cols, FP32, 4)
    _, mean, rstd = ags.layer_norm(x, w, b)
    dx, dw, db = ags.layer_norm_backward(dy, x, mean, rstd, w)

    def loss(x, w, b, plain=False):
        (y, tol), *_ = ref.norm(x, w, b, 1e-5)
        y = y if plain else ags.layer_norm(x, w, b)[0].to(F8)
        return float((y * dy.to(F8)).sum()), float((tol * dy.to(F8).abs()).sum())

    way_w, way_b = randn(cols, seed=5), randn(cols, seed=6)
    for d, grads in (((way, 0, 0), [(dx, way)]), ((0, way_w, way_b), [(dw[0], way_w), (db[0], way_b)])):
        up, down = [tuple(p + s * step * q for p, q in zip((x, w, b), d)) for s in (1, -1)]
        got = (loss(*up)[0] - loss(*down)[0]) / (2 * step)
        plain = (loss(*up, True)[0] - loss(*down, True)[0]) / (2 * step)
        want = sum(float((g.to(F8) * v.to(F8)).sum()) for g, v in grads)
        rounding = (loss(*up, True)[1] + loss(*down, True)[1]) / (2 * step)
        h = (x.to(F8) - mean.to(F8)[:, None]) * rstd.to(F8)[:, None]
        exact = ref.norm_gradient(dy, h, 0 * h, rstd, w, [0, rows], None, None, FP32)
        exact = ([exact[0][0]] if d[0] is way else [exact[1][0][0], exact[2][0][0]])
        truth = sum(float((g * v.to(F8)).sum()) for g, (_, v) in zip(exact, grads))
        assert abs(got - want) <= abs(plain - truth) + rounding + (rows + 200) * u * sum(
            float((g.to(F8) * v.to(F8)).abs().sum()) for g, v in grads)


# ----------------------------------------------------------------------- 8-bit checkpoints

PACKS = [(1, 1), (3, 5), (2, 127), (4, 128), (5, 129), (33, 1000), (7, 1001), (16, 4096), (3, 20_000), (300, 64), (2, 16)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", PACKS)
def test_pack(native, rows, cols, dtype):
    x = activations(rows, cols, dtype, seed=cols)
    kept = ags.checkpoint_pack(x)
    codes, scales = ref.pack(x)
    assert torch.equal(kept.scales.cpu(), scales)
    assert torch.equal(kept.codes[:, :cols].cpu(), codes)
    back = ags.checkpoint_unpack(kept)
    want = ref.unpacked(kept.codes, kept.scales, cols)
    close(back, want, HALF[dtype] * want.abs() + TINY, "unpacked")
    for other in TYPES:
        got = ags.checkpoint_unpack(kept, dtype=other)
        assert got.dtype == other
        close(got, want, (HALF[other] + u) * want.abs() + TINY, "unpacked to another type")
    top = torch.nn.functional.pad(x.to(F8).abs(), (0, -cols % 128)).view(rows, -1, 128).amax(2)
    half_step = (top / 254 * (1 + 200 * u)).repeat_interleave(128, 1)[:, :cols]
    close(want, x, half_step + TINY, "within half a step")


@pytest.mark.parametrize("dtype", TYPES)
def test_pack_values(native, dtype):
    """Zero blocks, tiny and huge blocks, ties, NaN and infinity: only their block is lost."""
    cols = 128 * 9 + 40
    x = randn(2, cols, seed=1)
    x[0, :128] = 0
    x[0, 128:256] *= 1e-30
    x[0, 256:384] *= 2.0 ** -122
    x[0, 384:512] *= 2.0 ** -119
    x[0, 512:640] *= 1e37
    x[0, 700] = math.nan
    x[0, 800] = -math.inf
    x[0, 900:1000] = math.inf
    x[0, 1024:1152] = 0
    x[0, 1024:1152:2] = -0.0
    x[0, -1] = 127.0
    x[0, -40:-1] = torch.arange(39, device=DEV) - 19.5
    x[1] = torch.arange(cols, device=DEV) % 255 - 127.5
    x[1, ::128] = 127.5
    x = x.to(dtype)
    kept = ags.checkpoint_pack(x)
    codes, scales = ref.pack(x)
    assert torch.equal(torch.nan_to_num(kept.scales.cpu(), -1.0), torch.nan_to_num(scales, -1.0))
    bad = scales.isnan().repeat_interleave(128, 1)[:, :cols]
    assert torch.equal(kept.codes[:, :cols].cpu()[~bad], codes[~bad])
    back = ags.checkpoint_unpack(kept)
    assert torch.equal(back.isnan().cpu(), bad) and bad.any() and not bad.all()
    assert not back[0, :128].any() and not back[0, 256:384].any() and back[0, 384:512].any()


@pytest.mark.parametrize("tanh", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", PACKS)
def test_gelu(native, rows, cols, dtype, tanh):
    x = (2 * randn(rows, cols, seed=cols)).to(dtype)
    dy = randn(rows, cols, seed=3, dtype=dtype)
    y, kept = ags.gelu_checkpointed(x, tanh=tanh)
    plain = ags.checkpoint_pack(x)
    assert torch.equal(kept.codes[:, :cols], plain.codes[:, :cols]) and torch.equal(kept.scales, plain.scales)
    x8 = x.to(F8)
    want = ref.gelu(x8, tanh)[0]
    close(y, want, x8.abs() * ref.PHI + (HALF[dtype] + 4 * u) * want.abs() + TINY, "gelu")
    v = ref.unpacked(kept.codes, kept.scales, cols)
    value, slope = ref.gelu(v, tanh)
    dx, again = ags.gelu_checkpointed_backward(dy, kept, tanh=tanh, with_output=True)
    want = dy.to(F8) * slope
    close(dx, want, dy.to(F8).abs() * (ref.SLOPE + 4 * u * slope.abs()) + HALF[dtype] * want.abs() + TINY, "gelu's slope")
    close(again, value, v.abs() * (ref.PHI + 2 * u) + (HALF[dtype] + 4 * u) * value.abs() + TINY, "gelu again")
    assert torch.equal(ags.gelu_checkpointed_backward(dy, kept, tanh=tanh), dx)


@pytest.mark.parametrize("tanh", [False, True])
def test_gelu_range(native, tanh):
    """Every bf16 number up to 2^30 in size, and fp32 over the range where gelu bends."""
    bits = torch.arange(0, 0x4E80, device=DEV, dtype=torch.int32).to(torch.int16)
    x = torch.cat([bits.view(BF16), -bits.view(BF16)]).view(-1, 64).contiguous()
    y = ags.gelu_checkpointed(x, tanh=tanh)[0]
    want = ref.gelu(x.to(F8), tanh)[0]
    close(y, want, x.to(F8).abs() * ref.PHI + (HALF[BF16] + 4 * u) * want.abs() + TINY, "gelu")
    x = torch.linspace(-12, 12, 1 << 16, device=DEV).view(512, 128)
    want = ref.gelu(x.to(F8), tanh)[0]
    close(ags.gelu_checkpointed(x, tanh=tanh)[0], want, x.to(F8).abs() * ref.PHI + 5 * u * want.abs() + TINY, "gelu")
    one = torch.tensor([[math.nan, 1.0, math.inf, 2.0]], device=DEV)
    y, kept = ags.gelu_checkpointed(one, tanh=tanh)
    assert y[0, 0].isnan() and y[0, 2] == math.inf and y[0, 1] > 0.84
    assert ags.gelu_checkpointed_backward(one, kept, tanh=tanh).isnan().all()


def test_gelu_difference(native):
    """The slope against the central difference of gelu at the kept values."""
    x, dy, step = 2 * randn(4, 256, seed=1), randn(4, 256, seed=2), 2.0 ** -6
    for tanh in (False, True):
        _, kept = ags.gelu_checkpointed(x, tanh=tanh)
        v = ags.checkpoint_unpack(kept)
        dx = ags.gelu_checkpointed_backward(dy, kept, tanh=tanh).to(F8)
        up, down = (ags.gelu_checkpointed(v + s * step, tanh=tanh)[0].to(F8) for s in (1, -1))
        got = dy.to(F8) * (up - down) / (2 * step)
        hi, lo = (v + step).to(F8), (v - step).to(F8)
        plain = dy.to(F8) * (ref.gelu(hi, tanh)[0] - ref.gelu(lo, tanh)[0]) / (2 * step)
        truth = dy.to(F8) * ref.gelu(v.to(F8), tanh)[1]
        tol = (plain - truth).abs() + dy.to(F8).abs() * ((hi.abs() + lo.abs()) * (ref.PHI + 6 * u) / (2 * step) + ref.SLOPE + 8 * u)
        assert ((got - dx).abs() <= tol).all()


@pytest.mark.parametrize("extra,shift", [(0, 1), (8, 0), (5, 0), (16, 3)])
@pytest.mark.parametrize("dtype", TYPES)
def test_checkpoints_strided(native, dtype, extra, shift):
    rows, cols = 21, 264
    x, dy = activations(rows, cols, dtype, 5), randn(rows, cols, seed=3, dtype=dtype)
    xs, dys = strided(x, extra, shift), strided(dy, extra, shift)
    for p, q in ((ags.checkpoint_pack(x), ags.checkpoint_pack(xs)), (ags.gelu_checkpointed(x)[1], ags.gelu_checkpointed(xs)[1])):
        assert torch.equal(p.codes[:, :cols], q.codes[:, :cols]) and torch.equal(p.scales, q.scales)
    assert torch.equal(ags.gelu_checkpointed(x)[0], ags.gelu_checkpointed(xs)[0])
    kept = ags.checkpoint_pack(x)
    assert torch.equal(ags.gelu_checkpointed_backward(dy, kept), ags.gelu_checkpointed_backward(dys, kept))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(33, 100), (129, 1024), (5, 2048), (3, 16383)])
def test_norm_checkpoint(native, rows, cols, dtype):
    """The forward pass is the same as without a checkpoint, and the codes are those of h."""
    x, (w, b) = activations(rows, cols, dtype, seed=cols), params(cols, FP32, seed=7)
    y, kept, rstd = ags.layer_norm_checkpointed(x, w, b)
    plain = ags.layer_norm(x, w, b)
    assert torch.equal(y, plain[0]) and torch.equal(rstd, plain[2])
    _, _, _, (h, h_tol) = ref.norm(x, w, b, 1e-5)
    got = ref.unpacked(kept.codes, kept.scales, cols)
    pad = (0, -cols % 128)
    top = torch.nn.functional.pad((h.abs() + h_tol), pad).view(rows, -1, 128).amax(2)
    step = (top / 254 * (1 + 200 * u)).repeat_interleave(128, 1)[:, :cols]
    close(got, h, step + 2 * h_tol + TINY, "h in 8 bits")


def test_empty_checkpoints(native):
    x = torch.empty(0, 100, dtype=BF16, device=DEV)
    kept = ags.checkpoint_pack(x)
    assert ags.checkpoint_unpack(kept).shape == (0, 100)
    y, kept = ags.gelu_checkpointed(x)
    assert ags.gelu_checkpointed_backward(x, kept).shape == (0, 100) and y.shape == (0, 100)


# ------------------------------------------------------- guards, streams, graphs, long tensors


class Guarded:
    """torch.empty and empty_like with 512 guard bytes after every CUDA tensor."""

    def __init__(self, monkeypatch):
        self.made, real = [], torch.empty

        def empty(*shape, dtype=None, device=None, **more):
            shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
            n = math.prod(shape) * torch.tensor([], dtype=dtype).element_size()
            buf = real(n + 512, dtype=torch.uint8, device=device).fill_(0xA5)
            self.made.append((buf, n))
            return buf[:n].view(dtype or FP32).view(shape)

        monkeypatch.setattr(torch, "empty", empty)
        monkeypatch.setattr(torch, "empty_like", lambda t: empty(*t.shape, dtype=t.dtype, device=t.device))

    def intact(self):
        assert self.made
        return all(bool((buf[n:] == 0xA5).all()) for buf, n in self.made)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (37, 100), (19, 1001), (64, 1024), (3, 4104), (5, 16383)])
def test_guards(native, monkeypatch, rows, cols, dtype):
    """Nothing is written past the end of an output, a checkpoint or the scratch memory."""
    x, dy, (w, b) = activations(rows, cols, dtype, 1), randn(rows, cols, seed=2, dtype=dtype), params(cols, dtype, 3)
    table, tokens = randn(50, cols, seed=4, dtype=dtype), skewed_tokens(rows, 50, seed=5)
    before = [t.clone() for t in (x, dy, w, b, table, tokens)]
    guard = Guarded(monkeypatch)
    offs = [0, rows // 2, rows]
    ags.embedding(table, tokens, scale=2.0)
    ags.embedding_backward(dy, tokens, 50, worker_offsets=offs)
    _, mean, rstd = ags.layer_norm(x, w, b)
    ags.layer_norm_backward(dy, x, mean, rstd, w, worker_offsets=offs)
    _, kept, rstd = ags.layer_norm_checkpointed(x, w, b)
    ags.layer_norm_checkpointed_backward(dy, kept, rstd, w, b, worker_offsets=offs, with_output=True)
    ags.checkpoint_unpack(ags.checkpoint_pack(x))
    _, kept = ags.gelu_checkpointed(x)
    ags.gelu_checkpointed_backward(dy, kept, with_output=True)
    torch.cuda.synchronize()
    assert guard.intact()
    assert all(torch.equal(p, q) for p, q in zip((x, dy, w, b, table, tokens), before))


def step(x, dy, w, b, table, tokens, offs):
    y, mean, rstd = ags.layer_norm(x, w, b)
    out = [y, *ags.layer_norm_backward(dy, x, mean, rstd, w, worker_offsets=offs)]
    y, kept, rstd = ags.layer_norm_checkpointed(x, w, b)
    out += [y, *ags.layer_norm_checkpointed_backward(dy, kept, rstd, w, b, worker_offsets=offs, with_output=True)]
    y, kept = ags.gelu_checkpointed(x)
    out += [y, ags.gelu_checkpointed_backward(dy, kept), ags.checkpoint_unpack(ags.checkpoint_pack(x))]
    out += [ags.embedding(table, tokens), *ags.embedding_backward(dy, tokens, table.shape[0], worker_offsets=offs)]
    return [t for o in out for t in (o if isinstance(o, list) else [o])]


def inputs(rows, cols, dtype, seed):
    w, b = params(cols, FP32, seed + 3)
    return (activations(rows, cols, dtype, seed), randn(rows, cols, seed=seed + 1, dtype=dtype), w, b,
            randn(3000, cols, seed=seed + 4, dtype=dtype), skewed_tokens(rows, 3000, seed=seed + 5))


def test_streams_overlap(native):
    """The same calls on four streams at once, without any order between them, and with the
    stream argument: the results of one stream."""
    offs = [0, 1000, 1700, 5000]
    args = [inputs(5000, 512, BF16, 10 * i) for i in range(4)]
    alone = [step(*a, offs) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in range(4)]
    for _ in range(5):
        got = []
        for s, a in zip(streams, args):
            with torch.cuda.stream(s):
                got.append(step(*a, offs))
        torch.cuda.synchronize()
        for g, w in zip(got, alone):
            assert all(torch.equal(p, q) for p, q in zip(g, w))
    x, dy, w, b, table, tokens = args[0]
    y, mean, rstd = ags.layer_norm(x, w, b, stream=streams[0])
    dx, dw, db = ags.layer_norm_backward(dy, x, mean, rstd, w, worker_offsets=offs, stream=streams[0])
    grads = ags.embedding_backward(dy, tokens, 3000, worker_offsets=offs, stream=streams[1])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip([y, dx, *dw, *db], alone[0]))
    assert all(torch.equal(p, q) for p, q in zip(grads, alone[0][-3:]))


def test_graph_capture_without_a_first_call(native):
    offs = [0, 300, 901]
    args = inputs(901, 384, BF16, 77)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*args, offs)
    want = None
    for seed in (1, 2):
        args[0].copy_(activations(901, 384, BF16, seed))
        args[5].copy_(skewed_tokens(901, 3000, seed))
        graph.replay()
        torch.cuda.synchronize()
        want = step(*args, offs)
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_offsets_beyond_32_bits(native):
    """More than 2^32 bytes and 2^31 elements in every tensor: first, middle and last rows."""
    cols = 8192
    rows = 2 ** 31 // cols + 3
    x = torch.empty(rows, cols, dtype=BF16, device=DEV)
    at = [0, 1, rows // 2, rows - 2, rows - 1]
    x.fill_(1.0)
    x[at] = randn(len(at), cols, seed=1, dtype=BF16)
    w, b = params(cols, FP32, 2)
    y, mean, rstd = ags.layer_norm(x, w, b)
    close(y[at], *ref.norm(x[at], w, b, 1e-5)[0], "y")
    dx = ags.layer_norm_backward(x, x, mean, rstd, w, parameter_grads=False)[0]
    small = ags.layer_norm_backward(x[at].clone(), x[at].clone(), mean[at].clone(), rstd[at].clone(), w, parameter_grads=False)[0]
    assert torch.equal(dx[at], small)
    del y, dx
    y, kept, rstd = ags.layer_norm_checkpointed(x, w, b)
    dx = ags.layer_norm_checkpointed_backward(x, kept, rstd, w, parameter_grads=False)[0]
    _, k2, r2 = ags.layer_norm_checkpointed(x[at].clone(), w, b)
    assert torch.equal(kept.codes[at], k2.codes) and torch.equal(kept.scales[at], k2.scales)
    assert torch.equal(dx[at], ags.layer_norm_checkpointed_backward(x[at].clone(), k2, r2, w, parameter_grads=False)[0])
    del y, dx, kept
    y, kept = ags.gelu_checkpointed(x)
    y2, k2 = ags.gelu_checkpointed(x[at].clone())
    assert torch.equal(y[at], y2) and torch.equal(kept.codes[at], k2.codes)
    dx = ags.gelu_checkpointed_backward(x, kept)
    assert torch.equal(dx[at], ags.gelu_checkpointed_backward(x[at].clone(), k2))
    del y, dx
    back = ags.checkpoint_unpack(kept)
    assert torch.equal(back[at], ags.checkpoint_unpack(k2))
    del back, kept
    # the table (and its gradient) beyond 2^31 elements, and the lookup's output
    tokens = torch.full((rows,), 5, device=DEV)
    tokens[at] = torch.tensor([rows - 1, 0, rows - 2, 3, rows - 1], device=DEV)
    got = ags.embedding(x, tokens)
    assert torch.equal(got[at], x[tokens[at]])
    del got
    few = tokens[at].clone()
    dy = randn(len(at), cols, seed=3, dtype=BF16)
    grad = ags.embedding_backward(dy, few, rows)[0]
    assert torch.equal(grad[rows - 2], dy[2]) and torch.equal(grad[3], dy[3]) and torch.equal(grad[0], dy[1])
    want = dy[0].to(F8) + dy[4].to(F8)
    close(grad[rows - 1], want, HALF[BF16] * want.abs() + 4 * u * (dy[0].to(F8).abs() + dy[4].to(F8).abs()), "last row")
    assert not grad[4:rows - 2].any()
    del grad
    # and the gradient's input: rows at both ends of a long dy
    skip = torch.full((rows,), -1, device=DEV)
    skip[at] = torch.tensor([0, 1, 2, 3, 4], device=DEV)
    assert torch.equal(ags.embedding_backward(x, skip, 5)[0], x[at])


def test_launches_are_the_librarys(native):
    before = ags.launch_count()
    x = randn(4, 64, seed=1)
    ags.layer_norm(x)
    assert ags.launch_count() == before + 1
    ags.profile_enable(True)
    try:
        ags.checkpoint_pack(x)
        torch.cuda.synchronize()
        stats = ags.profile_collect()
    finally:
        ags.profile_enable(False)
    assert stats["checkpoint_pack"][0] == 1


# --------------------------------------------------------------------------------- refusals


def test_refusals(native):
    x, (w, b) = activations(6, 64, BF16, 1), params(64, FP32, 2)
    y, mean, rstd = ags.layer_norm(x, w, b)
    table, tokens = randn(10, 64, seed=3), torch.arange(6, device=DEV)
    dy = randn(6, 64, seed=4, dtype=BF16)
    kept = ags.checkpoint_pack(x)
    bad = [
        (TypeError, lambda: ags.layer_norm(x.half())),
        (TypeError, lambda: ags.layer_norm([1.0])),
        (ValueError, lambda: ags.layer_norm(x.cpu())),
        (ValueError, lambda: ags.layer_norm(x.t())),
        (ValueError, lambda: ags.layer_norm(x[:, :0])),
        (ValueError, lambda: ags.layer_norm(x, w[:63], b)),
        (ValueError, lambda: ags.layer_norm(x, w, b.to(BF16))),
        (ValueError, lambda: ags.layer_norm(x, w, b, out=torch.empty(6, 64, device=DEV))),
        (ags.AdasumError, lambda: ags.layer_norm(x, w, b, out=x)),
        (ags.AdasumError, lambda: ags.layer_norm(x, w, b, eps=-1.0)),
        (ags.AdasumError, lambda: ags.layer_norm(x, w, b, eps=math.nan)),
        (ags.AdasumError, lambda: ags.layer_norm(torch.zeros(1, 16385, device=DEV))),
        (ValueError, lambda: ags.layer_norm_backward(dy.float(), x, mean, rstd, w)),
        (ValueError, lambda: ags.layer_norm_backward(dy[:5], x, mean, rstd, w)),
        (ValueError, lambda: ags.layer_norm_backward(dy, x, mean[:5], rstd, w)),
        (ValueError, lambda: ags.layer_norm_backward(dy, x, mean, rstd.to(F8), w)),
        (ValueError, lambda: ags.layer_norm_backward(dy, x, mean, rstd, w, worker_offsets=[0, 5])),
        (ags.AdasumError, lambda: ags.layer_norm_backward(dy, x, mean, rstd, w, worker_offsets=[0, 5, 3, 6])),
        (ags.AdasumError, lambda: ags.layer_norm_backward(dy, x, mean, rstd, w, worker_offsets=[1, 6])),
        (ags.AdasumError, lambda: ags.layer_norm_backward(dy, x, mean, rstd, w, worker_offsets=[0] * 257 + [6])),
        (ValueError, lambda: ags.layer_norm_backward(dy, x, mean, rstd, w, accumulate=True)),
        (ValueError, lambda: ags.layer_norm_backward(dy, x, mean, rstd, w, worker_offsets=[0, 3, 6], grad_weights=[w], grad_biases=[b])),
        (ags.AdasumError, lambda: ags.layer_norm_backward(dy, x, mean, rstd, w, grad_weights=w, grad_biases=b.clone())),
        (ags.AdasumError, lambda: ags.layer_norm_backward(dy, x, mean, rstd, None, grad_weights=b, grad_biases=b)),
        (ValueError, lambda: ags.layer_norm_checkpointed_backward(dy[:, :32], kept, rstd, w)),
        (ValueError, lambda: ags.layer_norm_checkpointed_backward(dy.float(), kept, rstd, w)),
        (TypeError, lambda: ags.layer_norm_checkpointed_backward(dy, (kept.codes, kept.scales), rstd, w)),
        (ValueError, lambda: ags.gelu_checkpointed_backward(dy, kept._replace(scales=kept.scales[:5]))),
        (ValueError, lambda: ags.checkpoint_unpack(kept._replace(codes=kept.codes[:, :48]))),
        (TypeError, lambda: ags.checkpoint_unpack(kept, dtype=torch.float16)),
        (ValueError, lambda: ags.checkpoint_unpack(kept, out=torch.empty(6, 64, device=DEV))),
        (TypeError, lambda: ags.checkpoint_pack(tokens)),
        (ags.AdasumError, lambda: ags.gelu_checkpointed(x, out=x)),
        (TypeError, lambda: ags.embedding(table, tokens.float())),
        (TypeError, lambda: ags.embedding(table, tokens.short())),
        (ValueError, lambda: ags.embedding(table, tokens.cpu())),
        (ValueError, lambda: ags.embedding(table.t(), tokens)),
        (ValueError, lambda: ags.embedding(table, tokens, out=torch.empty(5, 64, device=DEV))),
        (ags.AdasumError, lambda: ags.embedding(table, tokens, out=table[:6])),
        (ValueError, lambda: ags.embedding_backward(dy, tokens[:5], 10)),
        (ValueError, lambda: ags.embedding_backward(dy, tokens, -1)),
        (ValueError, lambda: ags.embedding_backward(dy, tokens, 10, accumulate=True)),
        (ValueError, lambda: ags.embedding_backward(dy, tokens, 10, grads=[table[:9]])),
        (ValueError, lambda: ags.embedding_backward(dy, tokens, 10, worker_offsets=[0, 2, 6], grads=[table, table.to(BF16)])),
        (ags.AdasumError, lambda: ags.embedding_backward(dy, tokens, 10, worker_offsets=[0, 2, 6], grads=[table, table])),
        (ags.AdasumError, lambda: ags.embedding_backward(dy, tokens, 6, grads=dy)),
    ]
    for i, (error, call) in enumerate(bad):
        before = ags.launch_count()
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was not refused")
        assert ags.launch_count() == before, f"call {i} launched something"


def test_refusals_of_the_c_entry(native):
    """Null pointers, bad sizes, types and strides, and scratch memory that is missing, too
    small or not aligned: a status, and nothing launched."""
    import ctypes
    lib = ags.load_library()
    x = activations(6, 64, FP32, 1)
    st = torch.empty(6, device=DEV)
    out, w = torch.empty(6, 64, device=DEV), torch.empty(64, device=DEV)
    i8 = torch.empty(6 * 64 + 16, dtype=torch.int8, device=DEV)
    offs = (ctypes.c_int64 * 2)(0, 6)
    p = lambda t: t.data_ptr()  # noqa: E731
    grads = (ctypes.c_void_p * 1)(p(w))
    null = (ctypes.c_void_p * 1)(None)
    BAD, ALIAS, BIG = 1, 3, 2
    norm = lambda **k: lib.adasum_layer_norm(*{**dict(x=p(x), rows=6, cols=64, ld=64, dt=0, w=None, b=None, wd=0, eps=1e-5, y=p(out), m=None, r=None, c=None, s=None, st=None), **k}.values())  # noqa: E731
    back = lambda **k: lib.adasum_layer_norm_backward(*{**dict(g=p(x), lg=64, x=p(x), lx=64, m=p(st), r=p(st), cols=64, dt=0, w=None, wd=0, o=offs, K=1, dx=p(out), dw=None, db=None, gd=0, acc=0, sc=None, sb=0, st=None), **k}.values())  # noqa: E731
    emb = lambda **k: lib.adasum_embedding_backward(*{**dict(g=p(x), cols=64, ld=64, dt=0, t=p(st), tb=4, o=offs, K=1, rows=1, sc=1.0, pad=-1, grads=grads, gd=0, acc=0, s=None, sb=0, st=None), **k}.values())  # noqa: E731
    before = ags.launch_count()
    assert norm(x=None) == BAD and norm(y=None) == BAD and norm(dt=2) == BAD and norm(wd=-1) == BAD
    assert norm(rows=-1) == BAD and norm(cols=0) == BAD and norm(ld=63) == BAD and norm(cols=16385, ld=16385) == BIG
    assert norm(c=p(i8)) == BAD and norm(c=p(i8) + 1, s=p(st)) == BAD and norm(y=p(x) + 4) == ALIAS and norm(rows=1 << 40) == BIG
    assert back(g=None) == BAD and back(m=None) == BAD and back(r=None) == BAD and back(dx=None) == BAD
    assert back(o=None) == BAD and back(K=0) == BAD and back(K=257) == BIG and back(lg=1) == BAD and back(lx=1) == BAD
    assert back(dw=null) == BAD and back(gd=7) == BAD and back(dx=p(x)) == ALIAS
    assert emb(g=None) == BAD and emb(t=None) == BAD and emb(tb=2) == BAD and emb(grads=None) == BAD
    assert emb(grads=null) == BAD and emb(rows=-1) == BAD and emb(cols=0) == BAD and emb(K=300) == BIG
    assert norm(x=p(x) + 2) == BAD and norm(m=p(st) + 1) == BAD and norm(ld=1 << 62) == BAD
    assert back(g=p(x) + 1) == BAD and back(dx=p(out) + 2) == BAD and emb(t=p(st) + 2) == BAD
    assert lib.adasum_embedding(p(x), 6, 64, 0, p(st), 8, -1, 1.0, p(out), None) == BAD
    assert lib.adasum_embedding(p(x), 6, 64, 0, p(st), 8, 1 << 40, 1.0, p(out), None) == BIG
    assert lib.adasum_checkpoint_pack(p(x), 6, 64, 64, 0, p(i8) + 8, p(st), None) == BAD
    assert lib.adasum_checkpoint_pack(p(x), 6, 64, 64, 0, None, p(st), None) == BAD
    assert lib.adasum_checkpoint_unpack(p(i8), None, 6, 64, 0, p(out), None) == BAD
    assert lib.adasum_gelu_checkpointed(p(x), 6, 64, 64, 0, 0, None, p(i8), p(st), None) == BAD
    assert lib.adasum_gelu_checkpointed_backward(None, 64, p(i8), p(st), 6, 64, 0, 0, p(out), None, None) == BAD
    assert lib.adasum_gelu_checkpointed_backward(p(x), 64, p(i8), p(st), 6, 64, 0, 0, p(out), p(out), None) == ALIAS
    assert ags.launch_count() == before
