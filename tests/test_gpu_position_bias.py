"""The relative position bias and its table's gradient on the GPU against plain 64-bit forms."""
import math

import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
import more_reference as more
from training_reference import F8, HALF, TINY, close, u

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
TYPES = [BF16, FP32]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(*shape, seed=0, dtype=FP32, std=1.0):
    return (std * torch.randn(*shape, generator=gen(seed), device=DEV)).to(dtype)


# batch, heads, queries, keys, offset: single tokens, rows and keys around the tiles' (4, 32, 128,
# 256), offsets on both sides, keys far beyond the last border
SIZES = [(1, 1, 1, 1, 0), (3, 2, 1, 9, 8), (2, 3, 5, 5, 0), (8, 4, 1, 513, 512), (1, 2, 33, 31, 0), (2, 2, 130, 257, 127),
         (1, 1, 3, 1000, 0), (5, 3, 17, 64, -20), (1, 2, 300, 300, 0), (2, 1, 64, 520, 456), (40, 1, 8, 16, 8), (1, 5, 7, 24, 1000)]
RULES = [(32, True, 128), (32, False, 128), (8, True, 64), (16, False, 100), (64, True, 300), (2, False, 2), (4, True, 2), (7, False, 50),
         (256, True, 2000), (32, True, 9)]


@pytest.mark.parametrize("buckets,both,distance", RULES)
def test_every_distance(native, buckets, both, distance):
    """The bucket of every relative position up to beyond the last border."""
    span = 2 * distance + 50
    table = torch.arange(buckets, dtype=FP32, device=DEV)[:, None].contiguous()
    got = ags.relative_position_bias(table, 1, 2 * span, offset=span, bidirectional=both, max_distance=distance)[0, 0]
    want = [more.bucket(k - span, buckets, both, distance) for k in range(2 * span)]
    assert got.int().tolist() == want


@pytest.mark.parametrize("buckets,both,distance", [(32, True, 128), (16, False, 100)])
@pytest.mark.parametrize("tdtype", TYPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,heads,queries,keys,offset", SIZES)
def test_bias(native, batch, heads, queries, keys, offset, dtype, tdtype, buckets, both, distance):
    table = randn(buckets, heads, seed=1, dtype=tdtype)
    index = more.bucket_matrix(queries, keys, offset, buckets, both, distance, DEV)
    bias = table.to(F8)[index].permute(2, 0, 1)
    kw = dict(bidirectional=both, max_distance=distance, offset=offset)
    alone = ags.relative_position_bias(table, queries, keys, **kw)
    assert alone.dtype == tdtype and torch.equal(alone.to(F8), bias)
    scores = randn(batch, heads, queries, keys, seed=2, dtype=dtype, std=3.0)
    got = ags.relative_position_bias(table, queries, keys, scores=scores, **kw)
    want = scores.to(F8) + bias
    assert got.dtype == dtype
    close(got, want, (u + HALF[dtype]) * want.abs() + TINY)
    inplace = scores.clone()
    assert ags.relative_position_bias(table, queries, keys, scores=inplace, out=inplace, **kw) is inplace
    assert torch.equal(inplace, got)


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_scores_and_strides(native, dtype):
    table = randn(32, 3, seed=1)
    x = randn(2, 3, 20, 40, seed=2, dtype=dtype)
    x[0, 1, 3] = -math.inf
    x[1, :, 5, 7] = math.nan
    x[1, 0, 6, 8] = torch.finfo(dtype).min
    want = ags.relative_position_bias(table, 20, 40, scores=x)
    assert (want[0, 1, 3] == -math.inf).all() and torch.isnan(want[1, :, 5, 7]).all()
    assert float(want[1, 0, 6, 8]) <= float(torch.finfo(dtype).min) / 2
    other = x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)     # heads behind queries
    wide = torch.full((2, 3, 20, 43), math.nan, dtype=dtype, device=DEV)[..., 1:41]
    wide.copy_(x)
    padded = torch.full((2, 3, 24, 48), math.nan, dtype=dtype, device=DEV)[:, :, 2:22, 8:]
    padded.copy_(x)
    for view in (other, wide, padded):
        got = ags.relative_position_bias(table, 20, 40, scores=view)
        assert torch.equal(torch.nan_to_num(got.float(), 1.0), torch.nan_to_num(want.float(), 1.0))


GRADS = [(1, 1, 1, 1, 0, [0, 1]), (3, 2, 1, 9, 8, [0, 1, 3]), (2, 3, 5, 5, 0, [0, 2]), (8, 4, 1, 513, 512, [0, 3, 3, 8]),
         (1, 2, 33, 31, 0, [0, 1]), (6, 2, 130, 257, 127, [0, 2, 6]), (1, 1, 3, 1000, 0, [0, 1]), (5, 3, 17, 64, -20, [0, 5]),
         (2, 2, 300, 300, 0, [0, 1, 2]), (40, 1, 8, 16, 8, [0, 40]), (1, 5, 7, 24, 1000, [0, 1]), (3, 2, 600, 520, 0, [0, 3]),
         (20, 12, 128, 128, 0, [0, 4, 8, 12, 16, 20])]


@pytest.mark.parametrize("buckets,both,distance", [(32, True, 128), (16, False, 100), (64, True, 300)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,heads,queries,keys,offset,offs", GRADS)
def test_gradient(native, batch, heads, queries, keys, offset, offs, dtype, buckets, both, distance):
    d = randn(batch, heads, queries, keys, seed=1, dtype=dtype)
    index = more.bucket_matrix(queries, keys, offset, buckets, both, distance, DEV)
    kw = dict(bidirectional=both, max_distance=distance, offset=offset, worker_offsets=offs)
    for gdtype, accumulate in ((FP32, False), (BF16, True)):
        old = [randn(buckets, heads, seed=5 + k, dtype=gdtype) for k in range(len(offs) - 1)]
        grads = [g.clone() for g in old]
        got = ags.relative_position_bias_backward(d, buckets, grads=grads, accumulate=accumulate, **kw)
        for k, (want, tol) in enumerate(more.bias_gradient(d, index, buckets, offs, old if accumulate else None, gdtype)):
            assert got[k] is grads[k]
            close(got[k], want, tol, f"worker {k}")
    fresh = ags.relative_position_bias_backward(d, buckets, **kw)
    assert len(fresh) == len(offs) - 1 and fresh[0].shape == (buckets, heads) and fresh[0].dtype == dtype


@pytest.mark.parametrize("buckets,both,distance", RULES)
def test_gradient_counts_exactly(native, buckets, both, distance):
    """Ones are counted: which value goes to which bucket, exactly."""
    for queries, keys, offset in ((70, 90, 20), (1, 700, 300), (290, 280, 0), (500, 40, 0)):
        d = torch.ones(2, 1, queries, keys, device=DEV)
        index = more.bucket_matrix(queries, keys, offset, buckets, both, distance, DEV)
        got = ags.relative_position_bias_backward(d, buckets, bidirectional=both, max_distance=distance, offset=offset)[0]
        assert got[:, 0].long().tolist() == (2 * torch.bincount(index.flatten(), minlength=buckets)).tolist()


@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_strides(native, dtype):
    for queries, keys in ((20, 40), (65, 77)):
        x = randn(4, 3, queries, keys, seed=2, dtype=dtype)
        index = more.bucket_matrix(queries, keys, 0, 32, True, 128, DEV)
        other = x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        wide = torch.full((4, 3, queries, keys + 3), math.nan, dtype=dtype, device=DEV)[..., 1:keys + 1]
        padded = torch.full((4, 3, queries + 4, (keys + 15) // 8 * 8), math.nan, dtype=dtype, device=DEV)[:, :, 2:queries + 2, 8 - 8:keys]
        for view in (other, wide, padded):
            view.copy_(x)
            got = ags.relative_position_bias_backward(view, 32, worker_offsets=[0, 1, 4], grads=[torch.empty(32, 3, device=DEV) for _ in range(2)])
            for k, (want, tol) in enumerate(more.bias_gradient(x, index, 32, [0, 1, 4], None, FP32)):
                close(got[k], want, tol, f"worker {k}")


def test_gradient_of_many(native):
    """Units by sequences, queries and keys; several CTAs a head; joined sums."""
    d = randn(70, 4, 300, 600, seed=3, dtype=BF16)
    offs = [0, 33, 33, 34, 70]
    index = more.bucket_matrix(300, 600, 300, 32, True, 128, DEV)
    got = ags.relative_position_bias_backward(d, 32, offset=300, worker_offsets=offs, grads=[torch.empty(32, 4, device=DEV) for _ in range(4)])
    for k, (want, tol) in enumerate(more.bias_gradient(d, index, 32, offs, None, FP32)):
        close(got[k], want, tol, f"worker {k}")
    again = ags.relative_position_bias_backward(d, 32, offset=300, worker_offsets=offs, grads=[torch.empty(32, 4, device=DEV) for _ in range(4)])
    assert all(torch.equal(a, b) for a, b in zip(got, again)) and not got[1].any()


def test_difference(native):
    table, s, d = randn(16, 2, seed=1), randn(2, 2, 9, 12, seed=2), randn(2, 2, 9, 12, seed=3)

    def loss(t):
        return float((ags.relative_position_bias(t, 9, 12, max_distance=20, offset=3, scores=s).double() * d.double()).sum())

    grad = ags.relative_position_bias_backward(d, 16, max_distance=20, offset=3)[0]
    for b in range(16):
        e = torch.zeros_like(table)
        e[b, b % 2] = 0.5
        diff = loss(table + e) - loss(table - e)  # linear: exact but for rounding
        assert abs(diff - float(grad[b, b % 2])) < 1e-3


def test_far_positions(native):
    """Positions and offsets beyond 32 bits."""
    table = randn(32, 1, seed=1)
    for offset in (2 ** 33, -2 ** 33, 2 ** 61, -2 ** 61):
        index = more.bucket(-offset, 32, True, 128)
        got = ags.relative_position_bias(table, 2, 8, offset=offset)
        assert torch.equal(got, table[index].expand(1, 2, 8))
        grad = ags.relative_position_bias_backward(torch.ones(1, 1, 2, 8, device=DEV), 32, offset=offset)[0]
        assert float(grad[index]) == 16 and float(grad.sum()) == 16


def test_empty(native):
    table = randn(32, 3, seed=1)
    assert ags.relative_position_bias(table, 0, 5).shape == (3, 0, 5)
    assert ags.relative_position_bias(table, 5, 0).shape == (3, 5, 0)
    guard = torch.full((3 * 4 * 5,), 7.0, device=DEV)
    assert ags.relative_position_bias(table, 4, 5, scores=torch.empty(0, 3, 4, 5, device=DEV)).shape == (0, 3, 4, 5)
    assert (guard == 7).all()
    for shape in ((0, 3, 4, 5), (2, 3, 0, 5), (2, 3, 4, 0)):
        d = torch.empty(shape, device=DEV)
        grads = [randn(32, 3, seed=2)]
        kept = grads[0].clone()
        ags.relative_position_bias_backward(d, 32, grads=grads, accumulate=True)
        assert torch.equal(grads[0], kept)
        ags.relative_position_bias_backward(d, 32, grads=grads)
        assert not grads[0].any()


def test_streams_and_capture(native):
    table, x = randn(32, 12, seed=1), randn(8, 12, 128, 128, seed=2, dtype=BF16)
    want, back = ags.relative_position_bias(table, 128, 128, scores=x), ags.relative_position_bias_backward(x, 32, worker_offsets=[0, 3, 8])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = ags.relative_position_bias(table, 128, 128, scores=x, stream=s)
    got_back = ags.relative_position_bias_backward(x, 32, worker_offsets=[0, 3, 8], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(got_back, back))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ags.relative_position_bias(table, 128, 128, scores=x)
        g = ags.relative_position_bias_backward(y, 32, worker_offsets=[0, 3, 8])
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    y2 = ags.relative_position_bias(table, 128, 128, scores=x)
    assert torch.equal(y, y2)
    assert all(torch.equal(a, b) for a, b in zip(g, ags.relative_position_bias_backward(y2, 32, worker_offsets=[0, 3, 8])))


def test_guards(native, monkeypatch):
    from adaptive_gradient_summation_gb300 import training as module
    guards = []

    def guarded(nbytes, index):
        if nbytes <= 0:
            return None
        t = torch.full((nbytes + 512,), 171, dtype=torch.uint8, device=DEV)
        guards.append(t[nbytes:])
        return t[:nbytes]

    monkeypatch.setattr(module, "_scratch", guarded)
    d = randn(70, 4, 300, 520, seed=3, dtype=BF16)
    flat = torch.full((2 * (32 * 4 + 16),), 7.0, device=DEV)
    grads = [flat[:128], flat[144:272]]
    ags.relative_position_bias_backward(d, 32, worker_offsets=[0, 30, 70], grads=grads)
    torch.cuda.synchronize()
    assert guards and all((g == 171).all() for g in guards)
    assert (flat[128:144] == 7).all() and (flat[272:] == 7).all()
    table = randn(32, 4, seed=1)
    for keys in (40, 37):
        buf = torch.full((4 * 20 * keys + 64,), 7.0, device=DEV)
        ags.relative_position_bias(table, 20, keys, out=buf[32:-32].view(4, 20, keys))
        assert (buf[:32] == 7).all() and (buf[-32:] == 7).all()


def test_refusals(native):
    table, x = randn(32, 3, seed=1), randn(2, 3, 4, 8, seed=2)
    for call in (lambda: ags.relative_position_bias(table.half(), 4, 8), lambda: ags.relative_position_bias(table, 4, 8, scores=x.half()),
                 lambda: ags.relative_position_bias_backward(x.long(), 32)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: ags.relative_position_bias(table[0], 4, 8), lambda: ags.relative_position_bias(table.t(), 4, 8),
                 lambda: ags.relative_position_bias(table, 4, 9, scores=x), lambda: ags.relative_position_bias(table, -1, 8),
                 lambda: ags.relative_position_bias(table, 4, 8, scores=x[0]), lambda: ags.relative_position_bias(table, 4, 8, scores=x, out=x[0]),
                 lambda: ags.relative_position_bias(table, 8, 4, scores=x.transpose(2, 3)),
                 lambda: ags.relative_position_bias(table, 4, 8, scores=x[:1].expand(2, 3, 4, 8)),
                 lambda: ags.relative_position_bias_backward(x, 0), lambda: ags.relative_position_bias_backward(x, 32, accumulate=True),
                 lambda: ags.relative_position_bias_backward(x, 32, worker_offsets=[0, 3]),
                 lambda: ags.relative_position_bias_backward(x, 32, grads=[table[:16]])):
        with pytest.raises(ValueError):
            call()
    for kw in (dict(max_distance=8), dict(max_distance=0), dict(max_distance=2 ** 31), dict(offset=2 ** 62)):
        with pytest.raises(ags.AdasumError):
            ags.relative_position_bias(table, 4, 8, **kw)
        with pytest.raises(ags.AdasumError):
            ags.relative_position_bias_backward(x, 32, **kw)
    for rows in (1, 2, 3, 31, 258):
        with pytest.raises(ags.AdasumError):
            ags.relative_position_bias(randn(rows, 3), 4, 8, max_distance=500)
    buf = torch.zeros(2 * 3 * 4 * 8 + 1, device=DEV)
    with pytest.raises(ags.AdasumError):  # shifted by one element
        ags.relative_position_bias(table, 4, 8, scores=buf[1:].view(2, 3, 4, 8), out=buf[:-1].view(2, 3, 4, 8))
    with pytest.raises(ags.AdasumError):
        ags.relative_position_bias_backward(x, 16, grads=[x.view(-1)[:48]])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,heads,queries,keys", [(2, 3, 37, 1), (2, 3, 37, 5), (1, 2, 5, 127), (2, 2, 33, 255), (2, 1, 40, 257),
                                                      (70, 1, 3, 263), (1, 2, 34, 511), (3, 1, 9, 514),
                                                      (2, 1, 9000, 1), (2, 2, 3, 8191), (1, 2, 2, 8195)])
def test_rows_that_begin_anywhere(native, batch, heads, queries, keys, dtype):
    """Dense scores whose rows are no multiple of 16 bytes, at every offset from a 16-byte
    boundary, the output at the same one or another, and in place; nothing beside it is written."""
    table = randn(32, heads, seed=1)
    size = batch * heads * queries * keys
    x = randn(batch, heads, queries, keys, seed=2, dtype=dtype, std=3.0)
    index = more.bucket_matrix(queries, keys, 7, 32, True, 128, DEV)
    want = x.to(F8) + table.to(F8)[index].permute(2, 0, 1)
    tol = (u + HALF[dtype]) * want.abs() + TINY
    for at in range(16 // dtype.itemsize):
        source = torch.full((size + 32,), math.nan, dtype=dtype, device=DEV)
        scores = source[at:at + size].view_as(x).copy_(x)
        for to in (at, at + 16, at + 3):
            room = torch.full((size + 64,), 77.0, dtype=dtype, device=DEV)
            got = ags.relative_position_bias(table, queries, keys, offset=7, scores=scores, out=room[to:to + size].view_as(x))
            close(got, want, tol, f"{at} to {to}")
            assert (room[:to] == 77).all() and (room[to + size:] == 77).all()
        assert ags.relative_position_bias(table, queries, keys, offset=7, scores=scores, out=scores) is scores
        close(scores, want, tol, f"{at} in place")
        assert torch.isnan(source[:at]).all() and torch.isnan(source[at + size:]).all()
    alone = torch.full((heads * queries * keys + 16,), 77.0, device=DEV)
    for at in range(4):
        got = ags.relative_position_bias(table, queries, keys, offset=7, out=alone[at:at + heads * queries * keys].view(heads, queries, keys))
        assert torch.equal(got, table[index].permute(2, 0, 1))
        assert (alone[at + heads * queries * keys:] == 77).all()


@pytest.mark.parametrize("buckets,both,distance", [(32, False, 4096), (24, True, 1000), (64, True, 65536), (48, False, 10 ** 6), (256, False, 2 ** 31 - 1)])
def test_borders_of_wide_rules(native, buckets, both, distance):
    """Positions next to where each bucket begins, found by bisection in whole numbers."""
    table = torch.arange(buckets, dtype=FP32, device=DEV)[:, None].contiguous()
    n = buckets // 2 if both else buckets
    for j in range(n // 2, n, max(1, n // 24)):
        lo, hi = 0, distance
        while lo < hi:
            at = (lo + hi) // 2
            lo, hi = (lo, at) if more.bucket(-at, n, False, distance) >= j else (at + 1, hi)
        got = ags.relative_position_bias(table, 1, 5, offset=lo + 2, bidirectional=both, max_distance=distance)[0, 0]
        assert got.int().tolist() == [more.bucket(k - lo - 2, buckets, both, distance) for k in range(5)]
