"""What the position bias' kernels read in 16-byte pieces stays inside the scores (of one head and
sequence, where the output may be the scores themselves), whatever boundary they begin and end on.
The test build checks every such read; what lies beside the scores is NaN."""
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


def randn(*shape, seed, dtype):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(dtype)


def placed(x, at, stride):
    """x at `at` elements from a 16-byte boundary, its rows `stride` apart, the last one's padding
    left out; NaN around it."""
    b, h, q, k = x.shape
    room = torch.full((at + b * h * q * stride + 64,), math.nan, dtype=x.dtype, device=DEV)
    view = room.as_strided((b, h, q, k), (h * q * stride, q * stride, stride, 1), at)
    return view.copy_(x)


# batch, heads, queries, keys: single values, rows shorter than a piece, one piece, ends inside
# one, units of many rows, two units of keys, two and more CTAs, one and more workers' sequences
SIZES = [(1, 1, 1, 1), (2, 3, 1, 1), (3, 2, 5, 1), (2, 2, 3, 3), (1, 4, 1, 7), (2, 1, 9, 9), (1, 1, 2, 255), (1, 2, 33, 257),
         (5, 3, 17, 63), (3, 1, 300, 31), (1, 1, 3, 9000), (70, 1, 3, 13), (9, 1, 2, 4101)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,heads,queries,keys", SIZES)
def test_dense_scores(native, hooks, batch, heads, queries, keys, dtype):
    assert ags.get_last_error() == ags.Status.OK
    table = randn(32, heads, seed=1, dtype=FP32)
    x = randn(batch, heads, queries, keys, seed=2, dtype=dtype)
    index = more.bucket_matrix(queries, keys, 3, 32, True, 128, DEV)
    want = x.to(F8) + table.to(F8)[index].permute(2, 0, 1)
    tol = (u + HALF[dtype]) * want.abs() + TINY
    for at in range(16 // dtype.itemsize):
        scores = placed(x, at, keys)
        out = placed(x, at, keys)
        close(ags.relative_position_bias(table, queries, keys, offset=3, scores=scores, out=out), want, tol, f"at {at}")
        assert ags.relative_position_bias(table, queries, keys, offset=3, scores=scores, out=scores) is scores
        close(scores, want, tol, f"at {at}, in place")
        assert ags.get_last_error() == ags.Status.OK


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,heads,queries,keys", SIZES)
def test_gradient(native, hooks, batch, heads, queries, keys, dtype):
    """Dense and behind strides: of the next 16-byte boundary (so that all rows begin on one), and odd."""
    assert ags.get_last_error() == ags.Status.OK
    piece = 16 // dtype.itemsize
    x = randn(batch, heads, queries, keys, seed=3, dtype=dtype)
    offs = [0, batch // 2, batch]
    index = more.bucket_matrix(queries, keys, 2, 32, True, 128, DEV)
    want = more.bias_gradient(x, index, 32, offs, None, dtype)
    for at in range(piece):
        for stride in (keys, -(-keys // piece) * piece, keys + 3):
            got = ags.relative_position_bias_backward(placed(x, at, stride), 32, offset=2, worker_offsets=offs)
            for k, (value, tol) in enumerate(want):
                close(got[k], value, tol, f"at {at}, stride {stride}, worker {k}")
            assert ags.get_last_error() == ags.Status.OK
