"""Nothing is written past the scratch memory that the training operators ask for."""
import ctypes

import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
from test_gpu_training import BF16, DEV, TYPES, Guarded, activations, params, randn, skewed_tokens

pytestmark = pytest.mark.gpu


def scratch_bytes(name, offs, *sizes):
    lib = ags.load_library()
    return getattr(lib, name + "_scratch_bytes")((ctypes.c_int64 * len(offs))(*offs), len(offs) - 1, *sizes)


def ragged(n, K):
    return [0] + [n * k // K + k % 3 for k in range(1, K)] + [n]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("offs,cols", [([0, 300], 40), ([0, 4096], 264), ([0, 5000], 40), (ragged(70_000, 3), 256), (ragged(70_000, 5), 769),
                                       (ragged(150_000, 2), 8), ([0, 200_000], 200), (ragged(76_800, 256), 24)])
def test_scratch_of_the_table_gradient(native, monkeypatch, offs, cols, accumulate):
    """Nothing is written past the scratch memory that a call asks for, in each form of it."""
    rows, n = 5000, offs[-1]
    assert scratch_bytes("adasum_embedding_backward", offs, rows, cols) > 0
    dy, tokens = randn(n, cols, seed=2, dtype=BF16), skewed_tokens(n, rows, seed=5)
    grads = list(torch.zeros(len(offs) - 1, rows * cols, device=DEV).unbind(0))
    guard = Guarded(monkeypatch)
    ags.embedding_backward(dy, tokens, rows, worker_offsets=offs, grads=grads, accumulate=accumulate)
    ags.embedding_backward(dy, torch.full_like(tokens, 3), rows, worker_offsets=offs, grads=grads, accumulate=accumulate)
    torch.cuda.synchronize()
    assert guard.intact()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offs,cols,some", [([0, 3000], 100, True), (ragged(3000, 7), 100, False), (ragged(9000, 7), 100, True),
                                            ([0, 300], 16_383, True), ([0, 900], 16_384, True), (ragged(2560, 256), 1000, True),
                                            (list(range(257)), 264, True)])
def test_scratch_of_the_norm_gradient(native, monkeypatch, offs, cols, some, dtype):
    """The same of its partial sums; few rows a worker (429 of 100 columns) need none."""
    rows = offs[-1]
    assert (scratch_bytes("adasum_layer_norm_backward", offs, cols) > 0) is some
    x, dy, (w, b) = activations(rows, cols, dtype, 1), randn(rows, cols, seed=2, dtype=dtype), params(cols, dtype, 3)
    guard = Guarded(monkeypatch)
    _, mean, rstd = ags.layer_norm(x, w, b)
    ags.layer_norm_backward(dy, x, mean, rstd, w, worker_offsets=offs)
    _, kept, rstd = ags.layer_norm_checkpointed(x, w, b)
    ags.layer_norm_checkpointed_backward(dy, kept, rstd, w, b, worker_offsets=offs, with_output=True)
    torch.cuda.synchronize()
    assert guard.intact()
