"""The table gradient of very many tokens: right, and in time proportional to their number."""
import statistics

import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
from test_gpu_training import BF16, DEV, FP32, TYPES, check_table_gradient, gen, randn, skewed_tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n_rows,offs", [(1000, [0, 70_001]), (50_304, [0, 300_000]), (300, [0, 5, 5, 131_072, 131_073, 400_000]),
                                         (70_000, [0, 1_050_000])])
def test_many_tokens(native, n_rows, offs, accumulate):
    """Workers of 65 to 1026 tiles of tokens, beside short and empty ones; one and two digits, and three."""
    tokens = skewed_tokens(offs[-1], n_rows, seed=n_rows, dtype=torch.int32 if n_rows % 2 else torch.int64)
    check_table_gradient(n_rows, 8, offs, BF16, FP32, accumulate, tokens)


@pytest.mark.parametrize("kind", ["same", "all different", "two", "none"])
def test_many_tokens_runs(native, kind):
    rows, n = 600_000, 500_000
    at = torch.arange(n, device=DEV)
    tokens = {"same": torch.full_like(at, 12345), "all different": rows - 1 - at, "two": 7 + (at * 7919 % 97 < 40).long(),
              "none": torch.full_like(at, -1)}[kind]
    check_table_gradient(rows, 4, [0, n // 3, n], BF16, FP32, False, tokens, seed=n)


@pytest.mark.parametrize("dtype", TYPES)
def test_equal_calls_give_equal_bits(native, dtype):
    n, rows, cols = 200_000, 5000, 24
    tokens, dy = skewed_tokens(n, rows, seed=4), randn(n, cols, seed=5, dtype=dtype)
    first = ags.embedding_backward(dy, tokens, rows)[0]
    for _ in range(3):
        assert torch.equal(ags.embedding_backward(dy, tokens, rows)[0], first)


def test_time_is_proportional_to_tokens(native):
    """Eight times the tokens of one worker: 8 times the bytes.  A cost per pair of tiles would
    be 64 times as much, so twice the proportion is the limit (and the smaller call has launches
    and latencies to hide, which only makes its time longer)."""
    rows, cols, ms = 50_304, 8, {}
    for n in (1 << 20, 1 << 23):
        dy, grad = randn(n, cols, seed=1, dtype=BF16), torch.zeros(rows * cols, device=DEV)
        tokens = torch.randint(0, rows, (n,), generator=gen(2), device=DEV, dtype=torch.int32)
        times = []
        for _ in range(7):
            start, stop = torch.cuda.Event(True), torch.cuda.Event(True)
            start.record()
            ags.embedding_backward(dy, tokens, rows, grads=grad, accumulate=True)
            stop.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(stop))
        ms[n] = statistics.median(times)
    assert ms[1 << 23] <= 16 * ms[1 << 20], ms
