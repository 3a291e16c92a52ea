"""CPU checks of what the root-mean-square norm, the position bias and the updates refuse before
any GPU work, and of the sizes the library answers without a GPU."""
import ctypes
import os
import re
from array import array

import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
from adaptive_gradient_summation_gb300 import training, updates

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "adasum.h")


def test_cpu_tensors_are_refused():
    x, s = torch.zeros(4, 8), torch.zeros(2, 3, 4, 8)
    kept = ags.Checkpoint(torch.zeros(4, 16, dtype=torch.int8), torch.zeros(4, 1), x.shape, x.dtype)
    for call in (lambda: ags.rms_norm(x), lambda: ags.rms_norm_checkpointed(x, residual=x), lambda: ags.rms_norm_backward(x, x, x[:, 0]),
                 lambda: ags.rms_norm_checkpointed_backward(x, kept, x[:, 0]), lambda: ags.relative_position_bias(torch.zeros(32, 3), 4, 8),
                 lambda: ags.relative_position_bias_backward(s, 32), lambda: ags.orthogonalize(x),
                 lambda: ags.muon_step(x[0], [0, 8], [(2, 4)], x[1], x[2], lr=0.1)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_matrices_of_views():
    x = torch.zeros(2, 3, 6, 8)
    assert updates._matrices(x) == (6, 6, 8, 48, 8)
    assert updates._matrices(x[..., :5]) == (6, 6, 5, 48, 8)
    assert updates._matrices(x[:, 1]) == (2, 6, 8, 144, 8)
    assert updates._matrices(x[0, 0, ::2]) == (1, 3, 8, 48, 16)
    assert updates._matrices(x[..., :1, :]) == (6, 1, 8, 48, 8)
    assert updates._matrices(x[:0])[0] == 0
    for bad in (x.transpose(2, 3), x.transpose(0, 1), x[..., ::2], x[0, 0, 0], x[0, 0, :1].expand(4, 8)):
        with pytest.raises(ValueError):
            updates._matrices(bad)


def test_coefficients():
    assert list(updates._coefficients((1, 2, 3), 2)) == [1, 2, 3, 1, 2, 3]
    assert list(updates._coefficients([(1, 2, 3), (4, 5, 6)], 2)) == [1, 2, 3, 4, 5, 6]
    assert list(updates._coefficients([(1, 2, 3)] * 3, 3)) == [1, 2, 3] * 3
    for bad, steps in (((1, 2), 5), ([(1, 2, 3)], 2), ([(1, 2)], 1), ((1, 2, 3), 0)):
        with pytest.raises(ValueError):
            updates._coefficients(bad, steps)


def test_scores_of_views():
    s = torch.zeros(2, 3, 4, 8)
    assert training._scores(s, "s") == (s.shape, (96, 32, 8))
    assert training._scores(s.permute(0, 2, 1, 3), "s")[1] == (96, 8, 32)
    for bad in (s[0], s.transpose(2, 3), s[:1].expand(2, 3, 4, 8), s[..., ::2]):
        with pytest.raises(ValueError):
            training._scores(bad, "s")


def test_scratch_sizes():
    lib = ags.load_library()
    # nothing to do, or refused: no scratch
    for args in ((0, 4, 4, 0), (1, 0, 4, 0), (1, 4, 0, 0), (1, 65537, 4, 0), (-1, 4, 4, 0)):
        assert lib.adasum_orthogonalize_scratch_bytes(*args) == 0
    # some ten bytes an element, and no more than about a gigabyte at a time
    one = lib.adasum_orthogonalize_scratch_bytes(1, 1024, 4096, 0)
    assert 8 * 1024 * 4096 < one < 12 * 1024 * 4096
    assert lib.adasum_orthogonalize_scratch_bytes(1, 4096, 1024, 0) == one
    assert lib.adasum_orthogonalize_scratch_bytes(10000, 1024, 1024, 0) < 1.1 * 2 ** 30
    assert lib.adasum_orthogonalize_scratch_bytes(1, 16384, 16384, 0) > 2 ** 31  # (one matrix is not split)

    def step(shapes):
        rows, cols = (array("q", [s[i] for s in shapes]) for i in (0, 1))
        return lib.adasum_muon_step_scratch_bytes(rows.buffer_info()[0], cols.buffer_info()[0], len(shapes))

    assert step([(0, 0)]) == 0 and step([(5, 0), (0, 7)]) == 0 and step([(70000, 2)]) == 0
    assert step([(64, 128)]) == step([(0, 0), (128, 64)]) > 0
    assert step([(64, 128)] * 3 + [(32, 32)]) > step([(64, 128)] * 3)  # together in one launch
    assert step([(1024, 4096)] * 100) < 1.1 * 2 ** 30
    offs = array("q", [0, 3, 40])
    size = lambda *a: lib.adasum_relative_position_bias_backward_scratch_bytes(offs.buffer_info()[0], 2, *a)
    assert size(4, 1, 1, 32) >= 0 and size(0, 5, 5, 32) == 0 and size(4, 0, 5, 32) == 0 and size(4, 5, 5, 1000) == 0
    assert size(4, 512, 512, 32) > 0
    assert lib.adasum_rms_norm_backward_scratch_bytes(offs.buffer_info()[0], 2, 64) == 0


def test_limits_are_the_headers():
    text = open(HEADER).read()
    assert int(re.search(r"#define ADASUM_BIAS_MAX_BUCKETS (\d+)", text).group(1)) == 256
    scales = re.search(r"typedef enum \{([^}]*)\} adasum_muon_scale_t", text).group(1)
    assert [int(v) for v in re.findall(r"= (\d)", scales)] == list(updates._SCALES.values())


def test_null_arguments_of_the_c_entries():
    """What needs no GPU to be refused."""
    lib = ags.load_library()
    co, offs = (ctypes.c_float * 3)(1, 1, 1), array("q", [0, 4])
    assert lib.adasum_orthogonalize(None, 1, 2, 2, 4, 2, 0, 1, ctypes.addressof(co), 0.0, None, None, 0, 0) == 1
    assert lib.adasum_orthogonalize(None, 1, 2, 2, 4, 2, 0, 1, None, 0.0, None, None, 0, 0) == 1
    assert lib.adasum_orthogonalize(None, 1, 2, 2, 4, 2, 7, 1, ctypes.addressof(co), 0.0, None, None, 0, 0) == 1
    assert lib.adasum_orthogonalize(None, 1, 2, 70000, 4, 2, 0, 1, ctypes.addressof(co), 0.0, None, None, 0, 0) == 2
    assert lib.adasum_orthogonalize(None, 0, 2, 2, 4, 2, 0, 1, ctypes.addressof(co), 0.0, None, None, 0, 0) == 0
    two = array("q", [2])
    step = lambda scale, rows=two: lib.adasum_muon_step(None, 0, offs.buffer_info()[0], rows.buffer_info()[0], two.buffer_info()[0], 1,
                                                        None, None, 0.1, 0.9, 1, 0.0, scale, 1, ctypes.addressof(co), 0.0, None, 0, 0)
    assert step(1) == 1 and step(3) == 1 and step(1, array("q", [3])) == 1 and step(1, array("q", [0])) == 0
    assert lib.adasum_relative_position_bias(None, 32, 4, 0, 1, 128, 0, 5, 5, None, 0, 0, 0, 0, 0, None, 0) == 1
    assert lib.adasum_relative_position_bias(None, 32, 4, 0, 1, 128, 0, 0, 5, None, 0, 0, 0, 0, 0, None, 0) == 0
    assert lib.adasum_relative_position_bias(None, 3, 4, 0, 1, 128, 0, 5, 5, None, 0, 0, 0, 0, 0, None, 0) == 1
    assert lib.adasum_relative_position_bias(None, 300, 4, 0, 1, 128, 0, 5, 5, None, 0, 0, 0, 0, 0, None, 0) == 2
    assert lib.adasum_rms_norm(None, 4, 8, 8, 0, None, 0, None, None, 0, 1e-6, None, None, None, None, 0) == 1
    assert lib.adasum_rms_norm(None, 0, 8, 8, 0, None, 0, None, None, 0, 1e-6, None, None, None, None, 0) == 0
    assert lib.adasum_rms_norm(None, 4, 20000, 20000, 0, None, 0, None, None, 0, 1e-6, None, None, None, None, 0) == 2
