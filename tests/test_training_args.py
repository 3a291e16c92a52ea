"""CPU checks of the training operators' binding: what it refuses before any GPU work, and
that the constants it lays checkpoints out with are the header's."""
import os
import re

import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
from adaptive_gradient_summation_gb300 import training

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "adasum.h")


def test_cpu_tensors_are_refused():
    x, tokens = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    kept = ags.Checkpoint(torch.zeros(4, 16, dtype=torch.int8), torch.zeros(4, 1), x.shape, x.dtype)
    for call in (lambda: ags.layer_norm(x), lambda: ags.layer_norm_checkpointed(x),
                 lambda: ags.layer_norm_backward(x, x, x[:, 0], x[:, 0]), lambda: ags.checkpoint_pack(x),
                 lambda: ags.checkpoint_unpack(kept), lambda: ags.gelu_checkpointed(x),
                 lambda: ags.gelu_checkpointed_backward(x, kept), lambda: ags.embedding(x, tokens),
                 lambda: ags.embedding_backward(x, tokens, 4)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_rows_of_views():
    x = torch.zeros(4, 6, 8)
    assert training._rows(x, "x") == (24, 8, 8)
    assert training._rows(x[:, :, :5], "x") == (24, 5, 8)
    assert training._rows(x[:, 2], "x") == (4, 8, 48)
    assert training._rows(x[:, ::2], "x") == (12, 8, 16)
    assert training._rows(x[0, 0], "x") == (1, 8, 8)
    assert training._rows(x[:, :1], "x") == (4, 8, 48)
    assert training._rows(x[:0], "x")[0] == 0
    for bad in (x.transpose(0, 1), x.transpose(1, 2), x[:, :5], x.expand(4, 6, 8)[:, :, ::2], torch.zeros(8).expand(3, 8)):
        with pytest.raises(ValueError):
            training._rows(bad, "x")


def test_worker_offsets():
    assert list(training._workers(None, 7)[0]) == [0, 7]
    assert list(training._workers(torch.tensor([0, 3, 7]), 7)[0]) == [0, 3, 7]
    for bad in ([0], [0, 6], []):
        with pytest.raises(ValueError):
            training._workers(bad, 7)


def test_checkpoint_layout_is_the_headers():
    text = open(HEADER).read()
    assert int(re.search(r"#define ADASUM_CHECKPOINT_BLOCK (\d+)", text).group(1)) == training.BLOCK
    kept = training._new_checkpoint(torch.zeros(3, 130, dtype=torch.bfloat16), 3, 130)
    assert kept.codes.shape == (3, 144) and kept.scales.shape == (3, 2) and kept.nbytes() == 3 * 144 + 3 * 8
