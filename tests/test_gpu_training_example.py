"""The example step: its gradients against autograd in 64 bits, and a falling loss."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "encoder_block_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("encoder_block_step", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def autograd(block, tokens, target, offsets, example):
    out = []
    for k in range(len(offsets) - 1):
        p = [q.double().requires_grad_() for q in block.parameters()]
        table, w1n, b1n, w1, w2, w2n, b2n = p
        t = tokens[offsets[k]:offsets[k + 1]]
        e = torch.nn.functional.embedding(t, table, padding_idx=example.PAD) * example.HIDDEN ** 0.5
        y1 = torch.nn.functional.layer_norm(e, (example.HIDDEN,), w1n, b1n)
        z = e + torch.nn.functional.gelu(y1 @ w1) @ w2
        y2 = torch.nn.functional.layer_norm(z, (example.HIDDEN,), w2n, b2n)
        (0.5 * (y2 - target[offsets[k]:offsets[k + 1]].double()).square().mean(1).mean()).backward()
        out.append(torch.cat([q.grad.reshape(-1) for q in p]))
    return out


def test_gradients(native, example):
    """Per worker and segment within 5% in 2-norm: the chain rounds at most eight tensors, each
    by an 8-bit step's rms (0.6% of a block of normal values) or less, added up linearly."""
    block = example.Block(seed=3)
    tokens, target, offsets = example.batch(workers=3, sequences=2, length=96, seed=4)
    offsets = [0, 100, 101, len(tokens)]  # unequal parts
    _, flat = example.gradients(block, tokens, target, offsets)
    for k, want in enumerate(autograd(block, tokens, target, offsets, example)):
        for name, a, b in zip(example.NAMES, block.offsets, block.offsets[1:]):
            w, g = want[a:b], flat[k, a:b].double()
            assert float((g - w).norm()) <= 0.05 * float(w.norm()), (k, name)
        row = flat[k, :example.HIDDEN]
        assert not row.any(), "the padding token learns nothing"


def test_loss_falls(native, example):
    block, data = example.Block(), example.batch()
    losses = [example.step(block, *data) for _ in range(20)]
    assert losses[-1] < 0.8 * losses[0] and all(l == l for l in losses)
