"""One training step of a small encoder block on K workers' microbatches, end to end.

Token embedding -> layer norm -> feed-forward with GELU -> residual -> layer norm, a squared
error to a fixed target, and the backward pass, all workers' rows in one call each.  Every
operator leaves its parameters' gradients per worker, in slices of the K flat gradients that
the Adasum combine takes; the fused combine and Momentum-SGD step then updates the fp32 master
weights.  Between the passes the first norm's and the GELU's activations are kept in 8 bits
only: the backward pass gives their outputs again for the weight gradients of the products.

    python examples/encoder_block_step.py [steps]
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import adaptive_gradient_summation_gb300 as ags  # noqa: E402

VOCAB, HIDDEN, FFN = 1000, 256, 1024
NAMES = ("table", "norm1.weight", "norm1.bias", "w1", "w2", "norm2.weight", "norm2.bias")
SHAPES = ((VOCAB, HIDDEN), (HIDDEN,), (HIDDEN,), (HIDDEN, FFN), (FFN, HIDDEN), (HIDDEN,), (HIDDEN,))
PAD = 0  # a token that is looked up but not learnt


class Block:
    """The parameters: one flat fp32 vector of 7 segments, and bf16 copies to compute with."""

    def __init__(self, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        parts = []
        for name, shape in zip(NAMES, SHAPES):
            if name.endswith("weight"):
                parts.append(torch.ones(shape, device=device))
            elif name.endswith("bias"):
                parts.append(torch.zeros(shape, device=device))
            else:
                parts.append(torch.randn(shape, generator=gen, device=device) / math.sqrt(shape[-1] if name == "table" else shape[0]))
        self.offsets = [0]
        for p in parts:
            self.offsets.append(self.offsets[-1] + p.numel())
        self.master = torch.cat([p.reshape(-1) for p in parts])
        self.momentum = torch.zeros_like(self.master)

    def parameters(self):
        flat = self.master.to(torch.bfloat16)
        return [flat[a:b].view(s) for a, b, s in zip(self.offsets, self.offsets[1:], SHAPES)]


def gradients(block: Block, tokens: torch.Tensor, target: torch.Tensor, worker_offsets):
    """(loss, K x N bf16 gradients): worker k's is that of its rows' mean squared error."""
    table, w1n, b1n, w1, w2, w2n, b2n = block.parameters()
    workers = len(worker_offsets) - 1
    flat = torch.empty(workers, block.offsets[-1], dtype=torch.bfloat16, device=tokens.device)
    part = {n: list(flat[:, a:b].unbind(0)) for n, a, b in zip(NAMES, block.offsets, block.offsets[1:])}
    scale = math.sqrt(HIDDEN)

    e = ags.embedding(table, tokens, scale=scale)
    y1, kept1, rstd1 = ags.layer_norm_checkpointed(e, w1n, b1n)
    a, kept_u = ags.gelu_checkpointed(y1 @ w1)
    z = e + a @ w2
    del y1, a  # only their 8-bit forms stay
    y2, mean2, rstd2 = ags.layer_norm(z, w2n, b2n)

    error = y2.float() - target
    rows = torch.tensor([worker_offsets[k + 1] - worker_offsets[k] for k in range(workers)], device=tokens.device)
    share = torch.repeat_interleave(1.0 / rows.clamp(min=1), rows, output_size=tokens.numel())
    loss = 0.5 * float((error.square().mean(1) * share).sum()) / workers
    dy2 = (error * share[:, None] / HIDDEN).to(torch.bfloat16)

    dz, _, _ = ags.layer_norm_backward(dy2, z, mean2, rstd2, w2n, worker_offsets=worker_offsets,
                                       grad_weights=part["norm2.weight"], grad_biases=part["norm2.bias"])
    du, a = ags.gelu_checkpointed_backward(dz @ w2.t(), kept_u, with_output=True)
    de, _, _, y1 = ags.layer_norm_checkpointed_backward(
        du @ w1.t(), kept1, rstd1, w1n, b1n, worker_offsets=worker_offsets, grad_weights=part["norm1.weight"],
        grad_biases=part["norm1.bias"], with_output=True)
    for k in range(workers):
        mine = slice(worker_offsets[k], worker_offsets[k + 1])
        torch.matmul(a[mine].t(), dz[mine], out=part["w2"][k].view(FFN, HIDDEN))
        torch.matmul(y1[mine].t(), du[mine], out=part["w1"][k].view(HIDDEN, FFN))
    ags.embedding_backward(de + dz, tokens, VOCAB, scale=scale, worker_offsets=worker_offsets, padding_idx=PAD,
                           grads=part["table"])
    return loss, flat


def step(block: Block, tokens, target, worker_offsets, lr=0.2, mu=0.9) -> float:
    loss, flat = gradients(block, tokens, target, worker_offsets)
    ags.reduce_momentum_sgd(flat, block.offsets, block.master, block.momentum, lr=lr, mu=mu)
    return loss


def batch(workers=4, sequences=4, length=128, device="cuda", seed=1):
    """Tokens with frequencies that fall off as 1 / rank, some of them padding, and a target."""
    gen = torch.Generator(device=device).manual_seed(seed)
    n = workers * sequences * length
    u = torch.rand(n, generator=gen, device=device)
    tokens = (torch.exp(u * math.log(VOCAB)) - 1).long().clamp_(0, VOCAB - 1)
    target = torch.randn(VOCAB, HIDDEN, generator=gen, device=device)[tokens]
    return tokens, target, [k * sequences * length for k in range(workers + 1)]


def main(steps: int = 20):
    block, data = Block(), batch()
    for i in range(steps):
        print(f"step {i}: loss {step(block, *data):.4f}")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 20)
