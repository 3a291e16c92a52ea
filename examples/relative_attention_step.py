"""One training step of a small attention block with relative positions, on K workers'
microbatches, its matrices stepped by orthogonalised updates.

Token embedding -> root-mean-square norm -> attention with a learned relative position bias ->
root-mean-square norm of the sum with the residual, kept in 8 bits -> feed-forward with GELU ->
root-mean-square norm -> squared error to a fixed target, and the backward pass, all workers' rows
in one call each.  Every operator leaves its parameters' gradients per worker in slices of K flat
gradients; the combine makes one of them.  Then the matrices take an orthogonalised step, and the
vectors and tables the combine's own momentum step.

    python examples/relative_attention_step.py [steps]
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import adaptive_gradient_summation_gb300 as ags  # noqa: E402

VOCAB, HIDDEN, HEADS, FFN, BUCKETS, DISTANCE = 500, 128, 4, 512, 16, 32
NAMES = ("table", "bias", "norm1", "wqkv", "wo", "norm2", "w1", "w2", "norm3")
SHAPES = ((VOCAB, HIDDEN), (BUCKETS, HEADS), (HIDDEN,), (HIDDEN, 3 * HIDDEN), (HIDDEN, HIDDEN), (HIDDEN,), (HIDDEN, FFN),
          (FFN, HIDDEN), (HIDDEN,))
MATRICES = ("wqkv", "wo", "w1", "w2")  # stepped by orthogonalised updates


class Block:
    """The parameters: one flat fp32 vector of 9 segments, and bf16 copies to compute with."""

    def __init__(self, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        parts = []
        for name, shape in zip(NAMES, SHAPES):
            if name.startswith("norm"):
                parts.append(torch.ones(shape, device=device))
            else:
                parts.append(torch.randn(shape, generator=gen, device=device) / math.sqrt(shape[0] if name in MATRICES else shape[-1]))
        self.offsets = [0]
        for p in parts:
            self.offsets.append(self.offsets[-1] + p.numel())
        self.master = torch.cat([p.reshape(-1) for p in parts])
        self.momentum = torch.zeros_like(self.master)

    def parameters(self, dtype=torch.bfloat16):
        flat = self.master.to(dtype)
        return [flat[a:b].view(s) for a, b, s in zip(self.offsets, self.offsets[1:], SHAPES)]


def _heads(x):
    """(sequences, tokens, hidden) as (sequences, heads, tokens, hidden / heads)."""
    return x.view(*x.shape[:2], HEADS, -1).transpose(1, 2)


def gradients(block: Block, tokens: torch.Tensor, target: torch.Tensor, workers: int, dtype=torch.bfloat16):
    """(loss, K x N gradients) of (sequences, tokens) and their target; worker k has the k-th
    equal part of the sequences, and its gradient is that of its rows' mean squared error."""
    table, bias, n1, wqkv, wo, n2, w1, w2, n3 = block.parameters(dtype)
    seqs, length = tokens.shape
    by_seq = [k * (seqs // workers) for k in range(workers + 1)]
    by_row = [s * length for s in by_seq]
    flat = torch.empty(workers, block.offsets[-1], dtype=dtype, device=tokens.device)
    part = {n: list(flat[:, a:b].unbind(0)) for n, a, b in zip(NAMES, block.offsets, block.offsets[1:])}
    root = 1.0 / math.sqrt(HIDDEN // HEADS)

    e = ags.embedding(table, tokens)
    y1, rstd1 = ags.rms_norm(e, n1)
    q, k, v = (_heads(t) for t in (y1 @ wqkv).chunk(3, -1))
    scores = ags.relative_position_bias(bias, length, length, max_distance=DISTANCE, scores=(q @ k.transpose(2, 3)) * root)
    p = torch.softmax(scores.float(), -1).to(dtype)
    o = (p @ v).transpose(1, 2).reshape(seqs, length, HIDDEN)
    y2, h, kept2, rstd2 = ags.rms_norm_checkpointed(o @ wo, n2, residual=e)
    a, kept_u = ags.gelu_checkpointed(y2 @ w1)
    y3, z, rstd3 = ags.rms_norm(a @ w2, n3, residual=h)
    del y2, a, h  # only their 8-bit forms stay

    error = y3.float() - target
    loss = 0.5 * float(error.square().mean())
    dy3 = (error * (workers / error.numel())).to(dtype)

    # (what goes into a norm's input past it is added by its gradient)
    dz, _ = ags.rms_norm_backward(dy3, z, rstd3, n3, worker_offsets=by_row, grad_weights=part["norm3"])
    du, a = ags.gelu_checkpointed_backward(dz @ w2.t(), kept_u, with_output=True)
    dh, _, y2 = ags.rms_norm_checkpointed_backward(du @ w1.t(), kept2, rstd2, n2, grad_residual=dz, worker_offsets=by_row,
                                                   grad_weights=part["norm2"], with_output=True)
    do = _heads(dh @ wo.t())
    dp = (do @ v.transpose(2, 3)).float()
    ds = (p.float() * (dp - (dp * p.float()).sum(-1, keepdim=True))).to(dtype)
    ags.relative_position_bias_backward(ds, BUCKETS, max_distance=DISTANCE, worker_offsets=by_seq, grads=part["bias"])
    dqkv = torch.cat([t.transpose(1, 2).reshape(seqs, length, HIDDEN) for t in ((ds @ k) * root, (ds.transpose(2, 3) @ q) * root,
                                                                               p.transpose(2, 3) @ do)], -1)
    de, _ = ags.rms_norm_backward(dqkv @ wqkv.t(), e, rstd1, n1, grad_residual=dh, worker_offsets=by_row, grad_weights=part["norm1"])
    for w in range(workers):
        mine = slice(by_seq[w], by_seq[w + 1])
        for name, left, right in (("w2", a, dz), ("w1", y2, du), ("wo", o, dh), ("wqkv", y1, dqkv)):
            left, right = left[mine].flatten(0, 1), right[mine].flatten(0, 1)
            torch.matmul(left.t(), right, out=part[name][w].view(left.shape[1], right.shape[1]))
    ags.embedding_backward(de, tokens, VOCAB, worker_offsets=by_row, grads=part["table"])
    return loss, flat


def step(block: Block, tokens, target, workers: int, lr=0.02, mu=0.9) -> float:
    loss, flat = gradients(block, tokens, target, workers)
    combined = ags.reduce(flat, block.offsets)
    shapes = [s if n in MATRICES else None for n, s in zip(NAMES, SHAPES)]
    ags.muon_step(combined, block.offsets, shapes, block.master, block.momentum, lr=lr, mu=mu)
    for name, a, b in zip(NAMES, block.offsets, block.offsets[1:]):
        if name not in MATRICES:
            ags.reduce_momentum_sgd([combined[a:b]], None, block.master[a:b], block.momentum[a:b], lr=lr, mu=mu)
    return loss


def batch(workers=4, sequences=4, length=48, device="cuda", seed=1):
    """Tokens, and as the target of each a vector of the token before it."""
    gen = torch.Generator(device=device).manual_seed(seed)
    tokens = torch.randint(0, VOCAB, (workers * sequences, length), generator=gen, device=device)
    target = torch.randn(VOCAB, HIDDEN, generator=gen, device=device)[tokens.roll(1, 1)]
    return tokens, target, workers


def main(steps: int = 20):
    block, data = Block(), batch()
    for i in range(steps):
        print(f"step {i}: loss {step(block, *data):.4f}")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 20)
