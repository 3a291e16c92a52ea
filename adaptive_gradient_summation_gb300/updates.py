"""Orthogonalised updates: the Newton-Schulz iteration, and the step of momentum, iteration and
fp32 master weights that follows the Adasum combine, as the Muon optimiser takes it.

With X = G / (|G| + eps) (the Frobenius norm; a matrix with more rows than columns
transposed) every step takes X to ``a X + (b A + c A A) X`` with ``A = X X'``, which moves all
singular values towards 1.  Marshalling only, with the conventions of training.py: CUDA
tensors, the current (or given) stream, scratch memory from torch's allocator.
"""
from __future__ import annotations

from array import array
from numbers import Real

import torch

from ._native import check, load_library
from .training import _address, _elsewhere, _kind, _output, _ptr, _raw_stream, _scratch, _there

__all__ = ["orthogonalize", "muon_step", "NEWTON_SCHULZ"]

#: The usual quintic's coefficients (a, b, c), for five steps.
NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)
_SCALES = {None: 0, "spectral": 1, "rms": 2}


def _coefficients(coefficients, steps: int) -> array:
    """3 * steps floats of one triple, or of one triple a step."""
    if steps < 1:
        raise ValueError("steps must be at least 1")
    flat = list(coefficients)
    if len(flat) == 3 and all(isinstance(c, Real) for c in flat):
        return array("f", flat * steps)
    if len(flat) != steps or any(len(c) != 3 for c in flat):
        raise ValueError(f"coefficients must be three numbers, or three for each of the {steps} steps")
    return array("f", [x for c in flat for x in c])


def _matrices(x: torch.Tensor):
    """(batch, rows, cols, distance of matrices, distance of rows) of matrices whose leading
    dimensions flatten."""
    if x.dim() < 2:
        raise ValueError("x must have at least two dimensions")
    rows, cols = x.shape[-2:]
    if x.is_contiguous():
        return x.numel() // (rows * cols) if rows and cols else 0, rows, cols, rows * cols, cols
    if x.numel() == 0:
        return 0, rows, cols, rows * cols, cols
    if cols > 1 and x.stride(-1) != 1:
        raise ValueError("x must have its columns next to each other")
    ld = x.stride(-2) if rows > 1 else cols
    n, apart = 1, None
    for size, stride in zip(reversed(x.shape[:-2]), reversed(x.stride()[:-2])):
        if size == 1:
            continue
        if apart is None:
            apart = stride
        elif stride != n * apart:
            raise ValueError("the leading dimensions of x must flatten to evenly spaced matrices")
        n *= size
    apart = rows * ld if apart is None else apart
    if ld < cols or (n > 1 and apart < (rows - 1) * ld + cols):
        raise ValueError("the rows and matrices of x must not overlap")
    return n, rows, cols, apart, ld


def orthogonalize(x: torch.Tensor, *, steps: int = 5, coefficients=NEWTON_SCHULZ, eps: float = 1e-7,
                  out: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Every matrix of ``x`` (its last two dimensions) after the Newton-Schulz iteration
    (``adasum_orthogonalize``), in x's shape and dtype.

    coefficients: (a, b, c), or one such triple for every step; they have to keep the singular
    values below 2.8.  Computed to fp32's accuracy for float32, to bf16's for bfloat16.
    """
    code, index = _kind(x, "x")
    batch, rows, cols, apart, ld = _matrices(x)
    coefficients = _coefficients(coefficients, steps)
    if _elsewhere(index, stream):
        return _there(index, stream, orthogonalize, x, steps=steps, coefficients=[coefficients[i:i + 3] for i in range(0, 3 * steps, 3)],
                      eps=eps, out=out)
    out = _output(out, x.shape, x.dtype, index)
    lib = load_library()
    nbytes = lib.adasum_orthogonalize_scratch_bytes(batch, rows, cols, code)
    scratch = _scratch(nbytes, index)
    st = lib.adasum_orthogonalize(x.data_ptr(), batch, rows, cols, apart, ld, code, steps, _address(coefficients), float(eps),
                                  out.data_ptr(), _ptr(scratch), nbytes, _raw_stream(index))
    if st:
        check(st, "adasum_orthogonalize")
    return out


def muon_step(grad: torch.Tensor, seg_offsets, shapes, master_w: torch.Tensor, momentum: torch.Tensor, *, lr: float,
              mu: float = 0.95, nesterov: bool = True, weight_decay: float = 0.0, scale: str | None = "spectral",
              steps: int = 5, coefficients=NEWTON_SCHULZ, eps: float = 1e-7, stream: torch.cuda.Stream | None = None):
    """One step of a flat vector's matrices (``adasum_muon_step``): for every segment that is a
    matrix ``v <- mu v + g``, X the orthogonalised ``g + mu v`` (or ``v`` without ``nesterov``),
    ``w <- (1 - lr weight_decay) w - lr s X``.  Returns ``(master_w, momentum)``, updated in place.

    grad: the flat gradient, for instance what :func:`reduce` returns.  seg_offsets: L+1
    offsets.  shapes: for each segment ``(rows, cols)``, or None for one that is not a matrix,
    whose weights and momentum are left alone.  master_w, momentum: float32, like grad.
    scale: the factor s of a matrix: "spectral" sqrt(max(1, rows / cols)), "rms"
    0.2 sqrt(max(rows, cols)), None 1.  The iteration is computed to fp32's accuracy.
    """
    code, index = _kind(grad, "grad")
    n = grad.numel()
    if grad.dim() != 1 or not grad.is_contiguous():
        raise ValueError("grad must be a contiguous vector")
    for name, t in (("master_w", master_w), ("momentum", momentum)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.get_device() != index or t.numel() != n \
                or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 tensor of {n} elements on cuda:{index}")
    if scale not in _SCALES:
        raise ValueError(f"scale must be one of {', '.join(map(repr, _SCALES))}")
    triples = _coefficients(coefficients, steps)
    offs = array("q", seg_offsets.tolist() if hasattr(seg_offsets, "tolist") else seg_offsets)
    shapes = list(shapes)
    if len(offs) != len(shapes) + 1 or offs[-1] != n:
        raise ValueError(f"seg_offsets must be one offset more than shapes, ending at the gradient's length {n}")
    rows, cols = (array("q", [0 if s is None else s[i] for s in shapes]) for i in (0, 1))
    if _elsewhere(index, stream):
        return _there(index, stream, muon_step, grad, offs, shapes, master_w, momentum, lr=lr, mu=mu, nesterov=nesterov,
                      weight_decay=weight_decay, scale=scale, steps=steps, coefficients=coefficients, eps=eps)
    lib = load_library()
    nbytes = lib.adasum_muon_step_scratch_bytes(_address(rows), _address(cols), len(shapes))
    scratch = _scratch(nbytes, index)
    st = lib.adasum_muon_step(grad.data_ptr(), code, _address(offs), _address(rows), _address(cols), len(shapes),
                              master_w.data_ptr(), momentum.data_ptr(), float(lr), float(mu), bool(nesterov), float(weight_decay),
                              _SCALES[scale], steps, _address(triples), float(eps), _ptr(scratch), nbytes, _raw_stream(index))
    if st:
        check(st, "adasum_muon_step")
    return master_w, momentum
