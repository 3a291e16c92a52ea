"""Operators of the training step around the Adasum combine: token embeddings, layer norm,
and activations kept in 8 bits between the forward and the backward pass.

Parameter gradients come per worker.  The rows of a call (all leading dimensions of a
tensor, flattened) are the microbatches of K workers one after the other, worker k's being
rows [worker_offsets[k], worker_offsets[k+1]); gradient k is summed over those rows only
and written (or, with ``accumulate``, added) where the caller wants it, for instance into
slices of the K flat gradients that :func:`reduce` takes.  Without ``worker_offsets`` all
rows are one worker's.

Like the rest of the package this module only marshals torch tensors into the C ABI of
include/adasum.h: inputs are CUDA tensors, float32 or bfloat16, the types of activations,
parameters and parameter gradients being independent of each other; their columns have to
be next to each other, while rows may be strided.  Outputs are dense.  Calls are
asynchronous on the current (or given) stream; scratch memory comes from torch's allocator
on that stream, so calls on several streams may overlap and may be captured.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from ._native import check, load_library

__all__ = ["Checkpoint", "checkpoint_pack", "checkpoint_unpack", "embedding", "embedding_backward",
           "gelu_checkpointed", "gelu_checkpointed_backward", "layer_norm", "layer_norm_backward",
           "layer_norm_checkpointed", "layer_norm_checkpointed_backward"]

_CODE = {torch.float32: 0, torch.bfloat16: 1}
#: Columns per scale of a checkpoint.
BLOCK = 128


class Checkpoint(NamedTuple):
    """An activation in 8 bits (``adasum_checkpoint_pack``): codes of rows x cols values, rows
    padded to a multiple of 16, and one scale per block of 128 columns of a row."""
    codes: torch.Tensor   # int8, rows x pitch
    scales: torch.Tensor  # float32, rows x blocks
    shape: torch.Size     # of the activation
    dtype: torch.dtype    # of the activation

    def nbytes(self) -> int:
        return self.codes.numel() + 4 * self.scales.numel()


class _On:
    """Makes a device and a stream current where they are not yet."""

    def __init__(self, device, stream):
        self.stack = []
        if device.index != torch.cuda.current_device():
            self.stack.append(torch.cuda.device(device))
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
            self.stack.append(torch.cuda.stream(stream))

    def __enter__(self):
        for s in self.stack:
            s.__enter__()

    def __exit__(self, *exc):
        while self.stack:
            self.stack.pop().__exit__(*exc)


def _float_tensor(t, what: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a tensor, got {type(t).__name__}")
    if t.dtype not in _CODE:
        raise TypeError(f"{what} must be float32 or bfloat16, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{what} must be a CUDA tensor")
    return t


def _rows(t: torch.Tensor, what: str):
    """(rows, cols, row stride) of an activation whose leading dimensions flatten."""
    if t.dim() < 1 or t.shape[-1] == 0:
        raise ValueError(f"{what} must have a last dimension of at least one column")
    cols = t.shape[-1]
    if t.is_contiguous():
        return t.numel() // cols, cols, cols
    if t.numel() == 0:
        return 0, cols, cols
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what} must have its columns next to each other")
    n, ld = 1, None
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if ld is None:
            ld = stride
        elif stride != n * ld:
            raise ValueError(f"the leading dimensions of {what} must flatten to evenly spaced rows")
        n *= size
    ld = cols if ld is None else ld
    if ld < cols:
        raise ValueError(f"the rows of {what} must not overlap")
    return n, cols, ld


def _same(t: torch.Tensor, like: torch.Tensor, what: str) -> None:
    if t.dtype != like.dtype or t.device != like.device or t.shape != like.shape:
        raise ValueError(f"{what} must have shape {tuple(like.shape)}, {like.dtype}, on {like.device}")


def _output(out, like: torch.Tensor, shape, what: str = "out") -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    if (not isinstance(out, torch.Tensor) or out.dtype != like.dtype or out.device != like.device
            or out.shape != torch.Size(shape) or not out.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous {like.dtype} tensor of shape {tuple(shape)} on {like.device}")
    return out


def _parameter(p, cols: int, device, what: str):
    """(pointer, dtype) of a weight or bias; None is allowed."""
    if p is None:
        return None, None
    _float_tensor(p, what)
    if p.device != device or p.numel() != cols or not p.is_contiguous():
        raise ValueError(f"{what} must be a contiguous tensor of {cols} elements on {device}")
    return p.data_ptr(), p.dtype


def _parameters(weight, bias, cols: int, device):
    w, wt = _parameter(weight, cols, device, "weight")
    b, bt = _parameter(bias, cols, device, "bias")
    if wt is not None and bt is not None and wt != bt:
        raise ValueError("weight and bias must share their dtype")
    return w, b, _CODE[wt or bt or torch.float32]


def _statistic(t, rows: int, device, what: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.device != device or t.numel() != rows \
            or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 tensor of {rows} elements on {device}")
    return t.data_ptr()


def _workers(worker_offsets, rows: int):
    """(ctypes array of K+1 offsets, K)."""
    if worker_offsets is None:
        return (ctypes.c_int64 * 2)(0, rows), 1
    if isinstance(worker_offsets, torch.Tensor):
        worker_offsets = worker_offsets.tolist()
    offs = [int(o) for o in worker_offsets]
    if len(offs) < 2 or offs[-1] != rows:
        raise ValueError(f"worker_offsets must be K+1 offsets ending at the row count {rows}")
    return (ctypes.c_int64 * len(offs))(*offs), len(offs) - 1


def _gradients(grads, K: int, numel: int, device, dtype, shape, what: str):
    """(list of K tensors, ctypes array of their pointers, their dtype); None allocates."""
    if grads is None:
        grads = list(torch.empty((K, *shape), dtype=dtype, device=device).unbind(0))
    elif isinstance(grads, torch.Tensor):
        grads = [grads] if K == 1 and grads.numel() == numel else list(grads.unbind(0))
    else:
        grads = list(grads)
    if len(grads) != K:
        raise ValueError(f"{what} must be one tensor for each of the {K} workers, got {len(grads)}")
    dtype = grads[0].dtype
    for g in grads:
        _float_tensor(g, what)
        if g.dtype != dtype or g.device != device or g.numel() != numel or not g.is_contiguous():
            raise ValueError(f"{what} must be contiguous tensors of {numel} elements and one dtype on {device}")
    return grads, (ctypes.c_void_p * K)(*[g.data_ptr() for g in grads]), dtype


def _current_stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _tokens(tokens, device, what: str = "tokens") -> int:
    if not isinstance(tokens, torch.Tensor) or tokens.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"{what} must be an int32 or int64 tensor")
    if tokens.device != device or not tokens.is_contiguous():
        raise ValueError(f"{what} must be a contiguous tensor on {device}")
    return tokens.element_size()


def _scratch(nbytes: int, device):
    """Scratch memory of one call, from torch's allocator on the current stream."""
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes > 0 else None


def _ptr(t):
    return None if t is None else t.data_ptr()


# ---------------------------------------------------------------------------- embeddings


def embedding(table: torch.Tensor, tokens: torch.Tensor, *, scale: float = 1.0, out: torch.Tensor | None = None,
              stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """``scale * table[tokens]`` (``adasum_embedding``), of shape ``(*tokens.shape, cols)`` in
    the table's dtype.  A token outside the table (the -1 that marks padding) gives zeros.
    tokens: int32 or int64."""
    _float_tensor(table, "table")
    if table.dim() != 2 or table.shape[1] == 0 or not table.is_contiguous():
        raise ValueError("table must be a contiguous matrix")
    device = table.device
    width = _tokens(tokens, device)
    with _On(device, stream):
        out = _output(out, table, (*tokens.shape, table.shape[1]))
        st = load_library().adasum_embedding(
            table.data_ptr(), table.shape[0], table.shape[1], _CODE[table.dtype], tokens.data_ptr(), width,
            tokens.numel(), float(scale), out.data_ptr(), _current_stream(device))
    check(st, "adasum_embedding")
    return out


def embedding_backward(grad_output: torch.Tensor, tokens: torch.Tensor, num_rows: int, *, scale: float = 1.0,
                       worker_offsets=None, padding_idx: int | None = None, grads=None, accumulate: bool = False,
                       stream: torch.cuda.Stream | None = None) -> list:
    """The gradient of an embedding table of ``num_rows`` rows, per worker
    (``adasum_embedding_backward``): a list of K tensors, tensor k holding
    ``scale * sum of grad_output[i]`` over worker k's tokens equal to v in row v.

    worker_offsets: K+1 offsets into the flattened tokens (None: one worker).  grads: K
    contiguous tensors of num_rows * cols elements (of any one dtype; None allocates them in
    grad_output's), overwritten whole, or with ``accumulate`` added to.  Tokens outside the
    table and ``padding_idx`` get no gradient.
    """
    _float_tensor(grad_output, "grad_output")
    device = grad_output.device
    width = _tokens(tokens, device)
    rows, cols, ld = _rows(grad_output, "grad_output")
    if grad_output.shape[:-1] != tokens.shape:
        raise ValueError(f"grad_output must have shape {(*tokens.shape, cols)}")
    if num_rows < 0:
        raise ValueError("num_rows must not be negative")
    if grads is None and accumulate:
        raise ValueError("accumulate needs grads to add to")
    offs, K = _workers(worker_offsets, rows)
    lib = load_library()
    with _On(device, stream):
        grads, ptrs, gtype = _gradients(grads, K, num_rows * cols, device, grad_output.dtype, (num_rows, cols), "grads")
        nbytes = lib.adasum_embedding_backward_scratch_bytes(rows, cols, K)
        scratch = _scratch(nbytes, device)
        st = lib.adasum_embedding_backward(
            grad_output.data_ptr(), cols, ld, _CODE[grad_output.dtype], tokens.data_ptr(), width, offs, K, num_rows,
            float(scale), -1 if padding_idx is None else int(padding_idx), ptrs, _CODE[gtype], bool(accumulate),
            _ptr(scratch), nbytes, _current_stream(device))
    check(st, "adasum_embedding_backward")
    return grads


# ---------------------------------------------------------------------------- layer norm


def _norm_forward(x, weight, bias, eps, out, stream, kept: bool):
    _float_tensor(x, "x")
    device = x.device
    rows, cols, ld = _rows(x, "x")
    w, b, wcode = _parameters(weight, bias, cols, device)
    with _On(device, stream):
        y = _output(out, x, x.shape)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=device)
        if kept:
            mean, saved = None, _new_checkpoint(x, rows, cols)
            codes, scales = saved.codes.data_ptr(), saved.scales.data_ptr()
        else:
            mean, codes, scales = torch.empty_like(rstd), None, None
            saved = mean
        st = load_library().adasum_layer_norm(
            x.data_ptr(), rows, cols, ld, _CODE[x.dtype], w, b, wcode, float(eps), y.data_ptr(), _ptr(mean),
            rstd.data_ptr(), codes, scales, _current_stream(device))
    check(st, "adasum_layer_norm")
    return y, saved, rstd


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
               eps: float = 1e-5, out: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """Layer norm over the last dimension (``adasum_layer_norm``): ``(y, mean, rstd)``, the
    last two in float32, for :func:`layer_norm_backward`."""
    return _norm_forward(x, weight, bias, eps, out, stream, False)


def layer_norm_checkpointed(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                            *, eps: float = 1e-5, out: torch.Tensor | None = None,
                            stream: torch.cuda.Stream | None = None):
    """Layer norm that keeps ``h = (x - mean) rstd`` in 8 bits: ``(y, checkpoint, rstd)``, for
    :func:`layer_norm_checkpointed_backward`; neither x nor y has to be kept."""
    return _norm_forward(x, weight, bias, eps, out, stream, True)


def _norm_gradients(lib, grad_weights, grad_biases, wanted, K, cols, device, dtype, rows, accumulate):
    if accumulate and (grad_weights is None or grad_biases is None) and wanted:
        raise ValueError("accumulate needs grad_weights and grad_biases to add to")
    if not wanted:
        if grad_weights is not None or grad_biases is not None:
            raise ValueError("grad_weights and grad_biases are not written with parameter_grads=False")
        return None, None, None, None, 0, 0, None
    dw, dwp, dt = _gradients(grad_weights, K, cols, device, dtype, (cols,), "grad_weights")
    db, dbp, bt = _gradients(grad_biases, K, cols, device, dt, (cols,), "grad_biases")
    if dt != bt:
        raise ValueError("grad_weights and grad_biases must share their dtype")
    nbytes = lib.adasum_layer_norm_backward_scratch_bytes(rows, cols, K)
    return dw, dwp, db, dbp, _CODE[dt], nbytes, _scratch(nbytes, device)


def layer_norm_backward(grad_output: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: torch.Tensor | None = None, *, worker_offsets=None, grad_weights=None,
                        grad_biases=None, accumulate: bool = False, parameter_grads: bool = True,
                        stream: torch.cuda.Stream | None = None):
    """``(grad_x, grad_weights, grad_biases)`` of layer norm (``adasum_layer_norm_backward``).

    grad_weights, grad_biases: K contiguous tensors of cols elements each (one dtype; None
    allocates them, in weight's dtype, else float32), overwritten, or with ``accumulate``
    added to; returned as lists.  ``parameter_grads=False`` leaves them out (None).
    """
    _float_tensor(grad_output, "grad_output")
    _float_tensor(x, "x")
    device = x.device
    _same(grad_output, x, "grad_output")
    rows, cols, ld_x = _rows(x, "x")
    ld_g = _rows(grad_output, "grad_output")[2]
    w, _, wcode = _parameters(weight, None, cols, device)
    mean_p, rstd_p = _statistic(mean, rows, device, "mean"), _statistic(rstd, rows, device, "rstd")
    offs, K = _workers(worker_offsets, rows)
    lib = load_library()
    with _On(device, stream):
        dx = torch.empty(x.shape, dtype=x.dtype, device=device)
        dw, dwp, db, dbp, gcode, nbytes, scratch = _norm_gradients(
            lib, grad_weights, grad_biases, parameter_grads, K, cols, device,
            torch.float32 if weight is None else weight.dtype, rows, accumulate)
        st = lib.adasum_layer_norm_backward(
            grad_output.data_ptr(), ld_g, x.data_ptr(), ld_x, mean_p, rstd_p, cols, _CODE[x.dtype], w, wcode, offs, K,
            dx.data_ptr(), dwp, dbp, gcode, bool(accumulate), _ptr(scratch), nbytes, _current_stream(device))
    check(st, "adasum_layer_norm_backward")
    return dx, dw, db


def layer_norm_checkpointed_backward(grad_output: torch.Tensor, checkpoint: Checkpoint, rstd: torch.Tensor,
                                     weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
                                     worker_offsets=None, grad_weights=None, grad_biases=None,
                                     accumulate: bool = False, parameter_grads: bool = True,
                                     with_output: bool = False, stream: torch.cuda.Stream | None = None):
    """``(grad_x, grad_weights, grad_biases)`` of layer norm from the 8-bit checkpoint of h
    (``adasum_layer_norm_backward_checkpointed``); with ``with_output`` also the output again,
    as a fourth.  bias is used for the output only.  The rest as in :func:`layer_norm_backward`."""
    _float_tensor(grad_output, "grad_output")
    device = grad_output.device
    rows, cols, ld_g = _rows(grad_output, "grad_output")
    codes, scales = _check_checkpoint(checkpoint, device, grad_output)
    w, b, wcode = _parameters(weight, bias, cols, device)
    rstd_p = _statistic(rstd, rows, device, "rstd")
    offs, K = _workers(worker_offsets, rows)
    lib = load_library()
    with _On(device, stream):
        dx = torch.empty(grad_output.shape, dtype=grad_output.dtype, device=device)
        y = torch.empty_like(dx) if with_output else None
        dw, dwp, db, dbp, gcode, nbytes, scratch = _norm_gradients(
            lib, grad_weights, grad_biases, parameter_grads, K, cols, device,
            torch.float32 if weight is None else weight.dtype, rows, accumulate)
        st = lib.adasum_layer_norm_backward_checkpointed(
            grad_output.data_ptr(), ld_g, codes, scales, rstd_p, cols, _CODE[grad_output.dtype], w, b, wcode, offs, K,
            dx.data_ptr(), _ptr(y), dwp, dbp, gcode, bool(accumulate), _ptr(scratch), nbytes, _current_stream(device))
    check(st, "adasum_layer_norm_backward_checkpointed")
    return (dx, dw, db, y) if with_output else (dx, dw, db)


# --------------------------------------------------------------------- 8-bit checkpoints


def _new_checkpoint(x, rows: int, cols: int) -> Checkpoint:
    codes = torch.empty((rows, (cols + 15) // 16 * 16), dtype=torch.int8, device=x.device)
    scales = torch.empty((rows, (cols + BLOCK - 1) // BLOCK), dtype=torch.float32, device=x.device)
    return Checkpoint(codes, scales, x.shape, x.dtype)


def _check_checkpoint(kept: Checkpoint, device, like: torch.Tensor | None = None):
    """(pointer of the codes, pointer of the scales)."""
    if not isinstance(kept, Checkpoint):
        raise TypeError("checkpoint must be a Checkpoint")
    if like is not None and (kept.shape != like.shape or kept.dtype != like.dtype):
        raise ValueError(f"grad_output must be like the activation: {tuple(kept.shape)}, {kept.dtype}")
    cols = kept.shape[-1]
    rows = 1
    for s in kept.shape[:-1]:
        rows *= s
    codes, scales = kept.codes, kept.scales
    if codes.dtype != torch.int8 or codes.device != device or not codes.is_contiguous() \
            or codes.shape != (rows, (cols + 15) // 16 * 16):
        raise ValueError(f"checkpoint codes do not belong to an activation of shape {tuple(kept.shape)} on {device}")
    if scales.dtype != torch.float32 or scales.device != device or not scales.is_contiguous() \
            or scales.shape != (rows, (cols + BLOCK - 1) // BLOCK):
        raise ValueError(f"checkpoint scales do not belong to an activation of shape {tuple(kept.shape)} on {device}")
    return codes.data_ptr(), scales.data_ptr()


def checkpoint_pack(x: torch.Tensor, *, stream: torch.cuda.Stream | None = None) -> Checkpoint:
    """An activation in 8 bits (``adasum_checkpoint_pack``): blocks of 128 columns, each with
    the scale max|x| / 127.  A block holding a NaN or an infinity comes back as NaN."""
    _float_tensor(x, "x")
    device = x.device
    rows, cols, ld = _rows(x, "x")
    with _On(device, stream):
        kept = _new_checkpoint(x, rows, cols)
        st = load_library().adasum_checkpoint_pack(
            x.data_ptr(), rows, cols, ld, _CODE[x.dtype], kept.codes.data_ptr(), kept.scales.data_ptr(),
            _current_stream(device))
    check(st, "adasum_checkpoint_pack")
    return kept


def checkpoint_unpack(checkpoint: Checkpoint, *, dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                      stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The values a checkpoint stands for (``adasum_checkpoint_unpack``), in the activation's
    shape and its dtype (or ``dtype``)."""
    if not isinstance(checkpoint, Checkpoint):
        raise TypeError("checkpoint must be a Checkpoint")
    device = checkpoint.codes.device
    if device.type != "cuda":
        raise ValueError("checkpoint must be on a CUDA device")
    codes, scales = _check_checkpoint(checkpoint, device)
    dtype = checkpoint.dtype if dtype is None else dtype
    if dtype not in _CODE:
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    rows, cols = checkpoint.codes.shape[0], checkpoint.shape[-1]
    with _On(device, stream):
        if out is None:
            out = torch.empty(checkpoint.shape, dtype=dtype, device=device)
        elif out.dtype != dtype or out.device != device or out.shape != checkpoint.shape or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous {dtype} tensor of shape {tuple(checkpoint.shape)} on {device}")
        st = load_library().adasum_checkpoint_unpack(codes, scales, rows, cols, _CODE[dtype], out.data_ptr(),
                                                     _current_stream(device))
    check(st, "adasum_checkpoint_unpack")
    return out


def gelu_checkpointed(x: torch.Tensor, *, tanh: bool = False, out: torch.Tensor | None = None,
                      stream: torch.cuda.Stream | None = None):
    """``(gelu(x), checkpoint of x)`` in one pass (``adasum_gelu_checkpointed``); ``tanh``
    selects the tanh form."""
    _float_tensor(x, "x")
    device = x.device
    rows, cols, ld = _rows(x, "x")
    with _On(device, stream):
        y = _output(out, x, x.shape)
        kept = _new_checkpoint(x, rows, cols)
        st = load_library().adasum_gelu_checkpointed(
            x.data_ptr(), rows, cols, ld, _CODE[x.dtype], bool(tanh), y.data_ptr(), kept.codes.data_ptr(),
            kept.scales.data_ptr(), _current_stream(device))
    check(st, "adasum_gelu_checkpointed")
    return y, kept


def gelu_checkpointed_backward(grad_output: torch.Tensor, checkpoint: Checkpoint, *, tanh: bool = False,
                               with_output: bool = False, stream: torch.cuda.Stream | None = None):
    """``grad_output * gelu'(x)`` for the x that the checkpoint stands for
    (``adasum_gelu_checkpointed_backward``); with ``with_output`` the pair of that and gelu(x),
    so that the forward pass's output need not be kept."""
    _float_tensor(grad_output, "grad_output")
    device = grad_output.device
    rows, cols, ld = _rows(grad_output, "grad_output")
    codes, scales = _check_checkpoint(checkpoint, device, grad_output)
    with _On(device, stream):
        dx = torch.empty(grad_output.shape, dtype=grad_output.dtype, device=device)
        y = torch.empty_like(dx) if with_output else None
        st = load_library().adasum_gelu_checkpointed_backward(
            grad_output.data_ptr(), ld, codes, scales, rows, cols, _CODE[grad_output.dtype], bool(tanh),
            dx.data_ptr(), _ptr(y), _current_stream(device))
    check(st, "adasum_gelu_checkpointed_backward")
    return (dx, y) if with_output else dx
