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
on that stream, so calls on several streams may overlap and may be captured.  Nothing is
recorded for autograd: outputs do not require gradients even where an input does, and the
caller makes the backward calls (for instance from a ``torch.autograd.Function``).
"""
from __future__ import annotations

from array import array
from operator import attrgetter
from typing import NamedTuple

import torch

from ._native import check, load_library

__all__ = ["Checkpoint", "checkpoint_pack", "checkpoint_unpack", "embedding", "embedding_backward",
           "gelu_checkpointed", "gelu_checkpointed_backward", "layer_norm", "layer_norm_backward",
           "layer_norm_checkpointed", "layer_norm_checkpointed_backward"]

_CODE = {torch.float32: 0, torch.bfloat16: 1}
_DEVICES = [torch.device("cuda", i) for i in range(128)]
_TOKEN_BYTES = {torch.int32: 4, torch.int64: 8}
# A small call is bound by the host, so the checks below use torch's cheapest accessors:
# on a Grace host torch.cuda.current_stream() takes 2.0 us, the raw handle 0.08 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_DTYPE = attrgetter("dtype")
_ptr_of, _device_of, _numel_of, _is_dense = (torch.Tensor.data_ptr, torch.Tensor.get_device, torch.Tensor.numel,
                                             torch.Tensor.is_contiguous)
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


def _elsewhere(index: int, stream) -> bool:
    """Whether a device or a stream has to be made current before the launch."""
    return stream is not None or index != _current_device()


def _there(index: int, stream, call, *args, **more):
    """`call` again, with device `index` and `stream` current."""
    if stream is None:
        with torch.cuda.device(index):
            return call(*args, **more)
    if stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
    with torch.cuda.device(index), torch.cuda.stream(stream):
        return call(*args, **more)


def _kind(t, what: str):
    """(type code, device index) of a float32 or bfloat16 CUDA tensor."""
    try:
        code, index = _CODE[t.dtype], t.get_device()
    except (AttributeError, KeyError):
        raise TypeError(f"{what} must be a float32 or bfloat16 tensor, got {getattr(t, 'dtype', type(t).__name__)}") from None
    if index < 0:
        raise ValueError(f"{what} must be a CUDA tensor")
    return code, index


def _rows(t: torch.Tensor, what: str):
    """(rows, cols, row stride) of an activation whose leading dimensions flatten."""
    shape = t.shape
    if len(shape) < 1 or shape[-1] == 0:
        raise ValueError(f"{what} must have a last dimension of at least one column")
    cols = shape[-1]
    if t.is_contiguous():
        return t.numel() // cols, cols, cols
    if t.numel() == 0:
        return 0, cols, cols
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what} must have its columns next to each other")
    n, ld = 1, None
    for size, stride in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
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


def _output(out, shape, dtype, index: int) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=_DEVICES[index])
    if (not isinstance(out, torch.Tensor) or out.dtype != dtype or out.get_device() != index
            or out.shape != torch.Size(shape) or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}")
    return out


def _parameters(weight, bias, cols: int, index: int):
    """(weight's pointer, bias's, the code of their type); either may be None."""
    w = b = code = None
    if weight is not None:
        code, at = _kind(weight, "weight")
        if at != index or weight.numel() != cols or not weight.is_contiguous():
            raise ValueError(f"weight must be a contiguous tensor of {cols} elements on cuda:{index}")
        w = weight.data_ptr()
    if bias is not None:
        other, at = _kind(bias, "bias")
        if at != index or bias.numel() != cols or not bias.is_contiguous():
            raise ValueError(f"bias must be a contiguous tensor of {cols} elements on cuda:{index}")
        if code is not None and other != code:
            raise ValueError("weight and bias must share their dtype")
        b, code = bias.data_ptr(), other
    return w, b, code or 0


def _statistic(t, rows: int, index: int, what: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.get_device() != index or t.numel() != rows \
            or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 tensor of {rows} elements on cuda:{index}")
    return t.data_ptr()


def _workers(worker_offsets, rows: int):
    """(K+1 offsets, K)."""
    if worker_offsets is None:
        return array("q", (0, rows)), 1
    offs = array("q", worker_offsets.tolist() if isinstance(worker_offsets, torch.Tensor) else worker_offsets)
    if len(offs) < 2 or offs[-1] != rows:
        raise ValueError(f"worker_offsets must be K+1 offsets ending at the row count {rows}")
    return offs, len(offs) - 1


def _gradients(grads, K: int, numel: int, index: int, dtype, shape, what: str):
    """(list of K tensors, their pointers, their type); None allocates them."""
    if grads is None:
        grads = torch.empty((K, *shape), dtype=dtype, device=_DEVICES[index]).unbind(0)
    elif isinstance(grads, torch.Tensor):
        grads = (grads,) if K == 1 and grads.numel() == numel else grads.unbind(0)
    grads = list(grads)
    if len(grads) != K:
        raise ValueError(f"{what} must be one tensor for each of the {K} workers, got {len(grads)}")
    _kind(grads[0], what)
    dtype = grads[0].dtype
    # (as passes over the list, which for many workers take half the time of a loop)
    try:
        good = (set(map(_DTYPE, grads)) == {dtype} and set(map(_device_of, grads)) == {index}
                and set(map(_numel_of, grads)) == {numel} and all(map(_is_dense, grads)))
    except (AttributeError, TypeError):
        raise TypeError(f"{what} must be tensors") from None
    if not good:
        raise ValueError(f"{what} must be contiguous tensors of {numel} elements and one dtype on cuda:{index}")
    return grads, array("Q", map(_ptr_of, grads)), dtype


def _address(a) -> int | None:
    """Of an array's elements; the library copies them before a call returns."""
    return None if a is None else a.buffer_info()[0]


def _tokens(tokens, index: int) -> int:
    width = _TOKEN_BYTES.get(getattr(tokens, "dtype", None))
    if width is None:
        raise TypeError("tokens must be an int32 or int64 tensor")
    if tokens.get_device() != index or not tokens.is_contiguous():
        raise ValueError(f"tokens must be a contiguous tensor on cuda:{index}")
    return width


def _scratch(nbytes: int, index: int):
    """Scratch memory of one call, from torch's allocator on the current stream."""
    return torch.empty(nbytes, dtype=torch.uint8, device=_DEVICES[index]) if nbytes > 0 else None


def _ptr(t):
    return None if t is None else t.data_ptr()


# ---------------------------------------------------------------------------- embeddings


def embedding(table: torch.Tensor, tokens: torch.Tensor, *, scale: float = 1.0, out: torch.Tensor | None = None,
              stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """``scale * table[tokens]`` (``adasum_embedding``), of shape ``(*tokens.shape, cols)`` in
    the table's dtype.  A token outside the table (the -1 that marks padding) gives zeros.
    tokens: int32 or int64."""
    code, index = _kind(table, "table")
    if table.dim() != 2 or table.shape[1] == 0 or not table.is_contiguous():
        raise ValueError("table must be a contiguous matrix")
    width = _tokens(tokens, index)
    if _elsewhere(index, stream):
        return _there(index, stream, embedding, table, tokens, scale=scale, out=out)
    rows, cols = table.shape
    out = _output(out, (*tokens.shape, cols), table.dtype, index)
    st = load_library().adasum_embedding(table.data_ptr(), rows, cols, code, tokens.data_ptr(), width, tokens.numel(),
                                         float(scale), out.data_ptr(), _raw_stream(index))
    if st:
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
    table and ``padding_idx`` get no gradient; ``padding_idx`` is the token itself, so a
    negative one is no row of the table and masks nothing (it does not count from the end).
    """
    code, index = _kind(grad_output, "grad_output")
    width = _tokens(tokens, index)
    rows, cols, ld = _rows(grad_output, "grad_output")
    if grad_output.shape[:-1] != tokens.shape:
        raise ValueError(f"grad_output must have shape {(*tokens.shape, cols)}")
    if num_rows < 0:
        raise ValueError("num_rows must not be negative")
    if grads is None and accumulate:
        raise ValueError("accumulate needs grads to add to")
    if _elsewhere(index, stream):
        return _there(index, stream, embedding_backward, grad_output, tokens, num_rows, scale=scale,
                      worker_offsets=worker_offsets, padding_idx=padding_idx, grads=grads, accumulate=accumulate)
    offs, K = _workers(worker_offsets, rows)
    grads, ptrs, gtype = _gradients(grads, K, num_rows * cols, index, grad_output.dtype, (num_rows, cols), "grads")
    lib = load_library()
    nbytes = lib.adasum_embedding_backward_scratch_bytes(_address(offs), K, num_rows, cols)
    scratch = _scratch(nbytes, index)
    st = lib.adasum_embedding_backward(
        grad_output.data_ptr(), cols, ld, code, tokens.data_ptr(), width, _address(offs), K, num_rows, float(scale),
        -1 if padding_idx is None else padding_idx, _address(ptrs), _CODE[gtype], bool(accumulate), _ptr(scratch), nbytes,
        _raw_stream(index))
    if st:
        check(st, "adasum_embedding_backward")
    return grads


# ---------------------------------------------------------------------------- layer norm


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
               eps: float = 1e-5, out: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """Layer norm over the last dimension (``adasum_layer_norm``): ``(y, mean, rstd)``, the
    last two in float32, for :func:`layer_norm_backward`."""
    code, index = _kind(x, "x")
    rows, cols, ld = _rows(x, "x")
    w, b, wcode = _parameters(weight, bias, cols, index)
    if _elsewhere(index, stream):
        return _there(index, stream, layer_norm, x, weight, bias, eps=eps, out=out)
    y = _output(out, x.shape, x.dtype, index)
    lead = x.shape[:-1]
    mean = torch.empty(lead, dtype=torch.float32, device=_DEVICES[index])
    rstd = torch.empty(lead, dtype=torch.float32, device=_DEVICES[index])
    st = load_library().adasum_layer_norm(x.data_ptr(), rows, cols, ld, code, w, b, wcode, float(eps), y.data_ptr(),
                                          mean.data_ptr(), rstd.data_ptr(), None, None, _raw_stream(index))
    if st:
        check(st, "adasum_layer_norm")
    return y, mean, rstd


def layer_norm_checkpointed(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                            *, eps: float = 1e-5, out: torch.Tensor | None = None,
                            stream: torch.cuda.Stream | None = None):
    """Layer norm that keeps ``h = (x - mean) rstd`` in 8 bits: ``(y, checkpoint, rstd)``, for
    :func:`layer_norm_checkpointed_backward`; neither x nor y has to be kept."""
    code, index = _kind(x, "x")
    rows, cols, ld = _rows(x, "x")
    w, b, wcode = _parameters(weight, bias, cols, index)
    if _elsewhere(index, stream):
        return _there(index, stream, layer_norm_checkpointed, x, weight, bias, eps=eps, out=out)
    y = _output(out, x.shape, x.dtype, index)
    kept = _new_checkpoint(x, rows, cols)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=_DEVICES[index])
    st = load_library().adasum_layer_norm(x.data_ptr(), rows, cols, ld, code, w, b, wcode, float(eps), y.data_ptr(), None,
                                          rstd.data_ptr(), kept.codes.data_ptr(), kept.scales.data_ptr(),
                                          _raw_stream(index))
    if st:
        check(st, "adasum_layer_norm")
    return y, kept, rstd


def _norm_gradients(grad_weights, grad_biases, weight, wanted, accumulate, offs, K, cols, index):
    """(weights' gradients, their pointers, biases', pointers, code, scratch bytes, scratch)."""
    if not wanted:
        if grad_weights is not None or grad_biases is not None:
            raise ValueError("grad_weights and grad_biases are not written with parameter_grads=False")
        return None, None, None, None, 0, 0, None
    if accumulate and (grad_weights is None or grad_biases is None):
        raise ValueError("accumulate needs grad_weights and grad_biases to add to")
    dtype = torch.float32 if weight is None else weight.dtype
    dw, dwp, dtype = _gradients(grad_weights, K, cols, index, dtype, (cols,), "grad_weights")
    db, dbp, other = _gradients(grad_biases, K, cols, index, dtype, (cols,), "grad_biases")
    if other is not dtype:
        raise ValueError("grad_weights and grad_biases must share their dtype")
    nbytes = load_library().adasum_layer_norm_backward_scratch_bytes(_address(offs), K, cols)
    return dw, dwp, db, dbp, _CODE[dtype], nbytes, _scratch(nbytes, index)


def layer_norm_backward(grad_output: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: torch.Tensor | None = None, *, worker_offsets=None, grad_weights=None,
                        grad_biases=None, accumulate: bool = False, parameter_grads: bool = True,
                        stream: torch.cuda.Stream | None = None):
    """``(grad_x, grad_weights, grad_biases)`` of layer norm (``adasum_layer_norm_backward``).

    grad_weights, grad_biases: K contiguous tensors of cols elements each (one dtype; None
    allocates them, in weight's dtype, else float32), overwritten, or with ``accumulate``
    added to; returned as lists.  ``parameter_grads=False`` leaves them out (None).
    """
    code, index = _kind(x, "x")
    if _kind(grad_output, "grad_output") != (code, index) or grad_output.shape != x.shape:
        raise ValueError(f"grad_output must have shape {tuple(x.shape)}, {x.dtype}, on cuda:{index}")
    rows, cols, ld_x = _rows(x, "x")
    ld_g = _rows(grad_output, "grad_output")[2]
    w, _, wcode = _parameters(weight, None, cols, index)
    mean_p, rstd_p = _statistic(mean, rows, index, "mean"), _statistic(rstd, rows, index, "rstd")
    if _elsewhere(index, stream):
        return _there(index, stream, layer_norm_backward, grad_output, x, mean, rstd, weight,
                      worker_offsets=worker_offsets, grad_weights=grad_weights, grad_biases=grad_biases,
                      accumulate=accumulate, parameter_grads=parameter_grads)
    offs, K = _workers(worker_offsets, rows)
    dw, dwp, db, dbp, gcode, nbytes, scratch = _norm_gradients(grad_weights, grad_biases, weight, parameter_grads,
                                                               accumulate, offs, K, cols, index)
    dx = _output(None, x.shape, x.dtype, index)
    st = load_library().adasum_layer_norm_backward(
        grad_output.data_ptr(), ld_g, x.data_ptr(), ld_x, mean_p, rstd_p, cols, code, w, wcode, _address(offs), K,
        dx.data_ptr(), _address(dwp), _address(dbp), gcode, bool(accumulate), _ptr(scratch), nbytes,
        _raw_stream(index))
    if st:
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
    code, index = _kind(grad_output, "grad_output")
    rows, cols, ld_g = _rows(grad_output, "grad_output")
    codes, scales = _check_checkpoint(checkpoint, index, grad_output)
    w, b, wcode = _parameters(weight, bias, cols, index)
    rstd_p = _statistic(rstd, rows, index, "rstd")
    if _elsewhere(index, stream):
        return _there(index, stream, layer_norm_checkpointed_backward, grad_output, checkpoint, rstd, weight, bias,
                      worker_offsets=worker_offsets, grad_weights=grad_weights, grad_biases=grad_biases,
                      accumulate=accumulate, parameter_grads=parameter_grads, with_output=with_output)
    offs, K = _workers(worker_offsets, rows)
    dw, dwp, db, dbp, gcode, nbytes, scratch = _norm_gradients(grad_weights, grad_biases, weight, parameter_grads,
                                                               accumulate, offs, K, cols, index)
    dx = _output(None, grad_output.shape, grad_output.dtype, index)
    y = _output(None, dx.shape, dx.dtype, index) if with_output else None
    st = load_library().adasum_layer_norm_backward_checkpointed(
        grad_output.data_ptr(), ld_g, codes, scales, rstd_p, cols, code, w, b, wcode, _address(offs), K, dx.data_ptr(),
        _ptr(y), _address(dwp), _address(dbp), gcode, bool(accumulate), _ptr(scratch), nbytes, _raw_stream(index))
    if st:
        check(st, "adasum_layer_norm_backward_checkpointed")
    return (dx, dw, db, y) if with_output else (dx, dw, db)


# --------------------------------------------------------------------- 8-bit checkpoints


def _new_checkpoint(x, rows: int, cols: int) -> Checkpoint:
    device = x.device
    codes = torch.empty((rows, (cols + 15) // 16 * 16), dtype=torch.int8, device=device)
    scales = torch.empty((rows, (cols + BLOCK - 1) // BLOCK), dtype=torch.float32, device=device)
    return Checkpoint(codes, scales, x.shape, x.dtype)


def _check_checkpoint(kept: Checkpoint, index: int, like: torch.Tensor | None = None):
    """(pointer of the codes, pointer of the scales)."""
    if not isinstance(kept, Checkpoint):
        raise TypeError("checkpoint must be a Checkpoint")
    codes, scales, shape, dtype = kept
    if like is not None and (shape != like.shape or dtype != like.dtype):
        raise ValueError(f"grad_output must be like the activation: {tuple(shape)}, {dtype}")
    cols = shape[-1]
    rows = 1
    for s in shape[:-1]:
        rows *= s
    if codes.dtype != torch.int8 or codes.get_device() != index or not codes.is_contiguous() \
            or codes.shape != (rows, (cols + 15) // 16 * 16):
        raise ValueError(f"checkpoint codes do not belong to an activation of shape {tuple(shape)} on cuda:{index}")
    if scales.dtype != torch.float32 or scales.get_device() != index or not scales.is_contiguous() \
            or scales.shape != (rows, (cols + BLOCK - 1) // BLOCK):
        raise ValueError(f"checkpoint scales do not belong to an activation of shape {tuple(shape)} on cuda:{index}")
    return codes.data_ptr(), scales.data_ptr()


def checkpoint_pack(x: torch.Tensor, *, stream: torch.cuda.Stream | None = None) -> Checkpoint:
    """An activation in 8 bits (``adasum_checkpoint_pack``): blocks of 128 columns, each with
    the scale max|x| / 127.  A block holding a NaN or an infinity comes back as NaN."""
    code, index = _kind(x, "x")
    rows, cols, ld = _rows(x, "x")
    if _elsewhere(index, stream):
        return _there(index, stream, checkpoint_pack, x)
    kept = _new_checkpoint(x, rows, cols)
    st = load_library().adasum_checkpoint_pack(x.data_ptr(), rows, cols, ld, code, kept.codes.data_ptr(),
                                               kept.scales.data_ptr(), _raw_stream(index))
    if st:
        check(st, "adasum_checkpoint_pack")
    return kept


def checkpoint_unpack(checkpoint: Checkpoint, *, dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                      stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The values a checkpoint stands for (``adasum_checkpoint_unpack``), in the activation's
    shape and its dtype (or ``dtype``)."""
    if not isinstance(checkpoint, Checkpoint):
        raise TypeError("checkpoint must be a Checkpoint")
    if not checkpoint.codes.is_cuda:
        raise ValueError("checkpoint must hold CUDA tensors")
    index = checkpoint.codes.get_device()
    codes, scales = _check_checkpoint(checkpoint, index)
    dtype = checkpoint.dtype if dtype is None else dtype
    if dtype not in _CODE:
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    if _elsewhere(index, stream):
        return _there(index, stream, checkpoint_unpack, checkpoint, dtype=dtype, out=out)
    out = _output(out, checkpoint.shape, dtype, index)
    st = load_library().adasum_checkpoint_unpack(codes, scales, checkpoint.codes.shape[0], checkpoint.shape[-1],
                                                 _CODE[dtype], out.data_ptr(), _raw_stream(index))
    if st:
        check(st, "adasum_checkpoint_unpack")
    return out


def gelu_checkpointed(x: torch.Tensor, *, tanh: bool = False, out: torch.Tensor | None = None,
                      stream: torch.cuda.Stream | None = None):
    """``(gelu(x), checkpoint of x)`` in one pass (``adasum_gelu_checkpointed``); ``tanh``
    selects the tanh form."""
    code, index = _kind(x, "x")
    rows, cols, ld = _rows(x, "x")
    if _elsewhere(index, stream):
        return _there(index, stream, gelu_checkpointed, x, tanh=tanh, out=out)
    y = _output(out, x.shape, x.dtype, index)
    kept = _new_checkpoint(x, rows, cols)
    st = load_library().adasum_gelu_checkpointed(x.data_ptr(), rows, cols, ld, code, bool(tanh), y.data_ptr(),
                                                 kept.codes.data_ptr(), kept.scales.data_ptr(), _raw_stream(index))
    if st:
        check(st, "adasum_gelu_checkpointed")
    return y, kept


def gelu_checkpointed_backward(grad_output: torch.Tensor, checkpoint: Checkpoint, *, tanh: bool = False,
                               with_output: bool = False, stream: torch.cuda.Stream | None = None):
    """``grad_output * gelu'(x)`` for the x that the checkpoint stands for
    (``adasum_gelu_checkpointed_backward``); with ``with_output`` the pair of that and gelu(x),
    so that the forward pass's output need not be kept."""
    code, index = _kind(grad_output, "grad_output")
    rows, cols, ld = _rows(grad_output, "grad_output")
    codes, scales = _check_checkpoint(checkpoint, index, grad_output)
    if _elsewhere(index, stream):
        return _there(index, stream, gelu_checkpointed_backward, grad_output, checkpoint, tanh=tanh,
                      with_output=with_output)
    dx = _output(None, grad_output.shape, grad_output.dtype, index)
    y = _output(None, dx.shape, dx.dtype, index) if with_output else None
    st = load_library().adasum_gelu_checkpointed_backward(grad_output.data_ptr(), ld, codes, scales, rows, cols, code,
                                                          bool(tanh), dx.data_ptr(), _ptr(y), _raw_stream(index))
    if st:
        check(st, "adasum_gelu_checkpointed_backward")
    return (dx, y) if with_output else dx
