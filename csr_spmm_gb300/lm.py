"""The operators at the two ends of a language model, on torch CUDA tensors.

:func:`embedding`, :func:`layer_norm` and :func:`token_logprob` and their
gradients: argument checks and marshalling over the C entry points of
``include/csr_spmm.h``, which define the operations.  Matrices are 2-D with
unit column stride (any row stride: the leading dimension) in float32, float16
or bfloat16; ids, targets and indices are int32.  Each call is enqueued on
``stream`` (default: torch's current stream) and returns without waiting; new
outputs are allocated for that stream, and the inputs' memory is held until
the stream has used it.
"""
from __future__ import annotations

import torch

from . import _lib

_TYPES = {torch.float32: _lib.SPMM_F32, torch.float16: _lib.SPMM_F16,
          torch.bfloat16: _lib.SPMM_BF16}


def _type(t, what: str) -> int:
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be float32, float16 or bfloat16")
    return code


def _matrix(t, what: str):
    """(rows, columns, leading dimension) of a matrix."""
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D with unit column stride")
    rows, cols = t.shape
    if cols > 1 and rows > 0 and t.stride(1) != 1:
        raise ValueError(f"{what} must be 2-D with unit column stride")
    return rows, cols, (t.stride(0) if rows > 1 else max(1, cols))


def _vector(t, n: int, dtype, what: str) -> None:
    """A 1-D array of n contiguous entries of one of the types in `dtype`."""
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{what} must be 1-D with {n} entries, got {tuple(t.shape)}")
    if t.dtype not in dtype:
        raise TypeError(f"{what} must be {' or '.join(str(d)[6:] for d in dtype)}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{what} must be contiguous")


_INT, _FLOAT = (torch.int32,), (torch.float32,)


def _address(t, device: int) -> int:
    """Device address of a tensor on the handle's GPU (0 for None)."""
    if t is None:
        return 0
    if not t.is_cuda:
        raise ValueError(f"expected a CUDA tensor, got one on {t.device}")
    if t.device.index != device:
        raise ValueError(f"tensor on {t.device}, but the handle is on cuda:{device}")
    return t.data_ptr()


class _Call:
    """The stream of one call: where its outputs are allocated and what it holds."""

    def __init__(self, handle, stream, tensors):
        self.device = handle.device
        self.given = stream
        self.addresses = [_address(t, self.device) for t in tensors]
        if stream is None:
            self.stream = torch.cuda.current_stream().cuda_stream
        else:
            self.stream = stream.cuda_stream
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)

    def empty(self, shape, dtype):
        if self.given is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.given):
            return torch.empty(shape, dtype=dtype, device=self.device)


def _output(call, out, rows: int, cols: int, dtype):
    """A [rows, cols] output: `out` after its checks, or a new tensor."""
    if out is None:
        out = call.empty((rows, cols), dtype)
        return out, out.data_ptr(), max(1, cols)
    return out, _address(out, call.device), _matrix(out, "out")[2]


def _check_out(out, rows: int, cols: int, dtype) -> None:
    if out is None:
        return
    if tuple(out.shape) != (rows, cols):
        raise ValueError(f"out must be {(rows, cols)}, got {tuple(out.shape)}")
    _matrix(out, "out")
    if out.dtype != dtype:
        raise TypeError(f"out must be {str(dtype)[6:]}")


def embedding(handle, ids, table, scale: float = 1.0, out=None, stream=None):
    """out[t, :] = scale * table[ids[t], :]; an id outside [0, vocabulary) gives zeros.

    ``ids`` is an int32 vector, ``table`` a [vocabulary, dim] matrix.  Returns
    ``out`` ([tokens, dim], the table's dtype; new when not given).
    """
    code = _type(table, "table")
    vocab, dim, ld = _matrix(table, "table")
    n = ids.numel()
    _vector(ids, n, _INT, "ids")
    _check_out(out, n, dim, table.dtype)
    call = _Call(handle, stream, (ids, table, out))
    a_ids, a_table, _ = call.addresses
    out, a_out, ld_out = _output(call, out, n, dim, table.dtype)
    _lib.spmm_embedding(handle.ptr, code, scale, a_ids, n, a_table, ld, vocab, dim, a_out, ld_out,
                        call.stream)
    return out


def embedding_grad(handle, ids, dout, dtable, scale: float = 1.0, beta: float = 0.0,
                   stream=None) -> None:
    """dtable <- beta * dtable + the gradient of :func:`embedding` with respect to its table.

    ``dout`` is [tokens, dim]; ``dtable`` is [vocabulary, dim] in dout's dtype
    or float32.  beta = 0 writes every row; beta = 1 adds to the rows of the
    ids that occur and leaves the others alone.
    """
    code, grad_code = _type(dout, "dout"), _type(dtable, "dtable")
    if grad_code != code and grad_code != _lib.SPMM_F32:
        raise TypeError("dtable must have dout's dtype or be float32")
    n, dim, ld = _matrix(dout, "dout")
    vocab, cols, ld_table = _matrix(dtable, "dtable")
    if cols != dim:
        raise ValueError(f"shape mismatch: dout {tuple(dout.shape)}, dtable {tuple(dtable.shape)}")
    _vector(ids, n, _INT, "ids")
    call = _Call(handle, stream, (ids, dout, dtable))
    a_ids, a_dout, a_table = call.addresses
    _lib.spmm_embedding_grad(handle.ptr, code, grad_code, scale, a_ids, n, a_dout, ld, beta,
                             a_table, ld_table, vocab, dim, call.stream)


def _params(x, dim: int, weight, bias) -> int:
    """The type code shared by weight and bias: x's or float32."""
    given = weight if weight is not None else bias
    if given is None:
        return _TYPES[x.dtype]
    if given.dtype != x.dtype and given.dtype != torch.float32:
        raise TypeError("weight and bias must have x's dtype or be float32")
    for t, what in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _vector(t, dim, (given.dtype,), what)
    return _TYPES[given.dtype]


def layer_norm(handle, x, weight=None, bias=None, eps: float = 1e-5, out=None, stream=None):
    """Layer norm of each row of ``x`` [rows, dim]; returns (y, mean, rstd).

    ``weight`` and ``bias`` (dim entries, either may be None) have x's dtype
    or are float32.  ``mean`` and ``rstd`` are float32 vectors for
    :func:`layer_norm_grad`.  ``out`` receives y; it may be ``x`` itself.
    """
    code = _type(x, "x")
    rows, dim, ld = _matrix(x, "x")
    param_code = _params(x, dim, weight, bias)
    _check_out(out, rows, dim, x.dtype)
    call = _Call(handle, stream, (x, weight, bias, out))
    a_x, a_w, a_b, _ = call.addresses
    y, a_y, ld_y = _output(call, out, rows, dim, x.dtype)
    stats = call.empty((2, rows), torch.float32)
    mean, rstd = stats[0], stats[1]
    a_stats = stats.data_ptr()
    _lib.spmm_layer_norm(handle.ptr, code, param_code, a_x, ld, rows, dim, a_w, a_b, eps, a_y,
                         ld_y, a_stats, a_stats + 4 * rows, call.stream)
    return y, mean, rstd


def layer_norm_grad(handle, dy, x, mean, rstd, weight=None, bias: bool = True, out=None,
                    stream=None):
    """Gradients of :func:`layer_norm`; returns (dx, dweight, dbias).

    ``mean`` and ``rstd`` are what the forward pass returned.  dweight is None
    without a weight, dbias with ``bias=False``; both have the weight's dtype
    (dbias x's dtype without a weight).  ``out`` receives dx; it may be ``dy``.
    """
    code = _type(x, "x")
    rows, dim, ld = _matrix(x, "x")
    if tuple(dy.shape) != (rows, dim):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, dy {tuple(dy.shape)}")
    if dy.dtype != x.dtype:
        raise TypeError("x and dy must share one dtype")
    ld_dy = _matrix(dy, "dy")[2]
    _vector(mean, rows, _FLOAT, "mean")
    _vector(rstd, rows, _FLOAT, "rstd")
    param_code = _params(x, dim, weight, None)
    _check_out(out, rows, dim, x.dtype)
    call = _Call(handle, stream, (dy, x, mean, rstd, weight, out))
    a_dy, a_x, a_mean, a_rstd, a_w, _ = call.addresses
    dx, a_dx, ld_dx = _output(call, out, rows, dim, x.dtype)
    pt = x.dtype if weight is None else weight.dtype
    dweight = call.empty(dim, pt) if weight is not None else None
    dbias = call.empty(dim, pt) if bias else None
    _lib.spmm_layer_norm_grad(handle.ptr, code, param_code, a_dy, ld_dy, a_x, ld, a_mean, a_rstd,
                              a_w, rows, dim, a_dx, ld_dx,
                              0 if dweight is None else dweight.data_ptr(),
                              0 if dbias is None else dbias.data_ptr(), call.stream)
    return dx, dweight, dbias


def token_logprob(handle, logits, targets=None, alpha: float = 1.0, top: int = 0, stream=None):
    """Log probabilities from ``logits`` [rows, vocabulary] at inverse temperature ``alpha``.

    Returns (logprob, entropy, lse), and with ``top`` > 0 also (top_logprob,
    top_index) of shape [rows, top], largest first.  ``targets`` (int32, one
    per row; outside the vocabulary: a row without one) may be None, and
    logprob is then None.  All but top_index (int32) are float32.
    """
    code = _type(logits, "logits")
    rows, vocab, ld = _matrix(logits, "logits")
    if targets is not None:
        _vector(targets, rows, _INT, "targets")
    if not 0 <= top <= _lib.SPMM_TOP_MAX:
        raise ValueError(f"top must be between 0 and {_lib.SPMM_TOP_MAX}")
    call = _Call(handle, stream, (logits, targets))
    a_x, a_t = call.addresses
    # one allocation for the vectors, the first a row without a target leaves out
    out = call.empty((3, rows), torch.float32)
    logprob, entropy, lse = out[0], out[1], out[2]
    a_out = out.data_ptr()
    top_logprob = top_index = None
    if top:
        top_logprob = call.empty((rows, top), torch.float32)
        top_index = call.empty((rows, top), torch.int32)
    _lib.spmm_token_logprob(handle.ptr, code, alpha, a_x, ld, rows, vocab, a_t, top,
                            a_out if targets is not None else 0, a_out + 4 * rows,
                            a_out + 8 * rows, top_logprob.data_ptr() if top else 0,
                            top_index.data_ptr() if top else 0, call.stream)
    if targets is None:
        logprob = None
    return (logprob, entropy, lse, top_logprob, top_index) if top else (logprob, entropy, lse)


def token_logprob_grad(handle, logits, targets, lse, entropy=None, dlogprob=None, dentropy=None,
                       alpha: float = 1.0, out=None, stream=None):
    """Gradient of :func:`token_logprob` with respect to the logits.

    ``dlogprob`` and ``dentropy`` (float32, one per row, either may be None)
    are the gradients of its first two results; ``lse`` and ``entropy`` are its
    results.  Returns dlogits ([rows, vocabulary], the logits' dtype) in
    ``out``, which may be ``logits`` itself, or in a new tensor.
    """
    code = _type(logits, "logits")
    rows, vocab, ld = _matrix(logits, "logits")
    if dlogprob is not None and targets is None:
        raise ValueError("dlogprob needs the targets")
    if dentropy is not None and entropy is None:
        raise ValueError("dentropy needs the entropy")
    if dlogprob is None:
        targets = None
    if dentropy is None:
        entropy = None
    if targets is not None:
        _vector(targets, rows, _INT, "targets")
    for t, what in ((lse, "lse"), (entropy, "entropy"), (dlogprob, "dlogprob"),
                    (dentropy, "dentropy")):
        if t is not None:
            _vector(t, rows, _FLOAT, what)
    _check_out(out, rows, vocab, logits.dtype)
    call = _Call(handle, stream, (logits, targets, lse, entropy, dlogprob, dentropy, out))
    a_x, a_t, a_lse, a_ent, a_dl, a_de, _ = call.addresses
    out, a_out, ld_out = _output(call, out, rows, vocab, logits.dtype)
    _lib.spmm_token_logprob_grad(handle.ptr, code, alpha, a_x, ld, rows, vocab, a_t, a_lse, a_ent,
                                 a_dl, a_de, a_out, ld_out, call.stream)
    return out
