"""The operators at the two ends of a language model, on torch CUDA tensors.

:func:`embedding`, :func:`layer_norm` and :func:`token_logprob` and their
gradients: argument checks and marshalling over the C entry points of
``include/csr_spmm.h``, which define the operations.  Matrices are 2-D with
unit column stride (any row stride: the leading dimension) in float32, float16
or bfloat16; ids, targets and indices are int32.  Each call is enqueued on
``stream`` (default: torch's current stream) and returns without waiting; new
outputs are allocated for that stream, and the inputs' memory is held until
the stream has used it.

One stream at a time per handle: :func:`embedding_grad` and :func:`layer_norm_grad` use the
handle's scratch, which their calls on two streams would share without an order.  Use a handle
for each stream, or order the streams.  The other functions use no scratch.

Nothing is recorded for autograd: results are detached also where an argument requires a
gradient, and the gradients are functions of their own.  New outputs come straight from
torch's caching allocator, so modes that intercept torch.empty do not see them.
"""
from __future__ import annotations

import torch

from . import _lib

_TYPES = {torch.float32: _lib.SPMM_F32, torch.float16: _lib.SPMM_F16,
          torch.bfloat16: _lib.SPMM_BF16}
_F32, _I32 = torch.float32, torch.int32
_INDEX = 3                               # beside the library's type codes: int32

# Small calls are bound by this file (a kernel of 2 us behind 6 us of host code), so
# each check reads a tensor's attributes once and nothing is built on the way.


def _type(t, what: str) -> int:
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be float32, float16 or bfloat16")
    return code


def _matrix(t, what: str):
    """(rows, columns, leading dimension) of a matrix."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2:
        raise ValueError(f"{what} must be 2-D with unit column stride")
    rows, cols = shape
    if stride[1] != 1 and cols > 1 and rows > 0:
        raise ValueError(f"{what} must be 2-D with unit column stride")
    return rows, cols, (stride[0] if rows > 1 else cols or 1)


def _vector(t, n: int, dtype, what: str) -> None:
    """A 1-D array of n contiguous entries of one type."""
    shape = t.shape
    if len(shape) != 1 or shape[0] != n:
        raise ValueError(f"{what} must be 1-D with {n} entries, got {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {str(dtype)[6:]}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{what} must be contiguous")


def _address(t, device: int) -> int:
    """Device address of a tensor on the handle's GPU (0 for None)."""
    if t is None:
        return 0
    if t.get_device() != device:
        if not t.is_cuda:
            raise ValueError(f"expected a CUDA tensor, got one on {t.device}")
        raise ValueError(f"tensor on {t.device}, but the handle is on cuda:{device}")
    return t.data_ptr()


def _current(device: int) -> int:
    """Torch's current stream on the handle's GPU."""
    return torch._C._cuda_getCurrentRawStream(device)


_make = None


def _new(stream, device: int, *what):
    """Tensors for outputs, allocated for the stream that writes them: `what` is a type
    code, rows and columns for each, columns < 0 for a vector.

    All of a call's at once and compiled (csrc/torch_outputs.cpp): three take 2.5 us, three
    torch.empty 4.4 and 3 more of what runs after them."""
    global _make
    if _make is None:
        _make = _lib.load_module("_torch_outputs").new
    if stream is None:
        return _make(device, *what)
    with torch.cuda.stream(stream):
        return _make(device, *what)


def _enter(device: int, stream, tensors) -> int:
    """The call's stream; on a given one the tensors' memory is held until it is used."""
    if stream is None:
        return _current(device)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


def _check_out(out, rows: int, cols: int, dtype) -> int:
    """Leading dimension of a given [rows, cols] output."""
    shape = out.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] != cols:
        raise ValueError(f"out must be {(rows, cols)}, got {tuple(shape)}")
    if out.dtype != dtype:
        raise TypeError(f"out must be {str(dtype)[6:]}")
    return _matrix(out, "out")[2]


def embedding(handle, ids, table, scale: float = 1.0, out=None, stream=None):
    """out[t, :] = scale * table[ids[t], :]; an id outside [0, vocabulary) gives zeros.

    ``ids`` is an int32 vector, ``table`` a [vocabulary, dim] matrix.  Returns
    ``out`` ([tokens, dim], the table's dtype; new when not given).
    """
    code = _type(table, "table")
    vocab, dim, ld = _matrix(table, "table")
    n = ids.numel()
    _vector(ids, n, _I32, "ids")
    ld_out = dim or 1
    if out is not None:
        ld_out = _check_out(out, n, dim, table.dtype)
    device = handle.device
    a_ids, a_table = _address(ids, device), _address(table, device)
    st = _enter(device, stream, (ids, table, out))
    if out is None:
        out, = _new(stream, device, code, n, dim)
    _lib.spmm_embedding(handle.ptr, code, scale, a_ids, n, a_table, ld, vocab, dim,
                        _address(out, device), ld_out, st)
    return out


def embedding_grad(handle, ids, dout, dtable, scale: float = 1.0, beta: float = 0.0,
                   stream=None) -> None:
    """dtable <- beta * dtable + the gradient of :func:`embedding` with respect to its table.

    ``dout`` is [tokens, dim]; ``dtable`` is [vocabulary, dim] in dout's dtype
    or float32.  beta = 0 writes every row; beta = 1 adds to the rows of the
    ids that occur and leaves the others alone.  Uses the handle's scratch: one stream at a
    time.
    """
    code, grad_code = _type(dout, "dout"), _type(dtable, "dtable")
    if grad_code != code and grad_code != _lib.SPMM_F32:
        raise TypeError("dtable must have dout's dtype or be float32")
    n, dim, ld = _matrix(dout, "dout")
    vocab, cols, ld_table = _matrix(dtable, "dtable")
    if cols != dim:
        raise ValueError(f"shape mismatch: dout {tuple(dout.shape)}, dtable {tuple(dtable.shape)}")
    _vector(ids, n, _I32, "ids")
    device = handle.device
    a_ids, a_dout, a_table = (_address(ids, device), _address(dout, device),
                              _address(dtable, device))
    _lib.spmm_embedding_grad(handle.ptr, code, grad_code, scale, a_ids, n, a_dout, ld, beta,
                             a_table, ld_table, vocab, dim,
                             _enter(device, stream, (ids, dout, dtable)))


def _params(x, code: int, dim: int, weight, bias) -> int:
    """The type code shared by weight and bias: x's or float32."""
    given = weight if weight is not None else bias
    if given is None:
        return code
    dtype = given.dtype
    if dtype != x.dtype and dtype != _F32:
        raise TypeError("weight and bias must have x's dtype or be float32")
    if weight is not None:
        _vector(weight, dim, dtype, "weight")
    if bias is not None:
        _vector(bias, dim, dtype, "bias")
    return _TYPES[dtype]


def layer_norm(handle, x, weight=None, bias=None, eps: float = 1e-5, out=None, stream=None):
    """Layer norm of each row of ``x`` [rows, dim]; returns (y, mean, rstd).

    ``weight`` and ``bias`` (dim entries, either may be None) have x's dtype
    or are float32.  ``mean`` and ``rstd`` are float32 vectors for
    :func:`layer_norm_grad`.  ``out`` receives y; it may be ``x`` itself.
    """
    code = _type(x, "x")
    rows, dim, ld = _matrix(x, "x")
    param_code = _params(x, code, dim, weight, bias)
    ld_y = dim or 1
    if out is not None:
        ld_y = _check_out(out, rows, dim, x.dtype)
    device = handle.device
    a_x, a_w, a_b = _address(x, device), _address(weight, device), _address(bias, device)
    st = _enter(device, stream, (x, weight, bias, out))
    if out is None:
        out, mean, rstd = _new(stream, device, code, rows, dim, 0, rows, -1, 0, rows, -1)
    else:
        mean, rstd = _new(stream, device, 0, rows, -1, 0, rows, -1)
    _lib.spmm_layer_norm(handle.ptr, code, param_code, a_x, ld, rows, dim, a_w, a_b, eps,
                         _address(out, device), ld_y, mean.data_ptr(), rstd.data_ptr(), st)
    return out, mean, rstd


def layer_norm_grad(handle, dy, x, mean, rstd, weight=None, bias: bool = True, out=None,
                    stream=None):
    """Gradients of :func:`layer_norm`; returns (dx, dweight, dbias).

    ``mean`` and ``rstd`` are what the forward pass returned.  dweight is None
    without a weight, dbias with ``bias=False``; both have the weight's dtype
    (dbias x's dtype without a weight).  ``out`` receives dx; it may be ``dy``.  Uses the
    handle's scratch: one stream at a time.
    """
    code = _type(x, "x")
    rows, dim, ld = _matrix(x, "x")
    dy_rows, dy_dim, ld_dy = _matrix(dy, "dy")
    if dy_rows != rows or dy_dim != dim:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, dy {tuple(dy.shape)}")
    if dy.dtype != x.dtype:
        raise TypeError("x and dy must share one dtype")
    _vector(mean, rows, _F32, "mean")
    _vector(rstd, rows, _F32, "rstd")
    param_code = _params(x, code, dim, weight, None)
    ld_dx = dim or 1
    if out is not None:
        ld_dx = _check_out(out, rows, dim, x.dtype)
    device = handle.device
    a_dy, a_x, a_w = _address(dy, device), _address(x, device), _address(weight, device)
    a_mean, a_rstd = _address(mean, device), _address(rstd, device)
    st = _enter(device, stream, (dy, x, mean, rstd, weight, out))
    what = ((code, rows, dim) if out is None else ()) + \
        ((param_code, dim, -1) if weight is not None else ()) + \
        ((param_code, dim, -1) if bias else ())
    made = iter(_new(stream, device, *what))
    if out is None:
        out = next(made)
    dweight = dbias = None
    a_dw = a_db = 0
    if weight is not None:
        dweight = next(made)
        a_dw = dweight.data_ptr()
    if bias:
        dbias = next(made)
        a_db = dbias.data_ptr()
    _lib.spmm_layer_norm_grad(handle.ptr, code, param_code, a_dy, ld_dy, a_x, ld, a_mean, a_rstd,
                              a_w, rows, dim, _address(out, device), ld_dx, a_dw, a_db, st)
    return out, dweight, dbias


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
        _vector(targets, rows, _I32, "targets")
    if not 0 <= top <= _lib.SPMM_TOP_MAX:
        raise ValueError(f"top must be between 0 and {_lib.SPMM_TOP_MAX}")
    device = handle.device
    a_x, a_t = _address(logits, device), _address(targets, device)
    st = _enter(device, stream, (logits, targets))
    # entropy, lse, logprob
    what = (0, rows, -1) * (2 if targets is None else 3)
    if top:
        what += (0, rows, top, _INDEX, rows, top)
    entropy, lse, *made = _new(stream, device, *what)
    logprob = top_logprob = top_index = None
    a_lp = a_tl = a_ti = 0
    if targets is not None:
        logprob = made[0]
        a_lp = logprob.data_ptr()
    if top:
        top_logprob, top_index = made[-2:]
        a_tl, a_ti = top_logprob.data_ptr(), top_index.data_ptr()
    _lib.spmm_token_logprob(handle.ptr, code, alpha, a_x, ld, rows, vocab, a_t, top, a_lp,
                            entropy.data_ptr(), lse.data_ptr(), a_tl, a_ti, st)
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
    if dlogprob is None:
        targets = None
    elif targets is None:
        raise ValueError("dlogprob needs the targets")
    else:
        _vector(targets, rows, _I32, "targets")
        _vector(dlogprob, rows, _F32, "dlogprob")
    if dentropy is None:
        entropy = None
    elif entropy is None:
        raise ValueError("dentropy needs the entropy")
    else:
        _vector(entropy, rows, _F32, "entropy")
        _vector(dentropy, rows, _F32, "dentropy")
    _vector(lse, rows, _F32, "lse")
    ld_out = vocab or 1
    if out is not None:
        ld_out = _check_out(out, rows, vocab, logits.dtype)
    device = handle.device
    a_x, a_t, a_lse = _address(logits, device), _address(targets, device), _address(lse, device)
    a_ent, a_dl, a_de = (_address(entropy, device), _address(dlogprob, device),
                         _address(dentropy, device))
    st = _enter(device, stream, (logits, targets, lse, entropy, dlogprob, dentropy, out))
    if out is None:
        out, = _new(stream, device, code, rows, vocab)
    _lib.spmm_token_logprob_grad(handle.ptr, code, alpha, a_x, ld, rows, vocab, a_t, a_lse, a_ent,
                                 a_dl, a_de, _address(out, device), ld_out, st)
    return out
