"""The operators around an AllReduce in a model split over N virtual ranks.

Binding of the entry points in include/rar.h, which has their definitions:
dropout and a residual in the one-shot AllReduce, log probabilities over a
vocabulary split between the ranks, low-rank adapters beside a row-parallel
projection, embeddings from a table split by vocabulary, the norms around a
block with its gate and residual scale, and row-parallel projections in 8-bit
integers.  Tensors are on one device, the current one or
another; a call runs there, on that device's current stream or the given one
of its streams, with that device current: a launch goes to the current device,
and the default stream's handle is the same on all.  What it allocates
(results, workspace) comes from torch's allocator on the call's stream.

No call records a gradient: as torch's functions that write into given
tensors, each refuses inputs that require one while torch records them.
Inside torch.no_grad() or a torch.autograd.Function it takes them, and the
*_backward calls compute the gradients.
"""
import collections
import ctypes
import functools

from . import _lib

__all__ = ["LogProbs", "adapter_allreduce", "dropout_allreduce", "dropout_allreduce_backward",
           "embedding_allreduce", "embedding_allreduce_backward", "int8_projection_allreduce",
           "logprobs", "logprobs_backward", "norm_allreduce", "norm_allreduce_backward",
           "quantize_rows"]

LogProbs = collections.namedtuple("LogProbs", "logprob entropy lse top_ids top_logprobs")
LogProbs.__doc__ = """Of each row: the given token's log probability, the entropy, the log of the
sum of exponentials (all fp32 [rows]) and the most probable tokens (int32 ids
and fp32 log probabilities, [rows, ntop])."""

_torch = None
_raw_stream = _current_device = None
_DTYPE = {}


def _start(ts, what):
    """The list's first tensor, its dtype code and device index."""
    global _torch, _raw_stream, _current_device
    if _torch is None:
        import torch
        # the handle without a Stream object around it, where torch has that
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda d: torch.cuda.current_stream(d).cuda_stream)
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _DTYPE.update({torch.float32: _lib.DTYPE["float32"], torch.bfloat16: _lib.DTYPE["bfloat16"]})
        _torch = torch
    if not isinstance(ts, (list, tuple)) or not ts:
        raise ValueError(f"{what} must be a list of tensors")
    like = ts[0]
    dt = _DTYPE.get(like.dtype)
    if dt is None:
        raise TypeError(f"unsupported dtype {like.dtype}: float32 or bfloat16")
    dev = like.get_device()
    if dev < 0:
        raise ValueError(f"{what} must be device tensors")
    return like, dt, dev


def _unrecorded(what):
    """Of inputs that require a gradient: an error while torch records them."""
    if _torch.is_grad_enabled():
        raise RuntimeError(f"{what}: a gradient is required, which this call would not record; call "
                           "it under torch.no_grad() or from a torch.autograd.Function")


def _on(dev, stream):
    """The stream handle of a call, and the stream if one was given."""
    if stream is None:
        return _raw_stream(dev), None
    if getattr(stream, "device_index", dev) != dev:
        raise ValueError(f"stream must be one of cuda:{dev}, as the tensors")
    return stream.cuda_stream, stream


def _new(stream, make):
    if stream is None:
        return make()
    with _torch.cuda.stream(stream):
        return make()


_ARRAYS = [ctypes.c_void_p * n for n in range(65)]  # of as many pointers


def _pointers(ts):
    n = len(ts)
    if n > 64:
        raise ValueError("at most 64 tensors of a kind")
    return _ARRAYS[n](*[t.data_ptr() for t in ts])


@functools.lru_cache(maxsize=1024)
def _longs(values):
    """A host array of int64, read only: kept for the next call of that shape."""
    return (ctypes.c_int64 * len(values))(*values)


def _rows(ts, rows, dtype, dev, what, read=True):
    """Widths and row strides (tuples) of [rows, width] tensors with unit column stride."""
    if not isinstance(ts, (list, tuple)) or not ts:
        raise ValueError(f"{what} must be a list of tensors")
    widths, strides = [], []
    for t in ts:
        if t.dtype is not dtype or t.get_device() != dev:
            raise ValueError(f"{what} must be on cuda:{dev} with dtype {dtype}")
        if read and t.requires_grad:
            _unrecorded(what)
        shape = t.shape
        if len(shape) != 2 or shape[0] != rows:
            raise ValueError(f"{what} must be [{rows}, width] tensors")
        w = shape[1]
        s, unit = t.stride()
        if unit != 1 and w > 1:
            raise ValueError(f"{what} must have unit column stride")
        if s < w:
            if rows > 1:
                raise ValueError(f"{what} must not have overlapping rows")
            s = w
        widths.append(w)
        strides.append(s)
    return tuple(widths), tuple(strides)


def _vector(t, n, dtype, dev, what, read=True):
    if t.dtype is not dtype or t.get_device() != dev or t.shape != (n,) or \
            not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous [{n}] {dtype} tensor on cuda:{dev}")
    if read and t.requires_grad:
        _unrecorded(what)
    return t.data_ptr()


def _flat(ts, count, dtype, dev, what, read=True):
    if not isinstance(ts, (list, tuple)) or not ts:
        raise ValueError(f"{what} must be a list of tensors")
    for t in ts:
        if t.dtype is not dtype or t.get_device() != dev or t.numel() != count or \
                not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous on cuda:{dev}, with {count} elements of "
                             f"{dtype} each")
        if read and t.requires_grad:
            _unrecorded(what)


@functools.lru_cache(maxsize=1024)
def _workspace(entry, *shape):
    """Bytes of workspace that calls of a shape need."""
    need = ctypes.c_size_t()
    _lib.check(getattr(_lib.load(), entry)(_longs(shape[0]), len(shape[0]), *shape[1:],
                                           ctypes.byref(need)))
    return need.value


def _dropout(fn, ins, outs, extra, extra_read, p, rng, call, stream):
    like, dt, dev = _start(ins, "the inputs")
    if _current_device() != dev:
        with _torch.cuda.device(dev):
            return _dropout(fn, ins, outs, extra, extra_read, p, rng, call, stream)
    dtype, count = like.dtype, like.numel()
    _flat(ins, count, dtype, dev, "the inputs")
    _flat(outs, count, dtype, dev, "the outputs", False)
    if extra is not None:
        _flat((extra,), count, dtype, dev, "the residual or its gradient", extra_read)
        extra = extra.data_ptr()
    rng_ptr = _vector(rng, 2, _torch.int64, dev, "rng", False)
    handle, _ = _on(dev, stream)
    _lib.check(fn(_pointers(ins), len(ins), _pointers(outs), len(outs), extra, count, dt, p,
                  rng_ptr, call, handle))


def dropout_allreduce(sends, recvs, p, rng, call=0, residual=None, stream=None):
    """``recvs[k] = residual + dropout(sum of sends)`` for every copy k.

    ``rng`` is an int64 tensor [seed, offset] on the device; ``call`` is added
    to the offset.  The mask is drawn from them, never stored.  An output may
    be one of the inputs or the residual."""
    _dropout(_lib.load().rar_dropout_allreduce, sends, recvs, residual, True, p, rng, call,
             stream)


def dropout_allreduce_backward(grads, dsends, p, rng, call=0, dresidual=None, stream=None):
    """The gradient of dropout_allreduce from the gradients of its copies:
    ``dresidual = sum of grads``, ``dsends[r] = dropout(sum of grads)``."""
    _dropout(_lib.load().rar_dropout_allreduce_backward, grads, dsends, dresidual, False, p, rng,
             call, stream)


def logprobs(shards, ids, ntop=0, scale=1.0, out=None, stream=None):
    """Log probabilities of the tokens ``ids`` (int64 [rows]; -1 for none)
    under the logits ``shards`` (one [rows, width] tensor per rank, the
    vocabulary in rank order), with the entropy and the ``ntop`` most probable
    tokens.  Returns a LogProbs, written into ``out`` if one is given."""
    like, dt, dev = _start(shards, "shards")
    if _current_device() != dev:
        with _torch.cuda.device(dev):
            return logprobs(shards, ids, ntop, scale, out, stream)
    dtype, rows, n = like.dtype, like.size(0), len(shards)
    widths, strides = _rows(shards, rows, dtype, dev, "shards")
    handle, other = _on(dev, stream)
    ids_ptr = _vector(ids, rows, _torch.int64, dev, "ids", False)
    need = _workspace("rar_logprobs_workspace", widths, rows, dt, ntop)
    f32, i32, device = _torch.float32, _torch.int32, like.device
    if out is None:
        def make():
            return LogProbs(*_torch.empty((3, rows), dtype=f32, device=device).unbind(0),
                            _torch.empty((rows, ntop), dtype=i32, device=device),
                            _torch.empty((rows, ntop), dtype=f32, device=device))
        out = _new(other, make)
    else:
        for t, what in zip(out[:3], ("logprob", "entropy", "lse")):
            _vector(t, rows, f32, dev, what, False)
        for t, d in ((out.top_ids, i32), (out.top_logprobs, f32)):
            if t.dtype is not d or t.get_device() != dev or tuple(t.shape) != (rows, ntop) or \
                    not t.is_contiguous():
                raise ValueError(f"the alternatives must be contiguous [{rows}, {ntop}] tensors")
    work = None
    if need:
        work = _new(other, lambda: _torch.empty(need, dtype=_torch.uint8, device=device))
    _lib.check(_lib.load().rar_logprobs(
        _pointers(shards), _longs(widths), _longs(strides), n, rows, dt, scale, ids_ptr, ntop,
        out.logprob.data_ptr(), out.entropy.data_ptr(), out.lse.data_ptr(),
        out.top_ids.data_ptr(), out.top_logprobs.data_ptr(),
        work.data_ptr() if need else None, need, handle))
    return out


def logprobs_backward(shards, ids, lse, entropy, grad_logprob, grad_entropy=None, grad_lse=None,
                      scale=1.0, grads=None, stream=None):
    """The gradients of every rank's logits from those of logprob, entropy and
    lse (fp32 [rows]; None for zero).  ``lse`` and ``entropy`` are those that
    logprobs returned (``entropy`` may be None without ``grad_entropy``).
    Writes into ``grads`` if given, which may be ``shards`` (in place)."""
    like, dt, dev = _start(shards, "shards")
    if _current_device() != dev:
        with _torch.cuda.device(dev):
            return logprobs_backward(shards, ids, lse, entropy, grad_logprob, grad_entropy,
                                     grad_lse, scale, grads, stream)
    dtype, rows = like.dtype, like.size(0)
    widths, strides = _rows(shards, rows, dtype, dev, "shards")
    handle, other = _on(dev, stream)
    if grads is None:
        grads = _new(other, lambda: [_torch.empty((rows, k), dtype=dtype, device=like.device)
                                     for k in widths])
    gwidths, gstrides = _rows(grads, rows, dtype, dev, "grads", False)
    if gwidths != widths:
        raise ValueError("grads must have the widths of shards")
    f32 = _torch.float32

    def vec(t, what):
        return None if t is None else _vector(t, rows, f32, dev, what)
    ids_ptr = _vector(ids, rows, _torch.int64, dev, "ids", False)
    _lib.check(_lib.load().rar_logprobs_backward(
        _pointers(shards), _longs(widths), _longs(strides), len(shards), rows, dt, scale, ids_ptr,
        vec(lse, "lse"), vec(entropy, "entropy"), vec(grad_logprob, "grad_logprob"),
        vec(grad_entropy, "grad_entropy"), vec(grad_lse, "grad_lse"), _pointers(grads),
        _longs(gstrides), handle))
    return grads


def adapter_allreduce(xs, partials, recvs, downs, up, ids, scales=None, stream=None):
    """``recvs[k][t] = sum_r partials[r][t] + scales[a] * up[a] @ (sum_r downs[r][a] @ xs[r][t])``
    with ``a = ids[t]`` (int64; outside [0, adapters): no adapter).

    ``xs``: a [tokens, width] tensor per rank; ``partials``, ``recvs``:
    [tokens, outer]; ``downs``: a [adapters, rank, width] tensor per rank;
    ``up``: [adapters, outer, rank]; ``scales``: fp32 [adapters].  An output
    may be one of the partials."""
    like, dt, dev = _start(xs, "xs")
    if _current_device() != dev:
        with _torch.cuda.device(dev):
            return adapter_allreduce(xs, partials, recvs, downs, up, ids, scales, stream)
    dtype, tokens, n = like.dtype, like.size(0), len(xs)
    widths, x_strides = _rows(xs, tokens, dtype, dev, "xs")
    outers, p_strides = _rows(partials, tokens, dtype, dev, "partials")
    recv_outers, r_strides = _rows(recvs, tokens, dtype, dev, "recvs", False)
    if up.dim() != 3 or up.dtype is not dtype or up.get_device() != dev or not up.is_contiguous():
        raise ValueError("up must be a contiguous [adapters, outer, rank] tensor like xs")
    if up.requires_grad:
        _unrecorded("up")
    adapters, outer, rank = up.shape
    if outers != (outer,) * n or recv_outers != (outer,) * len(recvs):
        raise ValueError(f"partials (one per rank) and recvs must be [{tokens}, {outer}] tensors")
    if not isinstance(downs, (list, tuple)) or len(downs) != n:
        raise ValueError("downs needs one tensor per rank")
    for t, k in zip(downs, widths):
        if t.dtype is not dtype or t.get_device() != dev or t.shape != (adapters, rank, k) or \
                not t.is_contiguous():
            raise ValueError(f"downs must be contiguous [{adapters}, {rank}, width] tensors like xs")
        if t.requires_grad:
            _unrecorded("downs")
    handle, other = _on(dev, stream)
    need = _workspace("rar_adapter_workspace", widths, tokens, dt, rank)
    work = _new(other, lambda: _torch.empty(need, dtype=_torch.uint8, device=like.device))
    _lib.check(_lib.load().rar_adapter_allreduce(
        _pointers(xs), _longs(widths), _longs(x_strides), _pointers(partials), _longs(p_strides),
        n, _pointers(recvs), _longs(r_strides), len(recvs), tokens, outer, dt, _pointers(downs),
        up.data_ptr(), adapters, rank, _vector(ids, tokens, _torch.int64, dev, "ids", False),
        None if scales is None else _vector(scales, adapters, _torch.float32, dev, "scales"),
        work.data_ptr(), need, handle))


def _table_rows(ts, width, dtype, dev, what, read=True):
    """Numbers of rows and row strides (tuples) of [rows, width] tensors with unit column stride."""
    if not isinstance(ts, (list, tuple)) or not ts:
        raise ValueError(f"{what} must be a list of tensors")
    rows, strides = [], []
    for t in ts:
        shape = t.shape
        if len(shape) != 2 or shape[1] != width:
            raise ValueError(f"{what} must be [rows, {width}] tensors")
        rows.append(shape[0])
        if shape[0] == 0 and t.dtype is dtype and t.get_device() == dev:
            strides.append(width)  # a rank without rows: its strides mean nothing
        else:
            strides.append(_rows((t,), shape[0], dtype, dev, what, read)[1][0])
    return tuple(rows), tuple(strides)


def embedding_allreduce(tables, ids, recvs, scale=1.0, stream=None):
    """``recvs[k][t] = scale * E[ids[t]]`` for every copy k, the table E split
    by vocabulary: ``tables`` has a [rows, width] tensor per rank, in rank
    order.  ``ids``: int64 [tokens]; outside the vocabulary (-1): zeros."""
    like, dt, dev = _start(tables, "tables")
    if _current_device() != dev:
        with _torch.cuda.device(dev):
            return embedding_allreduce(tables, ids, recvs, scale, stream)
    if like.dim() != 2 or ids.dim() != 1:
        raise ValueError("tables must be [rows, width] tensors and ids a [tokens] one")
    dtype, width, tokens = like.dtype, like.size(1), ids.size(0)
    rows, strides = _table_rows(tables, width, dtype, dev, "tables")
    handle, _ = _on(dev, stream)
    _lib.check(_lib.load().rar_embedding_allreduce(
        _pointers(tables), _longs(rows), _longs(strides), len(tables), width, dt,
        _vector(ids, tokens, _torch.int64, dev, "ids", False), tokens, scale,
        *_copies(recvs, tokens, width, dtype, dev, "recvs", False), handle))


def embedding_allreduce_backward(grads, ids, dtables, scale=1.0, accumulate=False, stream=None):
    """The gradient of embedding_allreduce's tables from those of its copies,
    into ``dtables`` (like the tables, of the gradients' dtype or float32):
    every row is written, or with ``accumulate`` the rows of tokens that occur
    are added to.  Equal tokens are summed in fp32, in an order that depends on
    the sizes and the ids alone."""
    like, dt, dev = _start(grads, "grads")
    if _current_device() != dev:
        with _torch.cuda.device(dev):
            return embedding_allreduce_backward(grads, ids, dtables, scale, accumulate, stream)
    if like.dim() != 2:
        raise ValueError("grads must be [tokens, width] tensors")
    dtype, (tokens, width) = like.dtype, like.shape
    grad_args = _copies(grads, tokens, width, dtype, dev, "grads", True)
    if not isinstance(dtables, (list, tuple)) or not dtables or \
            dtables[0].dtype not in (dtype, _torch.float32):
        raise ValueError(f"dtables must be a list of {dtype} or float32 tensors")
    out_dtype = dtables[0].dtype
    rows, strides = _table_rows(dtables, width, out_dtype, dev, "dtables", False)
    handle, other = _on(dev, stream)
    need = _workspace("rar_embedding_workspace", rows, tokens, width, dt)
    work = None
    if need:
        work = _new(other, lambda: _torch.empty(need, dtype=_torch.uint8, device=like.device))
    _lib.check(_lib.load().rar_embedding_allreduce_backward(
        *grad_args, tokens, width, dt,
        _vector(ids, tokens, _torch.int64, dev, "ids", False), scale, _pointers(dtables),
        _longs(rows), _longs(strides), len(dtables), _DTYPE[out_dtype], int(bool(accumulate)),
        work.data_ptr() if need else None, need, handle))


def _norm(rows, width, dtype, dt, dev, eps, residual_scale, post_weight, gate, pre_weight):
    """The arguments that a norm and its gradient share."""
    def weight(t, what):
        return None if t is None else _vector(t, width, dtype, dev, what)
    at, groups, stride = None, 0, 0
    if gate is not None:
        at, groups, stride = _gate(gate, width, dtype, dev, "gate")
        if not rows:  # then a gate has any number of groups, and no use
            at, groups, stride = None, 0, 0
        elif not groups:  # no address either, which would mean: no gate
            raise ValueError(f"gate must have groups that divide the {rows} rows")
    return _lib.Norm(rows, width, dt, eps, residual_scale, 0, weight(post_weight, "post_weight"),
                     weight(pre_weight, "pre_weight"), at, groups, stride)


def _gate(t, width, dtype, dev, what, read=True):
    """Address, groups and stride of a [width] or [groups, width] tensor."""
    if len(t.shape) == 1:
        return _vector(t, width, dtype, dev, what, read), 1, width
    if len(t.shape) != 2 or t.shape[1] != width:
        raise ValueError(f"{what} must be a [{width}] or [groups, {width}] tensor")
    return t.data_ptr(), t.shape[0], _rows((t,), t.shape[0], dtype, dev, what, read)[1][0]


def _copies(ts, rows, width, dtype, dev, what, read):
    """Addresses, strides and number of [rows, width] tensors (none allowed)."""
    if not isinstance(ts, (list, tuple)):
        raise ValueError(f"{what} must be a list of tensors")
    n = len(ts)
    if n == 0:
        return None, None, 0
    if n > 64:
        raise ValueError("at most 64 tensors of a kind")
    # what most calls have, checked at once; _rows says what is wrong with others
    shape, strides, recorded = (rows, width), (width, 1), read and _torch.is_grad_enabled()
    for t in ts:
        if t.stride() != strides or t.shape != shape or t.dtype is not dtype or \
                t.get_device() != dev or (recorded and t.requires_grad):
            break
    else:
        return _ARRAYS[n](*[t.data_ptr() for t in ts]), _longs((width,) * n), n
    widths, strides = _rows(ts, rows, dtype, dev, what, read)
    if widths != (width,) * n:
        raise ValueError(f"{what} must be [{rows}, {width}] tensors")
    return _pointers(ts), _longs(strides), n


def _single(t, rows, width, dtype, dev, what, read):
    """Address and stride of a [rows, width] tensor or None."""
    if t is None:
        return None, 0
    widths, strides = _rows((t,), rows, dtype, dev, what, read)
    if widths != (width,):
        raise ValueError(f"{what} must be a [{rows}, {width}] tensor")
    return t.data_ptr(), strides[0]


@functools.lru_cache(maxsize=1024)
def _norm_workspace(rows, width, dt, groups):
    """Bytes of workspace of a norm's gradient."""
    need = ctypes.c_size_t()
    n = _lib.Norm(rows, width, dt, 1.0, 1.0, 0, None, None, 1 << 40 if groups else None, groups, 0)
    _lib.check(_lib.load().rar_norm_workspace(ctypes.byref(n), ctypes.byref(need)))
    return need.value


def norm_allreduce(partials, hidden, outs, residual=None, residual_scale=1.0, post_weight=None,
                   gate=None, pre_weight=None, eps=1e-6, total=None, stream=None):
    """The AllReduce of a block's partial products with the norms around the
    block, with ``rms(x) = x / sqrt(mean(x^2) + eps)`` of each row:

        total     = sum of partials
        hidden[k] = residual_scale * residual + gate * (rms(total) * post_weight)
        outs[k]   = rms(hidden) * pre_weight

    All of them [rows, width] tensors; ``hidden`` and ``outs`` lists of copies
    (one of them may be empty), ``total`` what the gradient needs, if wanted.
    Without ``post_weight`` the sum is not normed.  ``gate``: a [width] vector,
    or [groups, width], where the rows are as many equal runs.  An output may
    be one of the partials or the residual."""
    like, dt, dev = _start(partials, "partials")
    if _current_device() != dev:
        with _torch.cuda.device(dev):
            return norm_allreduce(partials, hidden, outs, residual, residual_scale, post_weight,
                                  gate, pre_weight, eps, total, stream)
    if len(like.shape) != 2:
        raise ValueError("partials must be [rows, width] tensors")
    dtype, (rows, width) = like.dtype, like.shape
    n = _norm(rows, width, dtype, dt, dev, eps, residual_scale, post_weight, gate, pre_weight)
    handle, _ = _on(dev, stream)
    _lib.check(_lib.load().rar_norm_allreduce(
        ctypes.byref(n), *_copies(partials, rows, width, dtype, dev, "partials", True),
        *_single(residual, rows, width, dtype, dev, "residual", True),
        *_copies(hidden, rows, width, dtype, dev, "hidden", False),
        *_copies(outs, rows, width, dtype, dev, "outs", False),
        *_single(total, rows, width, dtype, dev, "total", False), handle))


def norm_allreduce_backward(grad_hidden, grad_outs, dpartials, total=None, hidden=None,
                            residual_scale=1.0, post_weight=None, gate=None, pre_weight=None,
                            eps=1e-6, dresidual=None, dpost_weight=None, dgate=None,
                            dpre_weight=None, stream=None):
    """The gradient of norm_allreduce from those of the copies of hidden and of
    outs (lists; one may be empty) and from its ``total`` (needed with a
    ``post_weight`` or for ``dgate``) and ``hidden`` (needed with
    ``grad_outs``).  Writes the partials' gradient, the same for every rank,
    into each tensor of ``dpartials``, and those of the residual, the weights
    and the gate where they are given."""
    given = list(grad_hidden) + list(grad_outs)
    like, dt, dev = _start(given, "grad_hidden and grad_outs")
    if _current_device() != dev:
        with _torch.cuda.device(dev):
            return norm_allreduce_backward(grad_hidden, grad_outs, dpartials, total, hidden,
                                           residual_scale, post_weight, gate, pre_weight, eps,
                                           dresidual, dpost_weight, dgate, dpre_weight, stream)
    if len(like.shape) != 2:
        raise ValueError("gradients must be [rows, width] tensors")
    dtype, (rows, width) = like.dtype, like.shape
    n = _norm(rows, width, dtype, dt, dev, eps, residual_scale, post_weight, gate, pre_weight)

    def vector(t, what):
        return None if t is None else _vector(t, width, dtype, dev, what, False)
    dgate_ptr, dgate_stride = None, 0
    if dgate is not None:
        if gate is None or dgate.shape != gate.shape:
            raise ValueError("dgate must have the shape of gate")
        dgate_ptr, _, dgate_stride = _gate(dgate, width, dtype, dev, "dgate", False)
        if not rows:  # zeroed below, whatever its number of groups
            dgate_ptr, dgate_stride = None, 0
    handle, other = _on(dev, stream)
    lib, need = _lib.load(), _norm_workspace(rows, width, dt, n.gate_groups)
    work = None
    if need:
        work = _new(other, lambda: _torch.empty(need, dtype=_torch.uint8, device=like.device))
    _lib.check(lib.rar_norm_allreduce_backward(
        ctypes.byref(n), *_copies(grad_hidden, rows, width, dtype, dev, "grad_hidden", True),
        *_copies(grad_outs, rows, width, dtype, dev, "grad_outs", True),
        *_single(total, rows, width, dtype, dev, "total", True),
        *_single(hidden, rows, width, dtype, dev, "hidden", True),
        *_copies(dpartials, rows, width, dtype, dev, "dpartials", False),
        *_single(dresidual, rows, width, dtype, dev, "dresidual", False),
        vector(dpost_weight, "dpost_weight"), dgate_ptr, dgate_stride,
        vector(dpre_weight, "dpre_weight"), work.data_ptr() if need else None, need, handle))
    if dgate is not None and not rows:
        _new(other, dgate.zero_)


def quantize_rows(xs, quantized=None, scales=None, stream=None):
    """Rows split over the ranks (``xs``: a [rows, width] tensor per rank) to
    8-bit integers with one scale a row for all ranks, the largest magnitude /
    127: returns (int8 tensors like xs, fp32 scales [rows]), written into those
    given.  New tensors have rows that begin on multiples of 16 bytes."""
    like, dt, dev = _start(xs, "xs")
    if _current_device() != dev:
        with _torch.cuda.device(dev):
            return quantize_rows(xs, quantized, scales, stream)
    dtype, rows = like.dtype, like.size(0)
    widths, strides = _rows(xs, rows, dtype, dev, "xs")
    handle, other = _on(dev, stream)
    int8, f32, device = _torch.int8, _torch.float32, like.device
    if quantized is None:
        # one buffer, the ranks' columns side by side
        pitches, pitch, even = _pitches(widths)
        held = _new(other, lambda: _torch.empty((rows, pitch), dtype=int8, device=device))
        quantized = list(held.split(pitches, 1))
        if not even:
            quantized = [t[:, :k] for t, k in zip(quantized, widths)]
        q_strides = (pitch,) * len(xs)
    else:
        q_widths, q_strides = _rows(quantized, rows, int8, dev, "quantized", False)
        if q_widths != widths:
            raise ValueError("quantized must have the widths of xs")
    if scales is None:
        scales = _new(other, lambda: _torch.empty(rows, dtype=f32, device=device))
    _lib.check(_lib.load().rar_quantize_rows(
        _pointers(xs), _longs(widths), _longs(strides), len(xs), rows, dt, _pointers(quantized),
        _longs(q_strides), _vector(scales, rows, f32, dev, "scales", False), handle))
    return quantized, scales


@functools.lru_cache(maxsize=1024)
def _pitches(widths):
    """Widths rounded up to multiples of 16, their sum, and whether all were."""
    pitches = [(k + 15) // 16 * 16 for k in widths]
    return pitches, sum(pitches), pitches == list(widths)


@functools.lru_cache(maxsize=1024)
def _bits(strides):
    """The low bits that strides have, all where one is beyond what tiles take."""
    bits = 15 if max(strides) >= (1 << 24) - 256 else 0
    for s in strides:
        bits |= s & 15
    return bits


def int8_projection_allreduce(xs, x_scales, weights, weight_scales, recvs, residual=None,
                              stream=None):
    """``recvs[k][t, d] = residual[t, d] + x_scales[t] * weight_scales[d] *
    sum_r xs[r][t] . weights[r][d]`` for every copy k, the sum in exact integers.

    ``xs``: an int8 [tokens, width] tensor per rank, ``weights``: an int8
    [outer, width] one, as quantize_rows gives them; the scales fp32 [tokens]
    and [outer].  ``recvs`` and ``residual`` are float32 or bfloat16; an output
    may be the residual."""
    like, dt, dev = _start(recvs, "recvs")
    if _current_device() != dev:
        with _torch.cuda.device(dev):
            return int8_projection_allreduce(xs, x_scales, weights, weight_scales, recvs, residual,
                                             stream)
    if len(like.shape) != 2:
        raise ValueError("recvs must be [tokens, outer] tensors")
    dtype, (tokens, outer) = like.dtype, like.shape
    int8, f32 = _torch.int8, _torch.float32
    widths, x_strides = _rows(xs, tokens, int8, dev, "xs", False)
    w_widths, w_strides = _rows(weights, outer, int8, dev, "weights", False)
    if w_widths != widths:
        raise ValueError("weights must have the widths of xs")
    recv_ptrs, r_strides, copies = _copies(recvs, tokens, outer, dtype, dev, "recvs", False)
    res, res_stride = _single(residual, tokens, outer, dtype, dev, "residual", True)
    handle, other = _on(dev, stream)
    x_ptrs, w_ptrs = _pointers(xs), _pointers(weights)
    bits = _bits(x_strides) | _bits(w_strides)  # odd where too far apart
    for p in x_ptrs:
        bits |= p or 0
    for p in w_ptrs:
        bits |= p or 0
    need = _workspace("rar_int8_projection_workspace", widths, tokens, outer, dt,
                      int(bits & 15 == 0))
    work = None
    if need:
        work = _new(other, lambda: _torch.empty(need, dtype=_torch.uint8, device=like.device))
    _lib.check(_lib.load().rar_int8_projection_allreduce(
        x_ptrs, _longs(widths), _longs(x_strides),
        _vector(x_scales, tokens, f32, dev, "x_scales"), w_ptrs, _longs(w_strides),
        _vector(weight_scales, outer, f32, dev, "weight_scales"), len(xs), tokens, outer, dt, res,
        res_stride, recv_ptrs, r_strides, copies, work.data_ptr() if need else None, need, handle))
