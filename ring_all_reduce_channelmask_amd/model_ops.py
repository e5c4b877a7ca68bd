"""The operators around an AllReduce in a model split over N virtual ranks.

Binding of the entry points in include/rar.h, which has their definitions:
dropout and a residual in the one-shot AllReduce, log probabilities over a
vocabulary split between the ranks, and low-rank adapters beside a
row-parallel projection.  Tensors are on one device, the current one or
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
           "logprobs", "logprobs_backward"]

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
