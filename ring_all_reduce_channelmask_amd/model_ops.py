"""The operators around an AllReduce in a model split over N virtual ranks.

Binding of the entry points in include/rar.h, which has their definitions:
dropout and a residual in the one-shot AllReduce, log probabilities over a
vocabulary split between the ranks, and low-rank adapters beside a
row-parallel projection.  Tensors are on one device; what a call allocates
(results, workspace) comes from torch's allocator on the call's stream.
"""
import collections
import ctypes

from . import _lib

__all__ = ["LogProbs", "adapter_allreduce", "dropout_allreduce", "dropout_allreduce_backward",
           "logprobs", "logprobs_backward"]

LogProbs = collections.namedtuple("LogProbs", "logprob entropy lse top_ids top_logprobs")
LogProbs.__doc__ = """Of each row: the given token's log probability, the entropy, the log of the
sum of exponentials (all fp32 [rows]) and the most probable tokens (int32 ids
and fp32 log probabilities, [rows, ntop])."""

_DTYPE = None


def _dtype(t):
    global _DTYPE
    if _DTYPE is None:
        import torch
        _DTYPE = {torch.float32: _lib.DTYPE["float32"], torch.bfloat16: _lib.DTYPE["bfloat16"]}
    if t.dtype not in _DTYPE:
        raise TypeError(f"unsupported dtype {t.dtype}: float32 or bfloat16")
    return _DTYPE[t.dtype]


def _on(like, stream):
    """The stream handle of a call, and the stream if it is not the current one."""
    import torch
    current = torch.cuda.current_stream(like.device)
    if stream is None or stream == current:
        return current.cuda_stream, None
    return stream.cuda_stream, stream


def _new(stream, make):
    if stream is None:
        return make()
    import torch
    with torch.cuda.stream(stream):
        return make()


def _check_list(ts, what):
    if not isinstance(ts, (list, tuple)) or not ts:
        raise ValueError(f"{what} must be a list of tensors")


def _same(t, like, what):
    if t.dtype != like.dtype or t.device != like.device or not t.is_cuda:
        raise ValueError(f"{what} must be on {like.device} with dtype {like.dtype}")


def _pointers(ts):
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


def _rows(ts, rows, what, like):
    """Widths and row strides of [rows, width] tensors with unit column stride."""
    widths, strides = [], []
    for t in ts:
        _same(t, like, what)
        if t.dim() != 2 or t.shape[0] != rows:
            raise ValueError(f"{what} must be [{rows}, width] tensors")
        w = t.shape[1]
        if w > 1 and t.stride(1) != 1:
            raise ValueError(f"{what} must have unit column stride")
        s = t.stride(0)
        if rows > 1 and s < w:
            raise ValueError(f"{what} must not have overlapping rows")
        widths.append(w)
        strides.append(s if s > w else w)
    n = len(ts)
    return (ctypes.c_int64 * n)(*widths), (ctypes.c_int64 * n)(*strides), widths


def _vector(t, n, dtype, like, what):
    if t.dtype != dtype or t.device != like.device or t.dim() != 1 or t.shape[0] != n or \
            (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} must be a contiguous [{n}] {dtype} tensor on {like.device}")
    return t.data_ptr()


def _flat(ts, count, like, what):
    for t in ts:
        _same(t, like, what)
        if t.numel() != count or not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous with {count} elements each")


def _dropout(fn, ins, outs, extra, p, rng, call, stream):
    import torch
    _check_list(ins, "the inputs")
    _check_list(outs, "the outputs")
    like = ins[0]
    dt, count = _dtype(like), like.numel()
    _flat(ins, count, like, "the inputs")
    _flat(outs, count, like, "the outputs")
    if extra is not None:
        _flat([extra], count, like, "the residual or its gradient")
    rng_ptr = _vector(rng, 2, torch.int64, like, "rng")
    handle, _ = _on(like, stream)
    _lib.check(fn(_pointers(ins), len(ins), _pointers(outs), len(outs),
                  None if extra is None else extra.data_ptr(), count, dt, p, rng_ptr, call,
                  handle))


def dropout_allreduce(sends, recvs, p, rng, call=0, residual=None, stream=None):
    """``recvs[k] = residual + dropout(sum of sends)`` for every copy k.

    ``rng`` is an int64 tensor [seed, offset] on the device; ``call`` is added
    to the offset.  The mask is drawn from them, never stored.  An output may
    be one of the inputs or the residual."""
    _dropout(_lib.load().rar_dropout_allreduce, sends, recvs, residual, p, rng, call, stream)


def dropout_allreduce_backward(grads, dsends, p, rng, call=0, dresidual=None, stream=None):
    """The gradient of dropout_allreduce from the gradients of its copies:
    ``dresidual = sum of grads``, ``dsends[r] = dropout(sum of grads)``."""
    _dropout(_lib.load().rar_dropout_allreduce_backward, grads, dsends, dresidual, p, rng, call,
             stream)


def logprobs(shards, ids, ntop=0, scale=1.0, out=None, stream=None):
    """Log probabilities of the tokens ``ids`` (int64 [rows]; -1 for none)
    under the logits ``shards`` (one [rows, width] tensor per rank, the
    vocabulary in rank order), with the entropy and the ``ntop`` most probable
    tokens.  Returns a LogProbs, written into ``out`` if one is given."""
    import torch
    _check_list(shards, "shards")
    like = shards[0]
    dt, rows = _dtype(like), like.shape[0]
    widths, strides, _ = _rows(shards, rows, "shards", like)
    n, lib = len(shards), _lib.load()
    handle, other = _on(like, stream)
    ids_ptr = _vector(ids, rows, torch.int64, like, "ids")
    need = ctypes.c_size_t()
    _lib.check(lib.rar_logprobs_workspace(widths, n, rows, dt, ntop, ctypes.byref(need)))
    if out is None:
        def make():
            f = torch.empty((3, rows), dtype=torch.float32, device=like.device).unbind(0)
            top = (torch.empty((rows, ntop), dtype=torch.int32, device=like.device),
                   torch.empty((rows, ntop), dtype=torch.float32, device=like.device))
            return LogProbs(*f, *top)
        out = _new(other, make)
    else:
        for t, what in zip(out[:3], ("logprob", "entropy", "lse")):
            _vector(t, rows, torch.float32, like, what)
        for t, d in ((out.top_ids, torch.int32), (out.top_logprobs, torch.float32)):
            if t.dtype != d or t.device != like.device or tuple(t.shape) != (rows, ntop) or \
                    not t.is_contiguous():
                raise ValueError(f"the alternatives must be contiguous [{rows}, {ntop}] tensors")
    work = _new(other, lambda: torch.empty(need.value, dtype=torch.uint8, device=like.device)) \
        if need.value else None
    _lib.check(lib.rar_logprobs(
        _pointers(shards), widths, strides, n, rows, dt, scale, ids_ptr, ntop,
        out.logprob.data_ptr(), out.entropy.data_ptr(), out.lse.data_ptr(),
        out.top_ids.data_ptr(), out.top_logprobs.data_ptr(),
        work.data_ptr() if work is not None else None, need.value, handle))
    return out


def logprobs_backward(shards, ids, lse, entropy, grad_logprob, grad_entropy=None, grad_lse=None,
                      scale=1.0, grads=None, stream=None):
    """The gradients of every rank's logits from those of logprob, entropy and
    lse (fp32 [rows]; None for zero).  ``lse`` and ``entropy`` are those that
    logprobs returned (``entropy`` may be None without ``grad_entropy``).
    Writes into ``grads`` if given, which may be ``shards`` (in place)."""
    import torch
    _check_list(shards, "shards")
    like = shards[0]
    dt, rows = _dtype(like), like.shape[0]
    widths, strides, w = _rows(shards, rows, "shards", like)
    handle, other = _on(like, stream)
    if grads is None:
        grads = _new(other, lambda: [torch.empty((rows, k), dtype=like.dtype, device=like.device)
                                     for k in w])
    _check_list(grads, "grads")
    gwidths, gstrides, gw = _rows(grads, rows, "grads", like)
    if gw != w:
        raise ValueError("grads must have the widths of shards")

    def vec(t, what):
        return None if t is None else _vector(t, rows, torch.float32, like, what)
    ids_ptr = _vector(ids, rows, torch.int64, like, "ids")
    _lib.check(_lib.load().rar_logprobs_backward(
        _pointers(shards), widths, strides, len(shards), rows, dt, scale, ids_ptr,
        vec(lse, "lse"), vec(entropy, "entropy"), vec(grad_logprob, "grad_logprob"),
        vec(grad_entropy, "grad_entropy"), vec(grad_lse, "grad_lse"), _pointers(grads), gstrides,
        handle))
    return grads


def adapter_allreduce(xs, partials, recvs, downs, up, ids, scales=None, stream=None):
    """``recvs[k][t] = sum_r partials[r][t] + scales[a] * up[a] @ (sum_r downs[r][a] @ xs[r][t])``
    with ``a = ids[t]`` (int64; outside [0, adapters): no adapter).

    ``xs``: a [tokens, width] tensor per rank; ``partials``, ``recvs``:
    [tokens, outer]; ``downs``: a [adapters, rank, width] tensor per rank;
    ``up``: [adapters, outer, rank]; ``scales``: fp32 [adapters].  An output
    may be one of the partials."""
    import torch
    for ts, what in ((xs, "xs"), (partials, "partials"), (recvs, "recvs"), (downs, "downs")):
        _check_list(ts, what)
    n, like = len(xs), xs[0]
    dt, tokens = _dtype(like), like.shape[0]
    if len(partials) != n or len(downs) != n:
        raise ValueError("xs, partials and downs need one tensor per rank")
    if up.dim() != 3:
        raise ValueError("up must be [adapters, outer, rank]")
    adapters, outer, rank = up.shape
    widths, x_strides, w = _rows(xs, tokens, "xs", like)
    _, p_strides, pw = _rows(partials, tokens, "partials", like)
    _, r_strides, rw = _rows(recvs, tokens, "recvs", like)
    if any(k != outer for k in pw + rw):
        raise ValueError(f"partials and recvs must be [{tokens}, {outer}] tensors")
    for t, k in zip(downs, w):
        _same(t, like, "downs")
        if tuple(t.shape) != (adapters, rank, k) or not t.is_contiguous():
            raise ValueError(f"downs must be contiguous [{adapters}, {rank}, width] tensors")
    _same(up, like, "up")
    if not up.is_contiguous():
        raise ValueError("up must be contiguous")
    handle, other = _on(like, stream)
    lib = _lib.load()
    need = ctypes.c_size_t()
    _lib.check(lib.rar_adapter_workspace(widths, n, tokens, dt, rank, ctypes.byref(need)))
    work = _new(other, lambda: torch.empty(need.value, dtype=torch.uint8, device=like.device))
    _lib.check(lib.rar_adapter_allreduce(
        _pointers(xs), widths, x_strides, _pointers(partials), p_strides, n, _pointers(recvs),
        r_strides, len(recvs), tokens, outer, dt, _pointers(downs), up.data_ptr(), adapters, rank,
        _vector(ids, tokens, torch.int64, like, "ids"),
        None if scales is None else _vector(scales, adapters, torch.float32, like, "scales"),
        work.data_ptr(), need.value, handle))
