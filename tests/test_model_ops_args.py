"""The operators around an AllReduce refuse bad arguments on the host: every
call below fails, or has nothing to do, before any HIP call.  The addresses
are made up and never dereferenced.  No GPU needed."""
import ctypes

import pytest
import torch

import ring_all_reduce_channelmask_amd as rar
from ring_all_reduce_channelmask_amd import _lib

A = 1 << 40
OK, BAD = _lib.SUCCESS, _lib.INVALID_ARGUMENT
F32, BF16, I32 = _lib.DTYPE["float32"], _lib.DTYPE["bfloat16"], _lib.DTYPE["int32"]


def _p(v):
    return None if v is None else (ctypes.c_void_p * max(1, len(v)))(*v)


def _l(v):
    return None if v is None else (ctypes.c_int64 * max(1, len(v)))(*v)


def _dropout(send=(A, A + 4096), recv=(A + 8192,), res=None, count=16, dtype=F32, p=0.1, rng=A + 65536, back=False,
             nsend=None, nrecv=None):
    lib = _lib.load()
    fn = lib.rar_dropout_allreduce_backward if back else lib.rar_dropout_allreduce
    return fn(_p(send), len(send or ()) if nsend is None else nsend, _p(recv), len(recv or ()) if nrecv is None else nrecv,
              res, count, dtype, p, rng, 0, None)


@pytest.mark.parametrize("back", [False, True])
def test_dropout_refusals(back):
    assert _dropout(count=0, back=back) == OK
    assert _dropout(count=0, send=(0,), recv=(0,), rng=None, back=back) == OK
    bad = [
        (dict(nsend=0), "no input"), (dict(nsend=65), "65 inputs"), (dict(nrecv=0), "no output"), (dict(nrecv=65), "65 outputs"),
        (dict(dtype=I32), "int32"), (dict(dtype=9), "unknown type"),
        (dict(p=-0.1), "p < 0"), (dict(p=1.1), "p > 1"), (dict(p=float("nan")), "p NaN"),
        (dict(send=None, nsend=2), "NULL array"), (dict(recv=None, nrecv=1), "NULL array"),
        (dict(send=(A, 0)), "NULL input"), (dict(recv=(0,)), "NULL output"), (dict(rng=None), "no rng"), (dict(rng=A + 65540), "rng at 4 mod 8"),
        (dict(send=(A, A + 4098)), "misaligned input"), (dict(recv=(A + 8193,)), "misaligned output"), (dict(res=A + 1), "misaligned residual"),
        (dict(dtype=BF16, recv=(A + 8193,)), "misaligned bf16"),
        (dict(recv=(A + 8192, A + 8192)), "one output twice"), (dict(recv=(A + 8192, A + 8192 + 60)), "outputs overlap"),
        (dict(recv=(A + 4,)), "an output in part over an input"), (dict(rng=A + 8192), "rng in an output"),
        (dict(count=(1 << 40) + 1), "too many"),
    ]
    for kw, why in bad:
        assert _dropout(back=back, **kw) == BAD, why
        assert _lib.load().rar_get_last_error(), why
    if back:
        assert _dropout(back=True, res=A + 8192) == BAD  # dresidual is an output
    else:
        assert _dropout(res=A + 8192 + 4) == BAD


def _logprobs(logits=(A, A + (1 << 20)), widths=(100, 50), strides=None, rows=4, dtype=F32, scale=1.0, ids=A + (2 << 20), ntop=0,
              lp=A + (3 << 20), ent=None, lse=None, tid=None, tlp=None, ws=A + (4 << 20), ws_bytes=1 << 20, n=None):
    return _lib.load().rar_logprobs(_p(logits), _l(widths), _l(strides), len(widths) if n is None else n, rows, dtype, scale, ids, ntop, lp,
                                    ent, lse, tid, tlp, ws, ws_bytes, None)


def test_logprobs_refusals():
    assert _logprobs(rows=0, logits=None, ids=None) == OK
    top = dict(ntop=3, tid=A + (5 << 20), tlp=A + (6 << 20))
    bad = [
        (dict(n=0), "no rank"), (dict(n=65), "65 ranks"), (dict(dtype=I32), "int32"), (dict(rows=-1), "rows < 0"), (dict(rows=(1 << 23) + 1), "rows"),
        (dict(widths=(100, -1)), "negative width"), (dict(widths=(0, 0)), "empty vocabulary"), (dict(widths=(1 << 30, 1)), "vocabulary too large"),
        (dict(strides=(99, 50)), "stride below width"),
        (dict(scale=0.0), "scale 0"), (dict(scale=-1.0), "scale < 0"), (dict(scale=float("inf")), "scale inf"), (dict(scale=float("nan")), "scale NaN"),
        (dict(scale=3e38), "scale overflows"), (dict(ntop=-1), "ntop < 0"), (dict(ntop=33), "ntop > 32"), (dict(ntop=3), "no room for alternatives"),
        (dict(ntop=3, tid=A + (5 << 20)), "no log probabilities"),
        (dict(logits=None), "NULL array"), (dict(logits=(A, 0)), "NULL logits"), (dict(logits=(A, A + 1)), "misaligned logits"),
        (dict(ids=None), "no ids"), (dict(ids=A + 4), "misaligned ids"), (dict(lp=None), "no output"), (dict(lp=A + (3 << 20) + 2), "misaligned output"),
        (dict(lp=A + 16), "an output in the logits"), (dict(lse=A + (3 << 20) + 8), "outputs overlap"), (dict(lp=A + (2 << 20)), "an output in ids"),
        (dict(widths=(100000, 50), ws=None), "no workspace"), (dict(widths=(100000, 50), ws_bytes=15), "workspace too small"),
        (dict(widths=(100000, 50), ws=A + (4 << 20) + 8), "misaligned workspace"), (dict(widths=(100000, 50), lp=A + (4 << 20)), "workspace overlaps"),
        (dict(top, tlp=A + (5 << 20)), "alternatives overlap"),
    ]
    for kw, why in bad:
        assert _logprobs(**kw) == BAD, why


def test_logprobs_workspace():
    lib, n = _lib.load(), ctypes.c_size_t()
    assert lib.rar_logprobs_workspace(_l([1 << 17]), 1, 1, BF16, 20, ctypes.byref(n)) == OK and n.value > 0
    assert lib.rar_logprobs_workspace(_l([1 << 17]), 1, 4096, BF16, 0, ctypes.byref(n)) == OK and n.value == 0
    assert lib.rar_logprobs_workspace(_l([0]), 1, 1, BF16, 0, ctypes.byref(n)) == BAD
    assert lib.rar_logprobs_workspace(_l([5]), 1, 1, BF16, 33, ctypes.byref(n)) == BAD
    assert lib.rar_logprobs_workspace(_l([5]), 1, 1, BF16, 0, None) == BAD
    assert lib.rar_logprobs_workspace(None, 1, 1, BF16, 0, ctypes.byref(n)) == BAD


def _backward(logits=(A, A + (1 << 20)), widths=(100, 50), strides=None, rows=4, dtype=F32, scale=1.0, ids=A + (2 << 20), lse=A + (3 << 20),
              ent=A + (4 << 20), g=A + (5 << 20), h=None, l=None, grads=(A + (6 << 20), A + (7 << 20)), gstrides=None):
    return _lib.load().rar_logprobs_backward(_p(logits), _l(widths), _l(strides), len(widths), rows, dtype, scale, ids, lse, ent, g, h, l,
                                             _p(grads), _l(gstrides), None)


def test_logprobs_backward_refusals():
    assert _backward(rows=0, logits=None, grads=None, ids=None) == OK
    bad = [
        (dict(dtype=I32), "int32"), (dict(scale=0.0), "scale"), (dict(widths=(0, 0)), "empty vocabulary"), (dict(logits=None), "NULL"), (dict(grads=None), "NULL"),
        (dict(grads=(0, A + (7 << 20))), "NULL gradient"), (dict(grads=(A + (6 << 20) + 2, A + (7 << 20))), "misaligned gradient"),
        (dict(gstrides=(99, 50)), "stride below width"), (dict(ids=None), "no ids"), (dict(lse=None), "no lse"), (dict(g=None), "no gradient in"),
        (dict(h=A + (8 << 20), ent=None), "no entropy"), (dict(g=A + (5 << 20) + 1), "misaligned"),
        (dict(grads=(A + (6 << 20), A + (6 << 20) + 40)), "gradients overlap"), (dict(grads=(A + 4, A + (7 << 20))), "in part over the logits"),
        (dict(grads=(A + (1 << 20), A + (7 << 20))), "over another rank's logits"), (dict(grads=(A + (3 << 20), A + (7 << 20))), "over lse"),
    ]
    for kw, why in bad:
        assert _backward(**kw) == BAD, why


def _adapters(xs=(A, A + (1 << 20)), widths=(64, 32), xstrides=None, ps=(A + (2 << 20), A + (3 << 20)), pstrides=None, outs=(A + (4 << 20),),
              ostrides=None, tokens=4, outer=40, dtype=F32, downs=(A + (5 << 20), A + (6 << 20)), up=A + (7 << 20), adapters=3, rank=8,
              ids=A + (8 << 20), scales=A + (9 << 20), ws=A + (10 << 20), ws_bytes=1 << 20, n=2, copies=1):
    return _lib.load().rar_adapter_allreduce(_p(xs), _l(widths), _l(xstrides), _p(ps), _l(pstrides), n, _p(outs), _l(ostrides), copies, tokens,
                                             outer, dtype, _p(downs), up, adapters, rank, ids, scales, ws, ws_bytes, None)


def test_adapter_refusals():
    assert _adapters(tokens=0, xs=None, ps=None, outs=None, downs=None, up=None, ids=None, ws=None, ws_bytes=0) == OK
    bad = [
        (dict(n=0), "no rank"), (dict(n=65), "65 ranks"), (dict(copies=0), "no output"), (dict(copies=65), "65 outputs"), (dict(dtype=I32), "int32"),
        (dict(tokens=-1), "tokens"), (dict(tokens=(1 << 24) + 1), "tokens"), (dict(adapters=0), "adapters"), (dict(rank=0), "rank"), (dict(rank=129), "rank"),
        (dict(outer=0), "outer"), (dict(widths=(-1, 32)), "width"), (dict(widths=None), "widths"), (dict(xs=None), "NULL"), (dict(xs=(A, 0)), "NULL input"),
        (dict(ps=(0, A)), "NULL partial"), (dict(outs=(0,)), "NULL output"), (dict(downs=(A + (5 << 20), 0)), "NULL weights"), (dict(up=None), "NULL weights"),
        (dict(ids=None), "no ids"), (dict(ids=A + (8 << 20) + 4), "misaligned ids"), (dict(scales=A + 2), "misaligned scales"),
        (dict(xs=(A + 2, A + (1 << 20))), "misaligned input"), (dict(xstrides=(63, 32)), "stride"), (dict(pstrides=(39, 40)), "stride"), (dict(ostrides=(39,)), "stride"),
        (dict(ws=None), "no workspace"), (dict(ws_bytes=100), "workspace too small"), (dict(ws=A + (10 << 20) + 4), "misaligned workspace"),
        (dict(outs=(A,)), "output over an input"), (dict(outs=(A + (2 << 20) + 4,)), "output in part over a partial"), (dict(outs=(A + (7 << 20),)), "output over weights"),
        (dict(outs=(A + (4 << 20),) * 2, copies=2), "outputs overlap"), (dict(ws=A + (2 << 20)), "workspace over a partial"), (dict(ws=A + (4 << 20)), "workspace over an output"),
    ]
    for kw, why in bad:
        assert _adapters(**kw) == BAD, why


def test_the_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(8)
    rng = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        rar.dropout_allreduce([x], [x.clone()], 0.1, rng)
    with pytest.raises(TypeError):
        rar.dropout_allreduce([x.int()], [x.int()], 0.1, rng)
    with pytest.raises(ValueError):
        rar.dropout_allreduce([], [x], 0.1, rng)
    with pytest.raises(ValueError):
        rar.logprobs([torch.zeros(2, 8)], torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        rar.logprobs_backward([torch.zeros(2, 8)], torch.zeros(2, dtype=torch.int64), x, x, x)
    with pytest.raises(ValueError):
        rar.adapter_allreduce([torch.zeros(2, 8)], [torch.zeros(2, 4)], [torch.zeros(2, 4)], [torch.zeros(1, 3, 8)], torch.zeros(1, 4, 3),
                              torch.zeros(2, dtype=torch.int64))
