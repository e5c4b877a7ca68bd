"""Embeddings, norms and 8-bit projections refuse bad arguments on the host:
every call below fails, or has nothing to do, before any HIP call.  The
addresses are made up and never dereferenced.  No GPU needed."""
import ctypes
import os
import shutil
import subprocess
import tempfile

import numpy as np
import pytest
import torch

import ring_all_reduce_channelmask_amd as rar
from oracle import model_ops as oracle
from ring_all_reduce_channelmask_amd import _lib

from .test_model_ops_args import A, BAD, BF16, F32, I32, OK, _l, _p

M = 1 << 20


def _message():
    return _lib.load().rar_get_last_error().decode()


def _embedding(tables=(A, A + M), rows=(10, 20), tstrides=None, n=2, width=16, dtype=F32, ids=A + 2 * M, tokens=4, scale=1.0, recvs=(A + 3 * M,),
               rstrides=None, copies=1):
    return _lib.load().rar_embedding_allreduce(_p(tables), _l(rows), _l(tstrides), n, width, dtype, ids, tokens, scale, _p(recvs), _l(rstrides), copies, None)


def test_embedding_refusals():
    assert _embedding(tokens=0, tables=None, ids=None, recvs=None) == OK
    bad = [
        (dict(n=0), "no rank"), (dict(n=65), "65 ranks"), (dict(copies=0), "no output"), (dict(copies=65), "65 outputs"), (dict(dtype=I32), "int32"),
        (dict(rows=None), "no rows"), (dict(rows=(-1, 20)), "negative rows"), (dict(rows=(0, 0)), "empty vocabulary"), (dict(rows=(1 << 30, 1)), "too many rows"),
        (dict(rows=((1 << 62), 1 << 62)), "rows overflow"), (dict(width=0), "width"), (dict(width=(1 << 24) + 1), "width"), (dict(tokens=-1), "tokens"),
        (dict(tokens=(1 << 24) + 1), "tokens"), (dict(scale=float("nan")), "scale NaN"), (dict(scale=float("inf")), "scale inf"),
        (dict(tables=None), "NULL array"), (dict(recvs=None), "NULL array"), (dict(tables=(A, 0)), "NULL table"), (dict(recvs=(0,)), "NULL output"),
        (dict(ids=None), "no ids"), (dict(ids=A + 2 * M + 4), "misaligned ids"), (dict(tables=(A + 2, A + M)), "misaligned table"),
        (dict(recvs=(A + 3 * M + 1,), dtype=BF16), "misaligned output"), (dict(tstrides=(15, 16)), "stride"), (dict(rstrides=(15,)), "stride"),
        (dict(tstrides=(1 << 60, 16)), "far stride"), (dict(rstrides=(1 << 60,)), "far stride"),
        (dict(recvs=(A + 64,)), "output over a table"), (dict(recvs=(A + 2 * M,)), "output over ids"), (dict(recvs=(A + 3 * M, A + 3 * M + 64), copies=2), "outputs overlap"),
        (dict(tokens=1 << 24, width=1 << 24), "too large"),
    ]
    for kw, why in bad:
        assert _embedding(**kw) == BAD, why
        assert _message(), why


def _embedding_back(grads=(A, A + M), gstrides=None, n=2, tokens=4, width=16, dtype=F32, ids=A + 2 * M, scale=1.0, tables=(A + 3 * M, A + 4 * M), rows=(10, 20),
                    tstrides=None, ranks=2, tdtype=F32, acc=0, ws=A + 5 * M, ws_bytes=1 << 30):
    return _lib.load().rar_embedding_allreduce_backward(_p(grads), _l(gstrides), n, tokens, width, dtype, ids, scale, _p(tables), _l(rows), _l(tstrides), ranks,
                                                        tdtype, acc, ws, ws_bytes, None)


def test_embedding_gradient_refusals():
    assert _embedding_back(tokens=0, acc=1, grads=None, ids=None, tables=None, ws=None, ws_bytes=0) == OK
    bad = [
        (dict(n=0), "no gradient"), (dict(n=65), "65 gradients"), (dict(ranks=0), "no rank"), (dict(ranks=65), "65 ranks"), (dict(dtype=I32), "int32"),
        (dict(tdtype=I32), "int32 table"), (dict(tdtype=BF16), "bf16 table of fp32 gradients"), (dict(acc=2), "accumulate"), (dict(acc=-1), "accumulate"),
        (dict(rows=(0, 0)), "empty"), (dict(rows=None), "no rows"), (dict(width=0), "width"), (dict(tokens=-1), "tokens"), (dict(scale=float("inf")), "scale"),
        (dict(grads=None), "NULL"), (dict(tables=None), "NULL"), (dict(grads=(A, 0)), "NULL gradient"), (dict(tables=(0, A)), "NULL table"),
        (dict(tables=None, tokens=0), "NULL table of no tokens"), (dict(ids=None), "ids"), (dict(ids=A + 2 * M + 2), "ids"), (dict(gstrides=(15, 16)), "stride"),
        (dict(tstrides=(15, 16)), "stride"), (dict(grads=(A + 1, A + M)), "misaligned"), (dict(tables=(A + 3 * M + 2, A + 4 * M)), "misaligned"),
        (dict(tables=(A, A + 4 * M)), "table over a gradient"), (dict(tables=(A + 3 * M, A + 3 * M + 64)), "tables overlap"), (dict(tables=(A + 2 * M, A + 4 * M)), "over ids"),
        (dict(tokens=2000, ws=None), "no workspace"), (dict(tokens=2000, ws_bytes=100), "workspace too small"), (dict(tokens=2000, ws=A + 5 * M + 8), "misaligned workspace"),
        (dict(tokens=2000, ws=A), "workspace over a gradient"), (dict(tokens=2000, ws=A + 3 * M), "workspace over a table"),
    ]
    for kw, why in bad:
        assert _embedding_back(**kw) == BAD, why
        assert _message(), why


def test_embedding_workspace():
    lib, n = _lib.load(), ctypes.c_size_t()
    assert lib.rar_embedding_workspace(_l([100]), 1, 5, 64, BF16, ctypes.byref(n)) == OK and n.value == 0
    assert lib.rar_embedding_workspace(_l([100]), 1, 50000, 64, BF16, ctypes.byref(n)) == OK and n.value > 0
    assert lib.rar_embedding_workspace(_l([100]), 1, 5, 64, BF16, None) == BAD
    assert lib.rar_embedding_workspace(None, 1, 5, 64, BF16, ctypes.byref(n)) == BAD
    assert lib.rar_embedding_workspace(_l([0]), 1, 5, 64, BF16, ctypes.byref(n)) == BAD
    assert lib.rar_embedding_workspace(_l([100]), 1, 5, 64, I32, ctypes.byref(n)) == BAD
    assert lib.rar_embedding_workspace(_l([100]), 1, -5, 64, BF16, ctypes.byref(n)) == BAD


def _config(rows=8, width=16, dtype=F32, eps=1e-6, residual_scale=1.0, post=A + 20 * M, pre=A + 21 * M, gate=A + 22 * M, groups=2, gate_stride=0):
    return _lib.Norm(rows=rows, width=width, dtype=dtype, eps=eps, residual_scale=residual_scale, post_weight=post, pre_weight=pre, gate=gate, gate_groups=groups,
                     gate_stride=gate_stride)


CONFIG = [
    (dict(rows=-1), "rows"), (dict(rows=(1 << 24) + 1), "rows"), (dict(width=0), "width"), (dict(width=32769), "width"), (dict(dtype=I32), "int32"),
    (dict(eps=0.0), "eps"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"), (dict(residual_scale=float("nan")), "scale"),
    (dict(residual_scale=float("inf")), "scale"), (dict(groups=3), "groups"), (dict(groups=0), "groups"), (dict(groups=16), "groups"), (dict(rows=0, groups=2), "groups"),
    (dict(post=A + 20 * M + 2), "misaligned weight"), (dict(pre=A + 21 * M + 1), "misaligned weight"), (dict(gate=A + 22 * M + 2), "misaligned gate"),
    (dict(gate_stride=15), "gate stride"), (dict(gate_stride=1 << 60), "gate stride"),
]


def _norm(partials=(A, A + M), pstrides=None, n=2, res=A + 2 * M, res_stride=0, hidden=(A + 3 * M,), hstrides=None, nh=1, outs=(A + 4 * M,), ostrides=None, no=1,
          total=A + 5 * M, total_stride=0, config=None, **kw):
    c = _config(**kw) if config is None else config
    return _lib.load().rar_norm_allreduce(ctypes.byref(c) if c else None, _p(partials), _l(pstrides), n, res, res_stride, _p(hidden), _l(hstrides), nh, _p(outs),
                                          _l(ostrides), no, total, total_stride, None)


def test_norm_refusals():
    assert _norm(rows=0, groups=1, partials=None, hidden=None, outs=None, total=None) == OK
    bad = CONFIG + [
        (dict(config=False), "no norm"), (dict(n=0), "no rank"), (dict(n=65), "65 ranks"), (dict(nh=-1), "outputs"), (dict(nh=65), "outputs"), (dict(no=65), "outputs"),
        (dict(nh=0, no=0), "no output"), (dict(pre=None), "no weight"), (dict(partials=None), "NULL"), (dict(hidden=None), "NULL"), (dict(outs=None), "NULL"),
        (dict(partials=(A, 0)), "NULL partial"), (dict(hidden=(0,)), "NULL hidden"), (dict(outs=(0,)), "NULL out"), (dict(partials=(A + 2, A + M)), "misaligned"),
        (dict(res=A + 2 * M + 1), "misaligned"), (dict(total=A + 5 * M + 2), "misaligned"), (dict(pstrides=(15, 16)), "stride"), (dict(res_stride=15), "stride"),
        (dict(hstrides=(15,)), "stride"), (dict(ostrides=(15,)), "stride"), (dict(total_stride=15), "stride"), (dict(pstrides=(1 << 60, 16)), "far stride"),
        (dict(hidden=(A + 4 * M,)), "outputs overlap"), (dict(hidden=(A + 3 * M, A + 3 * M + 64), nh=2), "outputs overlap"), (dict(total=A + 3 * M), "outputs overlap"),
        (dict(hidden=(A + 64,)), "in part over a partial"), (dict(hidden=(A + 2 * M,), hstrides=(32,)), "over the residual with another stride"),
        (dict(hidden=(A + 20 * M,)), "over a weight"), (dict(outs=(A + 21 * M,)), "over a weight"), (dict(total=A + 22 * M), "over the gate"),
        (dict(rows=1, groups=1, hidden=(A + 20 * M,)), "a row over a weight"),
    ]
    for kw, why in bad:
        assert _norm(**kw) == BAD, why
        assert _message(), why


def _norm_back(gh=(A, A + M), ghs=None, ngh=2, go=(A + 2 * M,), gos=None, ngo=1, total=A + 3 * M, ts=0, hidden=A + 4 * M, hs=0, dp=(A + 5 * M,), dps=None, ndp=1,
               dres=A + 6 * M, drs=0, dpost=A + 7 * M, dgate=A + 8 * M, dgs=0, dpre=A + 9 * M, ws=A + 10 * M, ws_bytes=1 << 30, config=None, **kw):
    c = _config(**kw) if config is None else config
    return _lib.load().rar_norm_allreduce_backward(ctypes.byref(c) if c else None, _p(gh), _l(ghs), ngh, _p(go), _l(gos), ngo, total, ts, hidden, hs, _p(dp), _l(dps),
                                                   ndp, dres, drs, dpost, dgate, dgs, dpre, ws, ws_bytes, None)


def test_norm_gradient_refusals():
    assert _norm_back(rows=0, groups=1, gh=None, go=None, total=None, hidden=None, dp=None, dres=None, dpost=None, dgate=None, dpre=None, ws=None, ws_bytes=0) == OK
    bad = CONFIG + [
        (dict(config=False), "no norm"), (dict(ngh=-1), "gradients"), (dict(ngh=65), "gradients"), (dict(ngo=65), "gradients"), (dict(ndp=65), "gradients"),
        (dict(ngh=0, ngo=0, dpre=None), "no gradient"), (dict(pre=None), "no weight"), (dict(ngo=0), "dpre without grad_outs"), (dict(post=None), "dpost without a weight"),
        (dict(gate=None), "dgate without a gate"), (dict(gh=None), "NULL"), (dict(go=None), "NULL"), (dict(dp=None), "NULL"), (dict(gh=(A, 0)), "NULL gradient"),
        (dict(total=None), "no total"), (dict(total=None, post=None, dpost=None), "no total for dgate"), (dict(hidden=None), "no hidden"),
        (dict(dres=A + 6 * M + 2), "misaligned"), (dict(dpost=A + 7 * M + 1), "misaligned"), (dict(dgate=A + 8 * M + 2), "misaligned"), (dict(dpre=A + 9 * M + 3), "misaligned"),
        (dict(ghs=(15, 16)), "stride"), (dict(gos=(15,)), "stride"), (dict(ts=15), "stride"), (dict(hs=15), "stride"), (dict(dps=(15,)), "stride"), (dict(drs=15), "stride"),
        (dict(dgs=15), "stride"), (dict(ws=None), "no workspace"), (dict(ws_bytes=60), "workspace too small"), (dict(ws=A + 10 * M + 8), "misaligned workspace"),
        (dict(dp=(A + 6 * M,)), "outputs overlap"), (dict(dp=(A + 64,)), "in part over a gradient"), (dict(dres=A + 20 * M), "over a weight"), (dict(dp=(A + 22 * M,)), "over the gate"),
        (dict(dpost=A + 4 * M), "a weight's gradient over hidden"), (dict(dpre=A + 20 * M), "over a weight"), (dict(dgate=A + 22 * M), "over the gate"),
        (dict(dgate=A), "the gate's gradient over a gradient"), (dict(dpost=A + 9 * M), "outputs overlap"), (dict(ws=A), "workspace over an input"),
        (dict(ws=A + 5 * M), "workspace over an output"), (dict(rows=1, groups=1, dpost=A), "a weight's gradient over the one row of another"),
        (dict(rows=8, groups=8, dgate=A), "a gate a row over a gradient"),
    ]
    for kw, why in bad:
        assert _norm_back(**kw) == BAD, why
        assert _message(), why


def test_norm_workspace():
    lib, n = _lib.load(), ctypes.c_size_t()
    assert lib.rar_norm_workspace(ctypes.byref(_config(rows=0, groups=1)), ctypes.byref(n)) == OK and n.value == 0
    assert lib.rar_norm_workspace(ctypes.byref(_config()), ctypes.byref(n)) == OK and n.value >= 2 * 16 * 4
    assert lib.rar_norm_workspace(ctypes.byref(_config()), None) == BAD
    assert lib.rar_norm_workspace(None, ctypes.byref(n)) == BAD
    assert lib.rar_norm_workspace(ctypes.byref(_config(eps=0.0)), ctypes.byref(n)) == BAD


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_the_norms_structure_is_the_headers():
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "rar.h"', "int main(void) {", '  printf("%zu\\n", sizeof(rar_norm_t));']
    lines += [f'  printf("%zu\\n", offsetof(rar_norm_t, {f}));' for f, _ in _lib.Norm._fields_]
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with tempfile.TemporaryDirectory() as tmp:
        src, exe = os.path.join(tmp, "l.c"), os.path.join(tmp, "l")
        open(src, "w").write("\n".join(lines + ["  return 0;", "}"]) + "\n")
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), src, "-o", exe], check=True)
        got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == [ctypes.sizeof(_lib.Norm)] + [getattr(_lib.Norm, f).offset for f, _ in _lib.Norm._fields_]


def _quantize(xs=(A, A + M), widths=(64, 32), xstrides=None, n=2, rows=4, dtype=F32, q=(A + 2 * M, A + 3 * M), qstrides=None, scales=A + 4 * M):
    return _lib.load().rar_quantize_rows(_p(xs), _l(widths), _l(xstrides), n, rows, dtype, _p(q), _l(qstrides), scales, None)


def test_quantize_refusals():
    assert _quantize(rows=0, xs=None, q=None, scales=None) == OK
    bad = [
        (dict(n=0), "no rank"), (dict(n=65), "65 ranks"), (dict(widths=None), "widths"), (dict(widths=(-1, 32)), "width"), (dict(widths=(131071, 1)), "widths"),
        (dict(widths=(1 << 62, 1 << 62)), "widths overflow"), (dict(rows=-1), "rows"), (dict(rows=(1 << 24) + 1), "rows"), (dict(dtype=I32), "int32"), (dict(xs=None), "NULL"),
        (dict(q=None), "NULL"), (dict(xs=(A, 0)), "NULL input"), (dict(q=(0, A)), "NULL output"), (dict(scales=None), "no scales"), (dict(scales=A + 4 * M + 2), "misaligned"),
        (dict(xs=(A + 2, A + M)), "misaligned"), (dict(xstrides=(63, 32)), "stride"), (dict(qstrides=(63, 32)), "stride"), (dict(qstrides=(1 << 60, 32)), "far stride"),
        (dict(q=(A, A + 3 * M)), "over an input"), (dict(q=(A + 2 * M, A + 2 * M + 5)), "outputs overlap"), (dict(scales=A + 4), "scales over an input"),
        (dict(scales=A + 2 * M), "scales over an output"),
    ]
    for kw, why in bad:
        assert _quantize(**kw) == BAD, why
        assert _message(), why


def _project(xs=(A, A + M), widths=(64, 32), xstrides=None, sx=A + 2 * M, ws=(A + 3 * M, A + 4 * M), wstrides=None, sw=A + 5 * M, n=2, tokens=4, outer=40, dtype=F32,
             res=None, res_stride=0, recvs=(A + 6 * M,), rstrides=None, copies=1, work=A + 7 * M, work_bytes=1 << 30):
    return _lib.load().rar_int8_projection_allreduce(_p(xs), _l(widths), _l(xstrides), sx, _p(ws), _l(wstrides), sw, n, tokens, outer, dtype, res, res_stride, _p(recvs),
                                                     _l(rstrides), copies, work, work_bytes, None)


def test_projection_refusals():
    assert _project(tokens=0, xs=None, ws=None, recvs=None, sx=None, sw=None, work=None, work_bytes=0) == OK
    bad = [
        (dict(n=0), "no rank"), (dict(n=65), "65 ranks"), (dict(copies=0), "no output"), (dict(copies=65), "65 outputs"), (dict(widths=None), "widths"),
        (dict(widths=(-1, 32)), "width"), (dict(widths=(131071, 1)), "widths"), (dict(tokens=-1), "tokens"), (dict(tokens=(1 << 24) + 1), "tokens"), (dict(outer=0), "outer"),
        (dict(outer=(1 << 24) + 1), "outer"), (dict(dtype=I32), "int32"), (dict(xs=None), "NULL"), (dict(ws=None), "NULL"), (dict(recvs=None), "NULL"),
        (dict(xs=(A, 0)), "NULL input"), (dict(ws=(0, A)), "NULL weight"), (dict(recvs=(0,)), "NULL output"), (dict(sx=None), "no scales"), (dict(sw=None), "no scales"),
        (dict(sx=A + 2 * M + 2), "misaligned"), (dict(sw=A + 5 * M + 1), "misaligned"), (dict(recvs=(A + 6 * M + 2,)), "misaligned"), (dict(res=A + 8 * M + 2), "misaligned"),
        (dict(xstrides=(63, 32)), "stride"), (dict(wstrides=(63, 32)), "stride"), (dict(rstrides=(39,)), "stride"), (dict(res=A + 8 * M, res_stride=39), "stride"),
        (dict(wstrides=(1 << 60, 32)), "far stride"), (dict(recvs=(A,)), "over an input"), (dict(recvs=(A + 3 * M,)), "over a weight"), (dict(recvs=(A + 5 * M,)), "over scales"),
        (dict(recvs=(A + 6 * M, A + 6 * M + 8), copies=2), "outputs overlap"), (dict(res=A + 6 * M + 8), "in part over the residual"),
        (dict(tokens=1 << 24, outer=1 << 24), "too large"),
        (dict(tokens=100, xs=(A + 1, A + M), work=None), "no workspace for rows to be laid out"), (dict(tokens=100, wstrides=(65, 32), work=None), "no workspace"),
        (dict(tokens=100, xs=(A + 1, A + M), work_bytes=100 * 64), "workspace too small"), (dict(tokens=100, xs=(A + 1, A + M), work=A + 7 * M + 8), "misaligned workspace"),
        (dict(tokens=100, xs=(A + 1, A + M), work=A + 3 * M), "workspace over a weight"), (dict(tokens=100, xs=(A + 1, A + M), work=A + 6 * M), "workspace over an output"),
        (dict(tokens=100, widths=(65536, 32), work=None, n=1), "no workspace for parts of the sums"),
    ]
    for kw, why in bad:
        assert _project(**kw) == BAD, why
        assert _message(), why


def test_projection_workspace():
    lib, n = _lib.load(), ctypes.c_size_t()
    assert lib.rar_int8_projection_workspace(_l([64]), 1, 5, 64, BF16, 1, ctypes.byref(n)) == OK
    assert lib.rar_int8_projection_workspace(_l([64]), 1, 5, 64, BF16, 1, None) == BAD
    assert lib.rar_int8_projection_workspace(None, 1, 5, 64, BF16, 1, ctypes.byref(n)) == BAD
    assert lib.rar_int8_projection_workspace(_l([64]), 1, 5, 0, BF16, 1, ctypes.byref(n)) == BAD
    # rows to be laid out need room, and so do parts of the sums
    sizes = {}
    for aligned in (0, 1):
        assert lib.rar_int8_projection_workspace(_l([6400]), 1, 100, 640, BF16, aligned, ctypes.byref(n)) == OK
        sizes[aligned] = n.value
    assert sizes[0] >= sizes[1] + 740 * 6400 and sizes[1] > 0
    assert lib.rar_int8_projection_workspace(_l([64]), 1, 5, 64, I32, 1, ctypes.byref(n)) == BAD


def test_the_binding_refuses_host_tensors_and_shapes():
    x, ids = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="device"):
        rar.embedding_allreduce([x], ids, [x])
    with pytest.raises(ValueError, match="device"):
        rar.embedding_allreduce_backward([x], ids, [x])
    with pytest.raises(ValueError, match="device"):
        rar.norm_allreduce([x], [x], [])
    with pytest.raises(ValueError, match="device"):
        rar.norm_allreduce_backward([x], [], [x])
    with pytest.raises(ValueError, match="list"):
        rar.norm_allreduce_backward([], [], [x])
    with pytest.raises(ValueError, match="device"):
        rar.quantize_rows([x])
    with pytest.raises(ValueError, match="device"):
        rar.int8_projection_allreduce([x.to(torch.int8)], torch.zeros(2), [x.to(torch.int8)], torch.zeros(2), [torch.zeros(2, 2)])
    for call in (lambda t: rar.embedding_allreduce([t], ids, [t]), lambda t: rar.norm_allreduce([t], [t], []), lambda t: rar.quantize_rows([t])):
        with pytest.raises(TypeError, match="dtype"):
            call(x.half())
    with pytest.raises(ValueError, match="list"):
        rar.quantize_rows(x)


# ---- the oracle ----

def test_the_oracles_gradient_of_the_norms_is_torchs():
    r = np.random.default_rng(0)
    rows, width, groups, eps = 6, 17, 3, float(np.float32(1e-5))
    s, h = r.standard_normal((rows, width)), r.standard_normal((rows, width))
    gh, go = [r.standard_normal((rows, width)) for _ in range(2)], [r.standard_normal((rows, width)) for _ in range(3)]
    post, pre, gate = 1 + 0.1 * r.standard_normal(width), 1 + 0.1 * r.standard_normal(width), r.standard_normal((groups, width))
    got = oracle.norms_backward(gh, go, s, h, 0.5, post, gate, pre, 1e-5, "float32")

    def leaf(a):
        return torch.tensor(a, requires_grad=True)

    def rms(x):
        return x / torch.sqrt((x * x).mean(1, keepdim=True) + eps)
    ts, th, tpost, tpre, tgate, res = leaf(s), leaf(h), leaf(post), leaf(pre), leaf(gate), leaf(np.zeros((rows, width)))
    dh, dpre = torch.autograd.grad(rms(th) * tpre, (th, tpre), torch.tensor(sum(go)))
    y = 0.5 * res + tgate.repeat_interleave(2, 0) * (rms(ts) * tpost)
    want = dict(zip(("dpartial", "dresidual", "dpost", "dgate"), torch.autograd.grad(y, (ts, res, tpost, tgate), torch.tensor(sum(gh)) + dh)), dpre=dpre)
    for k, v in want.items():
        assert np.abs(got[k][0] - v.numpy()).max() < 1e-13, k
        assert (got[k][1] < 1e-3).all(), k


def test_the_oracles_embedding_gradient_is_torchs():
    r = np.random.default_rng(1)
    ids = np.array([3, -1, 0, 3, 9, 3, 10])
    grads = [r.standard_normal((7, 5)) for _ in range(2)]
    got, _ = oracle.embedding_backward(grads, ids, 10, 0.25, "float32")
    table = torch.zeros(10, 5, dtype=torch.float64, requires_grad=True)
    there = torch.tensor([0, 2, 3, 4, 5])
    y = 0.25 * table[torch.tensor(ids)[there]]
    want, = torch.autograd.grad(y, table, torch.tensor(sum(grads))[there])
    assert np.abs(got - want.numpy()).max() < 1e-14
