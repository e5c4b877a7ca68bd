"""The AllReduce with dropout and a residual, and its gradient, against the
definition in 64 bits."""
import numpy as np
import pytest

from oracle import model_ops

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "bfloat16"]
SEED, OFFSET = 0x9E3779B97F4A7C15, 0x123456789ABCDEF0


def _torch_dtype(dtype):
    import torch
    return getattr(torch, dtype)


def _rng(seed=SEED, offset=OFFSET):
    import torch
    return torch.from_numpy(np.array([seed, offset], dtype=np.uint64).view(np.int64)).cuda()


def _values(shape, dtype, seed):
    """Device tensors of the payload type and their exact values."""
    import torch
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32))
    x = x.to(_torch_dtype(dtype))
    return [t.cuda() for t in x], x.double().numpy()


def _check(got, want, bound, what):
    off = np.abs(got.double().cpu().numpy() - want)
    assert (off <= bound).all(), f"{what}: {np.max(off - bound)} over its bound"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ranks,copies,count", [(1, 1, 1), (1, 1, 7), (2, 1, 8), (4, 4, 9), (3, 2, 2047),
                                                (5, 5, 4099), (8, 8, 65), (64, 64, 33), (9, 1, 20003)])
def test_forward(dtype, ranks, copies, count):
    import torch
    import ring_all_reduce_channelmask_amd as rar
    for p, with_residual in ((0.1, True), (0.5, False)):
        sends, x = _values((ranks, count), dtype, count)
        res, r = _values((1, count), dtype, count + 1)
        outs = [torch.full_like(sends[0], float("nan")) for _ in range(copies)]
        rar.dropout_allreduce(sends, outs, p, _rng(), call=3, residual=res[0] if with_residual else None)
        factor = model_ops.keep_factor(SEED, OFFSET + 3, count, p)
        want, bound = model_ops.dropout(x, r[0] if with_residual else None, factor, dtype)
        for k in range(copies):
            _check(outs[k], want, bound, f"copy {k}, p {p}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ranks,copies,count", [(1, 1, 5), (4, 1, 777), (4, 4, 4096), (2, 3, 20001)])
def test_backward_formula(dtype, ranks, copies, count):
    import torch
    import ring_all_reduce_channelmask_amd as rar
    grads, dy = _values((copies, count), dtype, count)
    dsends = [torch.full_like(grads[0], float("nan")) for _ in range(ranks)]
    dres = torch.full_like(grads[0], float("nan"))
    rar.dropout_allreduce_backward(grads, dsends, 0.25, _rng(), dresidual=dres)
    factor = model_ops.keep_factor(SEED, OFFSET, count, 0.25)
    want, bound = model_ops.dropout(dy, None, factor, dtype)
    for r in range(ranks):
        _check(dsends[r], want, bound, f"rank {r}")
    want, bound = model_ops.dropout(dy, None, np.ones(count), dtype)
    _check(dres, want, bound, "residual")


def test_backward_differences():
    """With whole numbers and p = 1/2 (factor 2) fp32 is exact: the change of
    the output with an input is the gradient exactly."""
    import torch
    import ring_all_reduce_channelmask_amd as rar
    n = 1003
    x = [torch.from_numpy(np.random.default_rng(r).integers(-50, 50, n).astype(np.float32)).cuda() for r in range(3)]
    res = torch.ones(n, device="cuda")
    y0, y1 = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    rar.dropout_allreduce(x, [y0], 0.5, _rng(), residual=res)
    rar.dropout_allreduce([x[0], x[1] + 1, x[2]], [y1], 0.5, _rng(), residual=res)
    dx = [torch.empty(n, device="cuda") for _ in range(3)]
    rar.dropout_allreduce_backward([torch.ones(n, device="cuda")], dx, 0.5, _rng())
    assert torch.equal(y1 - y0, dx[1]) and torch.equal(dx[0], dx[1])
    assert set(dx[1].unique().tolist()) == {0.0, 2.0}
    rar.dropout_allreduce(x, [y1], 0.5, _rng(), residual=res + 1)
    dres = torch.empty(n, device="cuda")
    rar.dropout_allreduce_backward([torch.ones(n, device="cuda")], dx, 0.5, _rng(), dresidual=dres)
    assert torch.equal(y1 - y0, dres)


@pytest.mark.parametrize("p", [0.0, 1.0, 1e-9, 2.0 ** -16, 1 - 2.0 ** -16])
def test_edge_probabilities(p):
    import torch
    import ring_all_reduce_channelmask_amd as rar
    n = 5000
    sends, x = _values((2, n), "float32", 5)
    out = torch.empty(n, device="cuda")
    rar.dropout_allreduce(sends, [out], p, _rng())
    want, bound = model_ops.dropout(x, None, model_ops.keep_factor(SEED, OFFSET, n, p), "float32")
    _check(out, want, bound, f"p {p}")


def test_dropped_elements_are_zero_whatever_they_were():
    import torch
    import ring_all_reduce_channelmask_amd as rar
    n = 4000
    x = torch.full((n,), float("inf"), device="cuda")
    x[1::2] = float("nan")
    out = torch.empty(n, device="cuda")
    rar.dropout_allreduce([x], [out], 0.5, _rng())
    kept = torch.from_numpy(model_ops.keep_factor(SEED, OFFSET, n, 0.5) > 0).cuda()
    assert (out[~kept] == 0).all() and not torch.isfinite(out[kept]).any()


def test_the_share_kept_and_its_independence():
    """The mask is that of the elements alone: the same for both types and any
    number of ranks, another for another call; 4 sigma for its share."""
    import torch
    import ring_all_reduce_channelmask_amd as rar
    n = 1 << 20
    masks = []
    for dtype, ranks, call in (("float32", 1, 0), ("bfloat16", 4, 0), ("float32", 1, 1)):
        x = [torch.ones(n, dtype=_torch_dtype(dtype), device="cuda") for _ in range(ranks)]
        out = torch.empty_like(x[0])
        rar.dropout_allreduce(x, [out], 0.1, _rng(), call=call)
        masks.append(out != 0)
    assert torch.equal(masks[0], masks[1])
    cut = round(0.1 * 65536) / 65536
    share = masks[0].double().mean().item()
    assert abs(share - (1 - cut)) < 4 * (cut * (1 - cut) / n) ** 0.5
    both = (masks[0] & masks[2]).double().mean().item()
    q = (1 - cut) ** 2
    assert abs(both - q) < 4 * (q * (1 - q) / n) ** 0.5


@pytest.mark.parametrize("dtype", DTYPES)
def test_in_place_and_misaligned(dtype):
    import torch
    import ring_all_reduce_channelmask_amd as rar
    n = 3001
    sends, x = _values((3, n + 3), dtype, 8)
    views = [s[k:k + n] for k, s in enumerate(sends)]
    x = np.stack([x[k, k:k + n] for k in range(3)])
    before = [s.clone() for s in sends]
    res = sends[2].clone()[1:1 + n]
    want, bound = model_ops.dropout(x, res.double().cpu().numpy(), model_ops.keep_factor(SEED, OFFSET, n, 0.1), dtype)
    rar.dropout_allreduce(views, [views[0], res, views[2]], 0.1, _rng(), residual=res)
    for k, v in enumerate((views[0], res, views[2])):
        _check(v, want, bound, f"copy {k}")
    for k in (0, 2):  # nothing outside the views is written
        assert torch.equal(sends[k][:k], before[k][:k]) and torch.equal(sends[k][k + n:], before[k][k + n:])
    assert torch.equal(sends[1], before[1])


def test_offset_carries_into_its_high_word():
    import torch
    import ring_all_reduce_channelmask_amd as rar
    n = 64
    out = torch.empty(n, device="cuda")
    rar.dropout_allreduce([torch.ones(n, device="cuda")], [out], 0.5, _rng(7, 0xFFFFFFFF), call=1)
    want = model_ops.keep_factor(7, 1 << 32, n, 0.5)
    assert np.array_equal(out.cpu().numpy(), want.astype(np.float32))


def test_more_than_2_31_elements():
    """Indexes beyond 32 bits, of elements and of bytes."""
    import torch
    import ring_all_reduce_channelmask_amd as rar
    n, tail = (1 << 31) + 1029, 1029
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    x[-tail:] = torch.arange(tail, device="cuda") % 100 + 1
    out = torch.empty_like(x)
    rar.dropout_allreduce([x], [out], 0.5, _rng())
    factor = (model_ops.philox_fields(SEED, OFFSET, tail, start=1 << 31) >= 32768) * 2.0
    assert np.array_equal(out[-tail:].double().cpu().numpy(), factor * (np.arange(tail) % 100 + 1))
    first = model_ops.keep_factor(SEED, OFFSET, 1024, 0.5)
    assert np.array_equal(out[:1024].double().cpu().numpy(), first)
    share = (out[:1 << 30] != 0).double().mean().item()
    assert abs(share - 0.5) < 4 * 0.5 / (1 << 15)


def test_streams_and_graph_replays():
    import torch
    import ring_all_reduce_channelmask_amd as rar
    n = 30001
    sends, x = _values((4, n), "float32", 9)
    out, rng = torch.empty(n, device="cuda"), _rng()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rar.dropout_allreduce(sends, [out], 0.1, rng, stream=side)
    side.synchronize()
    want, bound = model_ops.dropout(x, None, model_ops.keep_factor(SEED, OFFSET, n, 0.1), "float32")
    _check(out, want, bound, "side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rar.dropout_allreduce(sends, [out], 0.1, rng)
    for step in range(3):
        rng.copy_(_rng(SEED, OFFSET + step))
        out.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, bound = model_ops.dropout(x, None, model_ops.keep_factor(SEED, OFFSET + step, n, 0.1), "float32")
        _check(out, want, bound, f"replay {step}")
        eager = torch.empty(n, device="cuda")
        rar.dropout_allreduce(sends, [eager], 0.1, rng)
        torch.cuda.synchronize()
        assert torch.equal(eager, out)


def test_empty():
    import torch
    import ring_all_reduce_channelmask_amd as rar
    e = torch.empty(0, device="cuda")
    rar.dropout_allreduce([e], [e.clone()], 0.1, _rng())
    rar.dropout_allreduce_backward([e], [e.clone()], 0.1, _rng())
