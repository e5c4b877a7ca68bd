"""Log probabilities over a vocabulary split between the ranks, and their
gradient, against the definition in 64 bits."""
import numpy as np
import pytest

from oracle import model_ops

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "bfloat16"]
LOWEST = {"float32": float(np.finfo(np.float32).min), "bfloat16": -3.3895313892515355e38}


def _shards(x, widths, dtype, pad=0, skip=0):
    """Device shards of logits [rows, vocabulary] (row stride widened by pad,
    first element skip elements into its buffer), and their exact values."""
    import torch
    t = torch.from_numpy(np.asarray(x, dtype=np.float32)).to(getattr(torch, dtype))
    out, c = [], 0
    for w in widths:
        held = torch.full((t.shape[0] * (w + pad) + skip,), float("nan"), dtype=t.dtype, device="cuda")
        view = held[skip:].view(t.shape[0], w + pad)[:, :w]
        view.copy_(t[:, c:c + w])
        out.append(view)
        c += w
    assert c == t.shape[1]
    return out, t.double().numpy()


def _ids(ids):
    import torch
    return torch.tensor(list(ids), dtype=torch.int64, device="cuda")


def _close(got, want, bound, what):
    got = got.double().cpu().numpy()
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN at {np.argwhere(np.isnan(got) != np.isnan(want))[:4]}"
    rest = ~fine & ~np.isnan(want)
    assert np.array_equal(got[rest], want[rest]), f"{what}: infinities"
    off = np.abs(got[fine] - want[fine]) - np.broadcast_to(bound, want.shape)[fine]
    assert (off <= 0).all(), f"{what}: {off.max()} over its bound"


def _check(x, widths, dtype, ids, ntop=0, scale=1.0, pad=0, skip=0):
    import ring_all_reduce_channelmask_amd as rar
    shards, exact = _shards(x, widths, dtype, pad, skip)
    got = rar.logprobs(shards, _ids(ids), ntop=ntop, scale=scale)
    want = model_ops.logprobs(exact, ids, scale, ntop)
    for name in ("lse", "entropy", "logprob"):
        _close(getattr(got, name), want[name], want[name + "_bound"], name)
    if ntop:
        assert np.array_equal(got.top_ids.cpu().numpy(), want["top_ids"]), "top_ids"
        _close(got.top_logprobs, want["top_logprobs"], want["top_bound"], "top_logprobs")
    return shards, exact, got, want


def _normal(rows, vocab, seed, size=3.0):
    return np.random.default_rng(seed).standard_normal((rows, vocab)) * size


SHAPES = [(1, [1]), (1, [7]), (3, [5, 0, 9]), (2, [0, 1]), (5, [100, 100, 100, 83]), (1, [8191]), (2, [8192]), (2, [8193, 4097]),
          (17, [4095, 4096, 1]), (3, [20011, 19999]), (40, [3001] * 8), (2, [1] * 64)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,widths", SHAPES, ids=[f"{r}x{sum(w)}over{len(w)}" for r, w in SHAPES])
def test_forward(dtype, rows, widths):
    vocab = sum(widths)
    ids = [(i * 7919) % vocab for i in range(rows)]
    for ntop in (0, 1, 5, 32):
        _check(_normal(rows, vocab, rows + vocab), widths, dtype, ids, ntop, 0.7 if ntop == 5 else 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ntop", [0, 3, 32])
def test_many_rows_take_one_workgroup_each(dtype, ntop):
    """Over 1024 rows a row is not split: several tiles go through one workgroup."""
    rows, widths = 1030, [9001, 100, 4500]
    x = _normal(rows, sum(widths), 3)
    x[7] = np.sort(x[7])                         # every tile beats the one before
    x[8] = np.sort(x[8])[::-1]
    x[9] = 1.0                                   # all equal
    x[10] = np.arange(sum(widths)) % 3           # thousands of equal maxima
    x[11, :-3] = -np.inf                         # the last tile alone
    x[12, 5:] = -np.inf                          # the first tile alone
    x[13] = -np.inf
    x[14] = LOWEST[dtype]
    import ring_all_reduce_channelmask_amd as rar
    ids = [(i * 31) % sum(widths) for i in range(rows)]
    shards, exact = _shards(x, widths, dtype)
    got = rar.logprobs(shards, _ids(ids), ntop=ntop)
    rows_checked = list(range(16)) + [500, 1029]
    want = model_ops.logprobs(exact[rows_checked], [ids[i] for i in rows_checked], 1.0, ntop)
    for name in ("lse", "entropy", "logprob"):
        _close(getattr(got, name)[rows_checked], want[name], want[name + "_bound"], name)
    if ntop:
        assert np.array_equal(got.top_ids.cpu().numpy()[rows_checked], want["top_ids"])
        _close(got.top_logprobs[rows_checked], want["top_logprobs"], want["top_bound"], "top_logprobs")


@pytest.mark.parametrize("rows", [2, 60, 300, 600])
def test_every_cut_of_a_row(rows):
    """Few rows are split over workgroups; more take 16, 8 and 4 waves each.
    The first and last rows and the rows with many equal logits are checked."""
    import ring_all_reduce_channelmask_amd as rar
    widths = [33000, 1, 30011]
    x = np.random.default_rng(rows).standard_normal((rows, sum(widths))).astype(np.float32) * 3
    x[0] = np.floor(x[0])
    x[-1, 1000:] = -np.inf
    shards, exact = _shards(x, widths, "bfloat16")
    ids = [(i * 7919) % sum(widths) for i in range(rows)]
    at = sorted({0, 1, rows // 2, rows - 1})
    for ntop in (0, 1, 20, 32):
        got = rar.logprobs(shards, _ids(ids), ntop=ntop)
        want = model_ops.logprobs(exact[at], [ids[i] for i in at], 1.0, ntop)
        for name in ("lse", "entropy", "logprob"):
            _close(getattr(got, name)[at], want[name], want[name + "_bound"], name)
        assert np.array_equal(got.top_ids.cpu().numpy()[at], want["top_ids"])
        _close(got.top_logprobs[at], want["top_logprobs"], want["top_bound"], "top_logprobs")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ntop", [0, 2, 32])
def test_masks_infinities_and_nan(dtype, ntop):
    widths = [5000, 4000, 1001]
    vocab = sum(widths)
    x = _normal(14, vocab, 4)
    x[0] = -np.inf                               # nothing left
    x[1] = LOWEST[dtype]                         # masked by the lowest value: uniform
    x[2, :] = -np.inf
    x[2, 6000] = 2.0                             # one token left
    x[3, 1::2] = -np.inf
    x[4, 17] = np.nan
    x[5, 9000] = np.inf
    x[6] = np.nan
    x[7, :9999] = LOWEST[dtype]
    x[8] = 0.0
    x[8, ::3] = -0.0                             # equal to 0
    x[9, :5000] = -np.inf                        # a rank masked entirely
    x[10] = -1e30
    x[11] = 200.0
    x[11, 3] = -LOWEST[dtype]                    # the largest value
    x[12] = -np.inf
    x[12, -1] = LOWEST[dtype]
    ids = [0, 1, 6000, 2, 3, 9000, 5, 9999, 8, 9001, 10, 3, vocab - 1, 13]
    _check(x, widths, dtype, ids, ntop)
    _check(x[[0, 1, 2, 3, 7, 8, 9]], widths, dtype, [3] * 7, ntop, scale=0.5)


def test_ties_go_to_the_lowest_id():
    for dtype in DTYPES:
        x = np.zeros((4, 30000))
        x[1, ::1000] = 1.0
        x[2] = np.arange(30000) // 7 % 11
        x[3, 12345:12400] = 4.0
        _check(x, [10000, 1, 19999], dtype, [0, 1000, 2, 3], 32)


def test_rows_without_a_token():
    x = _normal(5, 300, 5)
    _check(x, [100, 200], "float32", [-1, 299, 300, 1 << 40, -(1 << 62)], 2)


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_and_alignment(dtype):
    for pad, skip in ((1, 0), (3, 1), (8, 5), (0, 3)):
        _check(_normal(6, 9007, pad + 9), [4503, 4504], dtype, range(6), 4, pad=pad, skip=skip)


def test_temperature_extremes():
    x = _normal(3, 500, 6)
    _check(x, [500], "float32", [1, 2, 3], 3, scale=30.0)
    _check(x, [500], "float32", [1, 2, 3], 3, scale=1e-6)


def test_same_bits_on_repeats_and_given_results():
    import torch
    import ring_all_reduce_channelmask_amd as rar
    shards, _ = _shards(_normal(9, 40000, 7), [10000] * 4, "bfloat16")
    ids = _ids(range(9))
    first = rar.logprobs(shards, ids, ntop=8)
    held = rar.LogProbs(*[torch.empty_like(t) for t in first])
    for _ in range(20):
        assert rar.logprobs(shards, ids, ntop=8, out=held) is held
        assert all(torch.equal(a, b) for a, b in zip(first, held))


def _grad_case(x, widths, dtype, ids, scale, seed, with_h=True, with_l=True, **kw):
    import torch
    import ring_all_reduce_channelmask_amd as rar
    shards, exact = _shards(x, widths, dtype, **kw)
    rows = len(ids)
    fwd = rar.logprobs(shards, _ids(ids), scale=scale)
    r = np.random.default_rng(seed)
    g, h, l = (r.standard_normal(rows).astype(np.float32) for _ in range(3))
    dev = [torch.from_numpy(v).cuda() for v in (g, h, l)]
    grads = rar.logprobs_backward(shards, _ids(ids), fwd.lse, fwd.entropy, dev[0], dev[1] if with_h else None,
                                  dev[2] if with_l else None, scale=scale)
    want, bound = model_ops.logprobs_backward(exact, ids, fwd.lse.double().cpu().numpy(), fwd.entropy.double().cpu().numpy(),
                                              g.astype(float), h.astype(float) * with_h, l.astype(float) * with_l, scale, dtype)
    got = torch.cat([t.double() for t in grads], 1).cpu().numpy()
    _close(torch.from_numpy(got), want, bound, "gradient")
    return shards, exact, fwd, (g, h, l), got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,widths", [(1, [1]), (3, [5, 0, 9]), (4, [8191, 8193]), (2, [4097, 1]), (33, [301] * 8)])
def test_backward_formula(dtype, rows, widths):
    vocab = sum(widths)
    ids = [(i * 7919) % vocab for i in range(rows)]
    if rows > 2:
        ids[1] = -1
    for k, (h, l) in enumerate(((True, True), (False, False), (True, False))):
        _grad_case(_normal(rows, vocab, k), widths, dtype, ids, 1.3, k, h, l, pad=k, skip=k)


@pytest.mark.parametrize("dtype", DTYPES)
def test_backward_masks(dtype):
    x = _normal(5, 3000, 12)
    x[0] = -np.inf
    x[1, ::2] = -np.inf
    x[2, 1:] = -np.inf
    x[3, 5:] = LOWEST[dtype]
    _, _, _, _, got = _grad_case(x, [1000, 2000], dtype, [0, 1, 0, 2, 4], 1.0, 3)
    assert (got[0] == 0).all() and (got[1, ::2] == 0).all()


def test_backward_differences():
    """Central differences of the definition in 64 bits: step 1e-4, whose
    third-order term stays under 1e-7 for logits of this size."""
    x = _normal(3, 200, 14, 1.0)
    ids, scale = [3, 150, -1], 1.3
    _, exact, _, (g, h, l), got = _grad_case(x, [70, 130], "float32", ids, scale, 5)

    def total(z):
        o = model_ops.logprobs(z, ids, scale, 0)
        return float((g * o["logprob"] + h * o["entropy"] + l * o["lse"]).sum())
    for i, j in ((0, 3), (0, 100), (1, 150), (1, 0), (2, 42), (2, 199)):
        up, down = exact.copy(), exact.copy()
        up[i, j] += 1e-4
        down[i, j] -= 1e-4
        assert abs((total(up) - total(down)) / 2e-4 - got[i, j]) < 2e-6


@pytest.mark.parametrize("dtype", DTYPES)
def test_backward_in_place_and_into_columns_of_one_tensor(dtype):
    import torch
    import ring_all_reduce_channelmask_amd as rar
    shards, _ = _shards(_normal(7, 5000, 15), [2500, 2500], dtype)
    ids = _ids(range(7))
    f = rar.logprobs(shards, ids)
    g = torch.ones(7, device="cuda")
    apart = rar.logprobs_backward(shards, ids, f.lse, None, g)
    whole = torch.empty((7, 5000), dtype=shards[0].dtype, device="cuda")
    rar.logprobs_backward(shards, ids, f.lse, None, g, grads=[whole[:, :2500], whole[:, 2500:]])
    rar.logprobs_backward(shards, ids, f.lse, None, g, grads=shards)
    for a, b, c in zip(apart, (whole[:, :2500], whole[:, 2500:]), shards):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_streams_and_graph_replays():
    import torch
    import ring_all_reduce_channelmask_amd as rar
    x = _normal(5, 40000, 16)
    shards, _ = _shards(x, [20000] * 2, "bfloat16")
    ids = _ids(range(5))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r = rar.logprobs(shards, ids, ntop=6, stream=side)
    grads = rar.logprobs_backward(shards, ids, r.lse, r.entropy, r.logprob, r.entropy, stream=side)
    side.synchronize()
    e = rar.logprobs(shards, ids, ntop=6)
    eg = rar.logprobs_backward(shards, ids, e.lse, e.entropy, e.logprob, e.entropy)
    assert all(torch.equal(a, b) for a, b in zip(list(r) + grads, list(e) + eg))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = rar.logprobs(shards, ids, ntop=6)
        cg = rar.logprobs_backward(shards, ids, c.lse, c.entropy, c.logprob, c.entropy)
    for step in range(3):
        for s in shards:
            s.copy_(torch.randn(s.shape, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        e = rar.logprobs(shards, ids, ntop=6)
        eg = rar.logprobs_backward(shards, ids, e.lse, e.entropy, e.logprob, e.entropy)
        assert all(torch.equal(a, b) for a, b in zip(list(c) + cg, list(e) + eg)), step


def test_more_than_2_31_logits():
    """Offsets beyond 32 bits in a shard, and gradients over them in place."""
    import torch
    import ring_all_reduce_channelmask_amd as rar
    rows, widths = 17000, [130003, 37]
    g = torch.Generator(device="cuda").manual_seed(3)
    shards = []
    for w in widths:
        t = torch.empty((rows, w), dtype=torch.bfloat16, device="cuda")
        for r0 in range(0, rows, 1000):
            t[r0:r0 + 1000] = torch.randn((1000, w), generator=g, device="cuda") * 3
        shards.append(t)
    assert shards[0].numel() > 1 << 31
    ids = torch.randint(0, sum(widths), (rows,), generator=g, device="cuda")
    at = [0, 8000, 16520, 16999]  # before and behind element 2^31 of the first shard
    exact = torch.cat([s[at].double() for s in shards], 1).cpu().numpy()
    own = ids[at].tolist()
    got = rar.logprobs(shards, ids, ntop=3)
    want = model_ops.logprobs(exact, own, 1.0, 3)
    for name in ("lse", "entropy", "logprob"):
        _close(getattr(got, name)[at], want[name], want[name + "_bound"], name)
    assert np.array_equal(got.top_ids[at].cpu().numpy(), want["top_ids"])
    ones = torch.ones(rows, device="cuda")
    rar.logprobs_backward(shards, ids, got.lse, None, ones, grads=shards)
    grad, bound = model_ops.logprobs_backward(exact, own, got.lse[at].double().cpu().numpy(), np.zeros(4), np.ones(4), np.zeros(4),
                                              np.zeros(4), 1.0, "bfloat16")
    _close(torch.cat([s[at] for s in shards], 1), grad, bound, "gradient")


def test_no_rows():
    import torch
    import ring_all_reduce_channelmask_amd as rar
    s = [torch.empty((0, 10), device="cuda")]
    r = rar.logprobs(s, _ids([]), ntop=3)
    assert r.top_ids.shape == (0, 3) and r.lse.shape == (0,)
    assert rar.logprobs_backward(s, _ids([]), r.lse, r.entropy, r.logprob)[0].shape == (0, 10)
