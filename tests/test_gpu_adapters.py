"""The AllReduce of a row-parallel projection with low-rank adapters, against
the definition in 64 bits."""
import numpy as np
import pytest

from oracle import model_ops

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "bfloat16"]


def _tensor(a, dtype, pad=0, skip=0):
    """A device tensor (rows widened by pad, starting skip elements into its
    buffer) and its exact values."""
    import torch
    t = torch.from_numpy(np.asarray(a, dtype=np.float32)).to(getattr(torch, dtype))
    if pad or skip:
        held = torch.full((t.shape[0] * (t.shape[1] + pad) + skip,), float("nan"), dtype=t.dtype, device="cuda")
        view = held[skip:].view(t.shape[0], t.shape[1] + pad)[:, :t.shape[1]]
        view.copy_(t)
        return view, t.double().numpy()
    return t.cuda(), t.double().numpy()


def _case(dtype, tokens, widths, outer, rank, adapters, ids, seed=0, pad=0, skip=0):
    import torch
    r = np.random.default_rng(seed)
    inner = max(1, sum(widths))
    xs = [_tensor(r.standard_normal((tokens, w)), dtype, pad, skip) for w in widths]
    ps = [_tensor(r.standard_normal((tokens, outer)), dtype, pad, skip) for _ in widths]
    ds = [_tensor(r.standard_normal((adapters, rank, w)) / inner ** 0.5, dtype) for w in widths]
    up = _tensor(r.standard_normal((adapters, outer, rank)) / rank ** 0.5, dtype)
    scales = (0.5 + r.random(adapters)).astype(np.float32)
    dev = dict(xs=[x[0] for x in xs], partials=[p[0] for p in ps], downs=[d[0] for d in ds], up=up[0],
               ids=torch.tensor(list(ids), dtype=torch.int64, device="cuda"), scales=torch.from_numpy(scales).cuda())
    want = model_ops.adapters([x[1] for x in xs], np.stack([p[1] for p in ps]), [d[1] for d in ds], up[1], list(ids),
                              scales.astype(float), dtype)
    return dev, want


def _run(dev, copies=1, recvs=None):
    import torch
    import ring_all_reduce_channelmask_amd as rar
    if recvs is None:
        recvs = [torch.full(dev["partials"][0].shape, float("nan"), dtype=dev["up"].dtype, device="cuda")
                 for _ in range(copies)]
    rar.adapter_allreduce(dev["xs"], dev["partials"], recvs, dev["downs"], dev["up"], dev["ids"], dev["scales"])
    return recvs


def _check(got, want, what=""):
    y, bound = want
    off = np.abs(got.double().cpu().numpy() - y) - bound
    assert (off <= 0).all(), f"{what}: {np.nanmax(off)} over its bound"


CASES = [
    # tokens, widths, outer, rank, adapters
    (1, [1], 1, 1, 1),
    (1, [64, 64], 64, 16, 3),
    (1, [1792] * 4, 300, 16, 2),
    (2, [0, 5], 17, 3, 2),
    (15, [33, 31, 1], 65, 8, 4),
    (16, [512], 256, 16, 1),
    (17, [257, 255], 129, 12, 5),
    (40, [100] * 8, 333, 32, 40),
    (33, [640, 640], 320, 64, 3),
    (48, [301], 200, 128, 2),
    (20, [129, 130], 77, 100, 6),
    (300, [513, 511], 140, 16, 9),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,widths,outer,rank,adapters", CASES, ids=[f"t{c[0]}-i{sum(c[1])}-o{c[2]}-r{c[3]}-a{c[4]}" for c in CASES])
def test_forward(dtype, tokens, widths, outer, rank, adapters):
    r = np.random.default_rng(tokens)
    spread = r.integers(-1, adapters, tokens)                  # any order, some without
    runs = np.sort(r.integers(0, adapters, tokens))            # requests' tokens together
    for k, ids in enumerate((spread, runs)):
        dev, want = _case(dtype, tokens, widths, outer, rank, adapters, ids, tokens + k)
        for y in _run(dev, copies=1 + k):
            _check(y, want, f"ids {k}")


# tokens * rank over 16384: the tokens go 16 at a time
TILED = [
    (150, [70, 61], 300, 128, 5),
    (257, [129], 257, 64, 4),
    (263, [33, 0, 100], 5, 65, 3),
    (300, [64] * 5, 1025, 100, 30),
    (529, [40, 41], 516, 32, 3),
    (700, [17], 63, 33, 200),
    (1100, [130, 126], 777, 16, 6),
    (2100, [31], 40, 9, 4),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,widths,outer,rank,adapters", TILED, ids=[f"t{c[0]}-i{sum(c[1])}-o{c[2]}-r{c[3]}-a{c[4]}" for c in TILED])
def test_tiles_of_tokens(dtype, tokens, widths, outer, rank, adapters):
    r = np.random.default_rng(tokens)
    spread = r.integers(-1, adapters, tokens)
    runs = np.sort(r.integers(-1, adapters, tokens))
    for k, ids in enumerate((spread, runs)):
        dev, want = _case(dtype, tokens, widths, outer, rank, adapters, ids, tokens + k, pad=3 * k, skip=k)
        for y in _run(dev, copies=1 + 2 * k):
            _check(y, want, f"ids {k}")


@pytest.mark.parametrize("dtype", DTYPES)
def test_tiles_with_more_than_four_ranks_in_place(dtype):
    ids = np.arange(700) // 50 % 5 - 1
    dev, want = _case(dtype, 700, [20, 21, 22, 23, 24, 25, 26], 333, 32, 4, ids, 11, pad=1, skip=1)
    got = _run(dev, recvs=[dev["partials"][6], dev["partials"][2]])
    for y in got:
        _check(y, want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_tiles_keep_a_broken_adapter_apart(dtype):
    import torch
    tokens = 600
    ids = [i % 4 for i in range(tokens)]
    dev, want = _case(dtype, tokens, [200, 100], 330, 32, 4, ids, 6)
    dev["downs"][0][1, 3, 7] = float("nan")
    dev["up"][2, 5, 2] = float("inf")
    dev["xs"][0][12, :] = float("inf")
    got = _run(dev)[0]
    clean = [t for t in range(tokens) if ids[t] in (0, 3) and t != 12]
    y, bound = want
    _check(got[clean], (y[clean], bound[clean]))
    assert not torch.isfinite(got[[1, 2]]).all(dim=1).any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_tokens(dtype):
    """Enough token tiles that workgroups take several in turn."""
    tokens, adapters = 2100, 6
    ids = np.repeat(np.arange(7) - 1, 300)
    dev, want = _case(dtype, tokens, [260, 252], 1100, 16, adapters, ids, 3)
    _check(_run(dev)[0], want)
    ids = np.random.default_rng(1).integers(0, adapters, tokens)
    dev, want = _case(dtype, tokens, [260, 252], 1100, 16, adapters, ids, 4)
    _check(_run(dev)[0], want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_ids_outside_mean_no_adapter(dtype):
    import torch
    ids = [-1, 3, 1 << 40, -(1 << 62), 2]
    dev, want = _case(dtype, 5, [40], 30, 4, 3, ids)
    got = _run(dev)[0]
    _check(got, want)
    assert torch.equal(got[:4], dev["partials"][0][:4])
    dev, want = _case(dtype, 37, [40, 41], 30, 4, 3, [-1] * 37)
    _check(_run(dev)[0], want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_alignment_and_in_place(dtype):
    for pad, skip in ((1, 0), (3, 1), (8, 5)):
        dev, want = _case(dtype, 19, [101, 99], 147, 16, 4, [i % 5 - 1 for i in range(19)], pad, pad=pad, skip=skip)
        got = _run(dev, recvs=[dev["partials"][1]])
        _check(got[0], want, f"pad {pad} skip {skip}")
        if pad:
            whole = got[0].as_strided((19, 147 + pad), (147 + pad, 1))[:, 147:]
            assert whole[:-1].isnan().all()  # nothing between the rows is written


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_broken_adapter_reaches_its_own_tokens_only(dtype):
    import torch
    for tokens in (20, 70):
        ids = [i % 4 for i in range(tokens)]
        dev, want = _case(dtype, tokens, [200, 100], 130, 16, 4, ids, 6)
        dev["downs"][0][1, 3, 7] = float("nan")
        dev["up"][2, 5, 2] = float("inf")
        dev["partials"][0][8, :] = float("nan")
        dev["xs"][0][12, :] = float("inf")
        got = _run(dev)[0]
        clean = [t for t in range(tokens) if ids[t] in (0, 3) and t not in (8, 12)]
        y, bound = want
        _check(got[clean], (y[clean], bound[clean]))
        assert not torch.isfinite(got[[1, 2]]).all(dim=1).any()


def test_without_scales_and_same_bits_on_repeats():
    import torch
    import ring_all_reduce_channelmask_amd as rar
    for dtype in DTYPES:
        dev, _ = _case(dtype, 50, [300, 300], 500, 16, 8, [i % 9 - 1 for i in range(50)], 7)
        dev["scales"].fill_(1.0)
        first = _run(dev)[0]
        out = torch.empty_like(first)
        for _ in range(10):
            rar.adapter_allreduce(dev["xs"], dev["partials"], [out], dev["downs"], dev["up"], dev["ids"])
            assert torch.equal(out, first)


def test_streams_and_graph_replays():
    import torch
    import ring_all_reduce_channelmask_amd as rar
    dev, _ = _case("bfloat16", 30, [300, 300], 500, 16, 8, [i % 9 - 1 for i in range(30)], 8)
    torch.cuda.synchronize()
    a = torch.empty_like(dev["partials"][0])
    b = torch.empty_like(a)
    args = (dev["downs"], dev["up"], dev["ids"], dev["scales"])
    side = torch.cuda.Stream()
    rar.adapter_allreduce(dev["xs"], dev["partials"], [a], *args, stream=side)
    side.synchronize()
    rar.adapter_allreduce(dev["xs"], dev["partials"], [b], *args)
    assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rar.adapter_allreduce(dev["xs"], dev["partials"], [a], *args)
    for step in range(3):
        for x in dev["xs"]:
            x.copy_(torch.randn(x.shape, device="cuda"))
        dev["ids"].copy_(torch.randint(-1, 8, (30,), device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        rar.adapter_allreduce(dev["xs"], dev["partials"], [b], *args)
        assert torch.equal(a, b), step


@pytest.mark.parametrize("dtype", DTYPES)
def test_ranks_without_columns(dtype):
    """No rank has a column of the input: the adapters add nothing."""
    import torch
    for tokens in (5, 600):
        dev, want = _case(dtype, tokens, [0, 0], 70, 16, 3, [t % 4 - 1 for t in range(tokens)], 9)
        _check(_run(dev)[0], want)


def test_more_than_2_31_elements_between_rows():
    """Row offsets beyond 32 bits in every strided operand, of few tokens and
    of tiles of them."""
    import torch
    import ring_all_reduce_channelmask_amd as rar
    for tokens, stride in ((40, 60_000_001), (600, 3_700_001)):
        dev, want = _case("bfloat16", tokens, [65, 64], 131, 16, 3, [t % 4 - 1 for t in range(tokens)], 10)
        held = torch.empty(tokens * stride, dtype=torch.bfloat16, device="cuda")
        assert held.numel() > 1 << 31
        column = 0

        def far(t):
            nonlocal column
            view = held.as_strided(t.shape, (stride, 1), column)
            column += t.shape[1] + 3
            return view.copy_(t)
        for k in ("xs", "partials"):
            dev[k] = [far(t) for t in dev[k]]
        out = held.as_strided((tokens, 131), (stride, 1), column)
        _check(_run(dev, recvs=[out])[0], want, f"{tokens} tokens")
        del held, out, dev


def test_no_tokens():
    import torch
    import ring_all_reduce_channelmask_amd as rar
    e = torch.empty((0, 8), device="cuda")
    rar.adapter_allreduce([e], [torch.empty((0, 4), device="cuda")], [torch.empty((0, 4), device="cuda")],
                          [torch.zeros((2, 3, 8), device="cuda")], torch.zeros((2, 4, 3), device="cuda"),
                          torch.empty(0, dtype=torch.int64, device="cuda"))
