"""The norms around a block with its AllReduce, gate and residual scale, and
their gradient, against the definition in 64 bits."""
import numpy as np
import pytest

from oracle import model_ops

from .test_gpu_embedding import _tensor

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "bfloat16"]
EPS = 1e-5


def _check(got, want, what=""):
    y, bound = want
    off = np.abs(got.double().cpu().numpy().reshape(y.shape) - y) - bound
    assert (off <= 0).all(), f"{what}: {np.nanmax(off)} over its bound"


class Case:
    """Operands of both directions, on the device (.dev) and exactly (.val)."""

    def __init__(self, dtype, ranks, rows, width, groups=0, post=True, pre=True, residual=True, scale=0.75, pad=0, skip=0, seed=0, copies=1):
        r = np.random.default_rng(seed)
        self.dtype, self.rows, self.width, self.scale, self.copies = dtype, rows, width, scale, copies
        self.shape, self.pad, self.skip = (rows, width), pad, skip
        self.dev, self.val = {}, {}

        def put(k, a, **kw):
            self.dev[k], self.val[k] = _tensor(a, dtype, **kw)
        far = dict(pad=pad, skip=skip)
        several = {"partials": ranks, "grad_hidden": copies, "grad_outs": ranks if pre else 0}
        for k, n in several.items():
            got = [_tensor(r.standard_normal(self.shape), dtype, **far) for _ in range(n)]
            self.dev[k], self.val[k] = [g[0] for g in got], [g[1] for g in got]
        put("total", r.standard_normal(self.shape) * 1.5, **far)
        put("hidden", r.standard_normal(self.shape) * 2, **far)
        self.dev["residual"] = self.val["residual"] = None
        if residual:
            put("residual", r.standard_normal(self.shape) * 2, **far)
        for k, on in (("post", post), ("pre", pre)):
            self.dev[k] = self.val[k] = None
            if on:
                put(k, (1 + 0.3 * r.standard_normal((1, width))))
                self.dev[k], self.val[k] = self.dev[k].view(width), self.val[k][0]
        self.dev["gate"] = self.val["gate"] = None
        if groups:
            put("gate", 0.5 + r.standard_normal((groups, width)), **far)

    def empty(self, like=None):
        import torch
        if like is not None:
            return torch.full_like(like, float("nan"), memory_format=torch.contiguous_format)
        return _tensor(np.full(self.shape, np.nan), self.dtype, self.pad, self.skip)[0]

    def config(self):
        d = self.dev
        return dict(residual_scale=self.scale, post_weight=d["post"], gate=d["gate"], pre_weight=d["pre"], eps=EPS)

    def forward(self, copies=1, **kw):
        import ring_all_reduce_channelmask_amd as rar
        d = self.dev
        out = dict(hidden=[self.empty() for _ in range(copies)], outs=[self.empty() for _ in range(copies if d["pre"] is not None else 0)],
                   total=self.empty())
        out.update(kw)
        rar.norm_allreduce(d["partials"], out["hidden"], out["outs"], residual=d["residual"], total=out["total"], **self.config())
        return out

    def check_forward(self, out, what=""):
        v = self.val
        want = model_ops.norms(np.stack(v["partials"]), v["residual"], self.scale, v["post"], v["gate"], v["pre"], EPS, self.dtype)
        for y in out["hidden"]:
            _check(y, want["hidden"], what + " hidden")
        for y in out["outs"]:
            _check(y, want["out"], what + " out")
        if out["total"] is not None:
            _check(out["total"], want["total"], what + " total")

    def backward(self, copies=1, **kw):
        import ring_all_reduce_channelmask_amd as rar
        d = self.dev
        out = dict(dpartials=[self.empty() for _ in range(copies)], dresidual=self.empty())
        for k, of in (("dpost_weight", "post"), ("dgate", "gate"), ("dpre_weight", "pre")):
            out[k] = None if d[of] is None else self.empty(d[of])
        out.update(kw)
        rar.norm_allreduce_backward(d["grad_hidden"], d["grad_outs"], out["dpartials"], total=d["total"], hidden=d["hidden"],
                                    **{k: v for k, v in out.items() if k != "dpartials"}, **self.config())
        return out

    def check_backward(self, out, what=""):
        v = self.val
        want = model_ops.norms_backward(v["grad_hidden"], v["grad_outs"], v["total"], v["hidden"], self.scale, v["post"], v["gate"], v["pre"],
                                        EPS, self.dtype)
        for y in out["dpartials"]:
            _check(y, want["dpartial"], what + " dpartial")
        for k, of in (("dresidual", "dresidual"), ("dpost_weight", "dpost"), ("dgate", "dgate"), ("dpre_weight", "dpre")):
            if out[k] is not None:
                _check(out[k], want[of], what + " " + k)


# ranks, rows, width
CASES = [
    (1, 1, 1),
    (2, 3, 7),
    (3, 5, 64),
    (4, 1, 7168),
    (5, 9, 513),
    (8, 4, 1001),
    (2, 13, 2051),
    (4, 6, 4100),
    (1, 3, 8192),
    (3, 2, 8200),
    (2, 2, 16390),
    (2, 3, 32768),
]
IDS = [f"n{c[0]}-r{c[1]}-d{c[2]}" for c in CASES]
KINDS = [dict(), dict(groups=1), dict(post=False, groups=1), dict(post=False), dict(pre=False, groups=1), dict(residual=False, scale=1.0)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ranks,rows,width", CASES, ids=IDS)
def test_forward(dtype, ranks, rows, width):
    for k, kind in enumerate(KINDS + [dict(groups=rows)]):
        case = Case(dtype, ranks, rows, width, pad=3 * (k % 2), skip=k % 2, seed=k, **kind)
        case.check_forward(case.forward(copies=1 + k % 3), str(kind))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ranks,rows,width", CASES, ids=IDS)
def test_gradient(dtype, ranks, rows, width):
    for k, kind in enumerate(KINDS + [dict(groups=rows)]):
        case = Case(dtype, ranks, rows, width, pad=3 * (k % 2), skip=k % 2, seed=k, copies=1 + k % 2, **kind)
        case.check_backward(case.backward(copies=1 + k % 3), str(kind))


# rows, groups: groups of one row, of several workgroups, more groups than workgroups
ROWS = [(700, 1), (700, 2), (700, 7), (700, 350), (700, 700), (1300, 0), (1300, 650), (3000, 1), (3000, 600)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,groups", ROWS)
def test_many_rows(dtype, rows, groups):
    case = Case(dtype, 2, rows, 130, groups=groups, seed=rows)
    case.check_forward(case.forward())
    case.check_backward(case.backward())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,groups,width", [(5001, 5001, 130), (9000, 4500, 60), (1640, 820, 2100), (3003, 1001, 2051)])
def test_more_runs_of_rows_than_workgroups(dtype, rows, groups, width):
    """A workgroup takes several gates' rows in turn, odd numbers of them too."""
    case = Case(dtype, 2, rows, width, groups=groups, seed=rows)
    case.check_backward(case.backward())


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_gate_as_a_vector(dtype):
    case = Case(dtype, 2, 20, 300, groups=1)
    case.dev["gate"] = case.dev["gate"].view(300)
    case.check_forward(case.forward())
    case.check_backward(case.backward())


@pytest.mark.parametrize("dtype", DTYPES)
def test_single_outputs(dtype):
    """Each output alone: those not asked for change nothing."""
    import torch
    case = Case(dtype, 3, 21, 400, groups=3)
    whole = case.forward()
    assert torch.equal(case.forward(hidden=[])["outs"][0], whole["outs"][0])
    assert torch.equal(case.forward(outs=[], total=None)["hidden"][0], whole["hidden"][0])
    all_of = case.backward()
    names = ("dresidual", "dpost_weight", "dgate", "dpre_weight")
    for k in names:
        got = case.backward(dpartials=[], **{o: None for o in names if o != k})
        assert torch.equal(got[k], all_of[k]), k
    got = case.backward(**{o: None for o in names})
    assert torch.equal(got["dpartials"][0], all_of["dpartials"][0])


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradients_of_one_side(dtype):
    """Only hidden, or only outs, has a gradient."""
    case = Case(dtype, 2, 30, 222, groups=1)
    case.dev["grad_hidden"], case.val["grad_hidden"] = [], []
    case.check_backward(case.backward())
    case = Case(dtype, 2, 30, 222, groups=1)
    case.dev["grad_outs"], case.val["grad_outs"] = [], []
    out = case.backward(dpre_weight=None)
    case.check_backward(out)


@pytest.mark.parametrize("dtype", DTYPES)
def test_in_place(dtype):
    """Outputs over the inputs of the same elements."""
    for pad in (0, 5):
        case = Case(dtype, 3, 25, 515, groups=5, pad=pad, skip=pad)
        d = case.dev
        case.check_forward(case.forward(hidden=[d["residual"]], outs=[d["partials"][2], d["partials"][0]], total=d["partials"][1]), f"pad {pad}")
        case = Case(dtype, 3, 25, 515, groups=5, pad=pad, skip=pad)
        d = case.dev
        case.check_backward(case.backward(dpartials=[d["grad_outs"][1], d["total"], d["grad_hidden"][0]], dresidual=d["hidden"]), f"pad {pad}")


def test_gradient_against_differences():
    """In fp32: the change of the loss sum(grad * output) along a random
    direction.  A step of 2^-7 leaves an error of its square times the third
    derivative, and 2^-24 of the loss's terms over the step."""
    import torch
    import ring_all_reduce_channelmask_amd as rar
    case = Case("float32", 2, 6, 96, groups=3, scale=0.5)
    d = case.dev
    fwd = case.forward()
    d["total"], d["hidden"] = fwd["total"], fwd["hidden"][0]
    d["grad_outs"] = d["grad_outs"][:1]
    got = case.backward()

    def loss():
        out = case.forward()
        return (out["hidden"][0].double() * d["grad_hidden"][0].double()).sum().item() + (out["outs"][0].double() * d["grad_outs"][0].double()).sum().item()
    step = 2.0 ** -7
    for what, grad in ((d["partials"][0], got["dpartials"][0]), (d["residual"], got["dresidual"]), (d["post"], got["dpost_weight"]),
                       (d["gate"], got["dgate"]), (d["pre"], got["dpre_weight"])):
        way = torch.randn(what.shape, device="cuda").sign()
        kept = what.clone()
        what.copy_(kept + step * way)
        up = loss()
        what.copy_(kept - step * way)
        down = loss()
        what.copy_(kept)
        want = (grad.double() * way.double()).sum().item()
        size = (grad.double().abs()).sum().item()
        # third derivatives are of the gradient's own order here: step^2 = 6e-5 of
        # its size, and 2 * 576 terms * 2^-24 / 2^-6 = 4e-3
        assert abs((up - down) / (2 * step) - want) < 1e-3 * size + 0.01
    assert rar is not None


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_of_zeros_and_broken_rows(dtype):
    """A row of zeros stays zero; NaN and infinity stay in their rows."""
    import torch
    case = Case(dtype, 2, 9, 300, residual=False)
    d = case.dev
    for p in d["partials"]:
        p[2] = 0
    d["partials"][0][4, 7] = float("nan")
    d["partials"][1][6, 299] = float("inf")
    out = case.forward()
    for k in ("hidden", "outs"):
        y = out[k][0]
        assert not y[2].any()
        clean = [i for i in range(9) if i not in (4, 6)]
        assert torch.isfinite(y[clean]).all() and y[4].isnan().all() and y[6].isnan().any()
    case = Case(dtype, 2, 9, 300)
    d = case.dev
    d["total"][2] = 0
    d["hidden"][3] = 0
    d["grad_outs"][0][4, 5] = float("nan")
    got = case.backward()
    clean = [i for i in range(9) if i != 4]
    assert torch.isfinite(got["dpartials"][0][clean]).all() and got["dpartials"][0][4].isnan().all()


def test_same_bits_on_repeats_and_any_copy():
    import torch
    for dtype in DTYPES:
        case = Case(dtype, 4, 333, 700, groups=3)
        f0, b0 = case.forward(), case.backward()
        for _ in range(5):
            f, b = case.forward(copies=2), case.backward(copies=2)
            assert torch.equal(f["hidden"][1], f0["hidden"][0]) and torch.equal(f["outs"][1], f0["outs"][0])
            assert torch.equal(b["dpartials"][1], b0["dpartials"][0])
            assert all(torch.equal(b[k], b0[k]) for k in ("dresidual", "dpost_weight", "dgate", "dpre_weight"))


def test_streams_and_graph_replays():
    import torch
    import ring_all_reduce_channelmask_amd as rar
    case = Case("bfloat16", 3, 200, 640, groups=4)
    d, cfg = case.dev, case.config()
    wants = ("dresidual", "dpost_weight", "dgate", "dpre_weight")

    def buffers():
        return case.forward(), case.backward()
    (fa, ba), (fb, bb) = buffers(), buffers()

    def both(f, b, stream=None):
        rar.norm_allreduce(d["partials"], f["hidden"], f["outs"], residual=d["residual"], total=f["total"], stream=stream, **cfg)
        rar.norm_allreduce_backward(d["grad_hidden"], d["grad_outs"], b["dpartials"], total=d["total"], hidden=d["hidden"], stream=stream,
                                    **{k: b[k] for k in wants}, **cfg)

    def same():
        return all(torch.equal(x, y) for x, y in [(fa["hidden"][0], fb["hidden"][0]), (fa["outs"][0], fb["outs"][0]), (fa["total"], fb["total"]),
                                                  (ba["dpartials"][0], bb["dpartials"][0])] + [(ba[k], bb[k]) for k in wants])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    both(fa, ba, side)
    side.synchronize()
    both(fb, bb)
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(fa, ba)
    for step in range(3):
        for k in ("partials", "grad_hidden", "grad_outs"):
            for t in d[k]:
                t.copy_(torch.randn(t.shape, device="cuda"))
        d["gate"].copy_(torch.randn(4, 640, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        both(fb, bb)
        assert same(), step


def test_more_than_2_31_elements_between_rows():
    import torch
    case = Case("bfloat16", 2, 40, 130, groups=40)
    stride, d, column = 60_000_001, case.dev, 0
    held = torch.empty(40 * stride, dtype=torch.bfloat16, device="cuda")
    assert held.numel() > 1 << 31

    def far(t=None):
        nonlocal column
        view = held.as_strided((40, 130), (stride, 1), column)
        column += 133
        return view if t is None else view.copy_(t)
    for k in ("partials", "grad_hidden", "grad_outs"):
        d[k] = [far(t) for t in d[k]]
    for k in ("total", "hidden", "residual", "gate"):
        d[k] = far(d[k])
    case.check_forward(case.forward(hidden=[far()], outs=[far()], total=far()))
    case.check_backward(case.backward(dpartials=[far()], dresidual=far(), dgate=far()))


def test_no_rows():
    import torch
    import ring_all_reduce_channelmask_amd as rar
    e, w = torch.empty((0, 8), device="cuda"), torch.ones(8, device="cuda")
    rar.norm_allreduce([e], [e], [e], post_weight=w, pre_weight=w, gate=torch.empty((0, 8), device="cuda"))
    dpost, dpre, dgate = (torch.ones(8, device="cuda") for _ in range(3))
    rar.norm_allreduce_backward([e], [e], [e], total=e, hidden=e, post_weight=w, pre_weight=w, gate=w, dpost_weight=dpost, dpre_weight=dpre,
                                dgate=dgate)
    assert not dpost.any() and not dpre.any() and not dgate.any()
