"""The norms around a block and their gradient for rows of every magnitude that
the types have, against the definition in 64 bits: sums of squares and of
products that leave fp32's range while the results do not."""
import numpy as np
import pytest

from oracle import model_ops

from .test_gpu_embedding import _tensor
from .test_gpu_norms import EPS, Case

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "bfloat16"]
# a row each: ordinary ones between those whose squares, or the sum of them, leave fp32's range
SIZES = [1.0, 1e18, 3e-18, 2e17, 1e19, 0.0, 3e19, 1e25, 1e-25, 3e37, 1.0, 3e38]
# one wave, several, the row's end within a vector, more than a vector a thread in fp32 and in both types
WIDTHS = [7, 130, 515, 2048, 7168, 16390]
TINY = 2.0 ** -149  # results below fp32's normal numbers: half of it for each of a few roundings
# A result's own rounding: below 2^-126, where both types' normal numbers end,
# their steps are 2^-126 times 2^-23 and 2^-7, and a rounding is half a step off.
LAST = {"float32": 2.0 ** -150, "bfloat16": 2.0 ** -134}


def _rows(r, width, size=1.0):
    """Rows of the magnitudes of SIZES, at most 3.3e38."""
    a = np.clip(r.standard_normal((len(SIZES), width)), -1.1, 1.1) * np.array(SIZES)[:, None]
    return np.clip(a * size, -3.3e38, 3.3e38)


def _check(got, want, slack, what):
    y, bound = want
    off = np.abs(got.double().cpu().numpy().reshape(y.shape) - y) - bound
    assert (off <= slack).all(), f"{what}: rows {np.unique(np.nonzero(~(off <= slack))[0])}, {np.nanmax(off)} over its bound"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_forward(dtype, width):
    """The norm behind the block (rows of the sum) and the one in front of the
    next (rows of the residual, the sum's norm of ordinary size beside them)."""
    r = np.random.default_rng(width)
    for post in (True, False):
        case = Case(dtype, 1, len(SIZES), width, groups=1, post=post, residual=post, scale=1.0, seed=width)
        case.dev["partials"], case.val["partials"] = [[v] for v in _tensor(_rows(r, width), dtype)]
        if post:
            case.dev["residual"], case.val["residual"] = _tensor(_rows(r, width)[::-1].copy(), dtype)
        else:  # the gate may take the sum beyond the range
            case.dev["gate"], case.val["gate"] = _tensor(0.5 + 0.5 * r.random((1, width)), dtype)
        out, v = case.forward(), case.val
        want = model_ops.norms(np.stack(v["partials"]), v["residual"], 1.0, v["post"], v["gate"], v["pre"], EPS, dtype)
        # the statistic's product with an element, with the weight and the gate: three roundings
        for k, y in (("hidden", out["hidden"][0]), ("out", out["outs"][0])):
            _check(y, want[k], 4 * TINY + LAST[dtype], f"post {post} {k}")
        assert out["outs"][0].isfinite().all() and out["outs"][0][1:5].any(1).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("kind", ["pre", "post"])
def test_gradient(dtype, width, kind):
    """Of rows of `hidden`, and of rows of `total`: the gradient is that of the
    row's direction over its magnitude, the weights' one of ordinary size."""
    r = np.random.default_rng(width + 1)
    case = Case(dtype, 2, len(SIZES), width, groups=1, post=kind == "post", pre=kind == "pre", residual=False, scale=1.0, seed=width)
    name = "hidden" if kind == "pre" else "total"
    case.dev[name], case.val[name] = _tensor(_rows(r, width), dtype)
    if kind == "pre":
        case.dev["grad_hidden"], case.val["grad_hidden"] = [], []
        case.dev["total"], case.val["total"] = _tensor(r.standard_normal((len(SIZES), width)), dtype)
    got, v = case.backward(dresidual=None), case.val
    want = model_ops.norms_backward(v["grad_hidden"], v["grad_outs"], v["total"], v["hidden"], 1.0, v["post"], v["gate"], v["pre"], EPS, dtype)
    # at the largest rows 1 / rms is below the normal numbers, half a step off, and
    # multiplies gradients (of two copies, the weight and the gate with them, and
    # the part along the row, which is not larger in the root of the mean square)
    n = sum(np.abs(g) for g in v["grad_outs"] + v["grad_hidden"]).max()
    factor = np.abs(v["pre" if kind == "pre" else "post"]).max() * max(1.0, np.abs(v["gate"]).max())
    slack = TINY * (2 + n * factor * (1 + width ** 0.5)) + LAST[dtype]
    _check(got["dpartials"][0], want["dpartial"], slack, "dpartials")
    weight = {"pre": ("dpre_weight", "dpre"), "post": ("dpost_weight", "dpost")}[kind]
    _check(got[weight[0]], want[weight[1]], 0.0, weight[0])
    if kind == "post":
        _check(got["dgate"], want["dgate"], 0.0, "dgate")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_products_beyond_the_range(dtype, width):
    """The sum of gradient times row leaves fp32's range, neither the squares
    nor the results do; a row of ordinary size beside it."""
    r = np.random.default_rng(width + 2)
    case = Case(dtype, 1, 4, width, post=False, residual=False, scale=1.0, seed=width)
    size = np.array([[1e15], [1.0], [1e10], [1e16]])
    # of one sign, so that nothing cancels within a partial sum
    case.dev["hidden"], case.val["hidden"] = _tensor((0.5 + r.random((4, width))) * size, dtype)
    outs = _tensor((0.5 + r.random((4, width))) * np.array([[1e25], [1.0], [1e30], [1e23]]), dtype)
    case.dev["grad_outs"], case.val["grad_outs"] = [[v] for v in outs]
    case.dev["grad_hidden"], case.val["grad_hidden"] = [], []
    case.dev["pre"], case.val["pre"] = case.dev["pre"].abs(), np.abs(case.val["pre"])
    got, v = case.backward(dresidual=None), case.val
    want = model_ops.norms_backward([], v["grad_outs"], None, v["hidden"], 1.0, None, None, v["pre"], EPS, dtype)
    _check(got["dpartials"][0], want["dpartial"], 0.0, "dpartials")
    _check(got["dpre_weight"], want["dpre"], 0.0, "dpre_weight")


@pytest.mark.parametrize("dtype", DTYPES)
def test_broken_rows_beside_large_ones(dtype):
    """NaN and infinity stay in their rows, and what such a row gives elsewhere
    than at the broken element does not depend on the others' magnitude."""
    import torch
    r = np.random.default_rng(5)
    case = Case(dtype, 1, len(SIZES), 300, post=True, residual=False, scale=1.0)
    rows = _rows(r, 300)
    rows[0, 7], rows[3, 299], rows[9, 0] = np.nan, np.inf, -np.inf
    case.dev["partials"], _ = [[v] for v in _tensor(rows, dtype)]
    y = case.forward()["outs"][0]
    broken, clean = [0, 3, 9], [i for i in range(len(SIZES)) if i not in (0, 3, 9)]
    assert torch.isfinite(y[clean]).all() and y[broken].isnan().any(1).all()
    case.dev["hidden"], _ = _tensor(rows, dtype)
    case.dev["total"], _ = _tensor(rows[::-1].copy(), dtype)
    got = case.backward()
    both = [i for i in clean if len(SIZES) - 1 - i not in broken]
    assert torch.isfinite(got["dpartials"][0][both]).all() and got["dpartials"][0][[11, 8, 2]].isnan().any(1).all()
    assert torch.isfinite(got["dresidual"][clean]).all()
