"""The operators around an AllReduce on the paths that only large calls take:
adapters by runs of two token tiles and on both sides of the bound between few
and many tokens, log probabilities of exceptional rows that several workgroups
share."""
import numpy as np
import pytest

from oracle import model_ops

from . import test_gpu_adapters, test_gpu_logprobs
from .test_gpu_logprobs import LOWEST, _normal

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "bfloat16"]


def _adapters_definition(dev, dtype):
    """model_ops.adapters on the device, in float64: (y, bound) of every token."""
    import torch
    u = model_ops.U
    y, size = (sum(f(p.double()) for p in dev["partials"]) for f in (lambda v: v, torch.abs))
    bound = size * len(dev["partials"]) * u
    x, down = torch.cat(dev["xs"], 1).double(), torch.cat(dev["downs"], 2).double()
    n, outer, rank = dev["up"].shape
    for a in range(n):
        at = (dev["ids"] == a).nonzero()[:, 0]
        h, hs = x[at] @ down[a].T.contiguous(), x[at].abs() @ down[a].abs().T.contiguous()
        up, s = dev["up"][a].double(), dev["scales"][a].double()
        y[at] += s * (h @ up.T.contiguous())
        off = hs * (x.shape[1] + 64) * 2 * u + h.abs() * (2.0 ** -16 + (rank + 8) * 2 * u)
        bound[at] += s.abs() * (off @ up.abs().T.contiguous())
    bound = bound + y.abs() * 4 * u
    return y, bound + (y.abs() + bound) * model_ops.ROUND[dtype]


def _within(got, want, what):
    y, bound = want
    over = (got.double() - y).abs() - bound
    assert (over <= 0).all(), f"{what}: {over.max().item()} over its bound, first at {(over > 0).nonzero()[:3].tolist()}"


def _ids(kind, tokens, adapters):
    import torch
    t = torch.arange(tokens)
    if kind == "kept":        # a run's two tiles have the same adapter, which its workgroup keeps
        return t // 96 % adapters
    if kind == "changing":    # inside tiles and between a run's
        return t // 24 % (adapters + 1) - 1
    return t * 7 % (adapters + 1) - 1


# ceil(outer / 256) * ceil(tokens / 32) >= 2048: a workgroup takes two tiles
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["kept", "changing", "mixed"])
@pytest.mark.parametrize("tokens,outer,rank,ranks", [(2070, 8200, 16, 5), (2049, 8192, 64, 1), (2080, 8091, 128, 6), (8209, 2041, 33, 3)])
def test_runs_of_two_tiles(dtype, kind, tokens, outer, rank, ranks):
    """The last run ends inside its second tile, in its first, or at its end;
    then the same in place over two of the partials."""
    import torch
    assert -(-outer // 256) * -(-tokens // 32) >= 2048
    g = torch.Generator(device="cuda").manual_seed(tokens)

    def make(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(getattr(torch, dtype))
    widths = [20 + 3 * r for r in range(ranks)]
    widths[-1] = 0 if ranks > 1 else 77
    adapters = 5
    dev = dict(xs=[make(tokens, w) for w in widths], partials=[make(tokens, outer) for _ in widths], downs=[make(adapters, rank, w) * 0.1 for w in widths],
               up=make(adapters, outer, rank) * 0.2, ids=_ids(kind, tokens, adapters).cuda(), scales=torch.rand(adapters, generator=g, device="cuda") + 0.5)
    want = _adapters_definition(dev, dtype)
    for y in test_gpu_adapters._run(dev, copies=2):
        _within(y, want, "apart")
    first = y
    for y in test_gpu_adapters._run(dev, recvs=[dev["partials"][-1], dev["partials"][0]][:ranks]):
        assert torch.equal(y, first), "in place"


# tokens * rank up to 8192 go token by token
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,rank", [(127, 64), (128, 64), (129, 64), (512, 16), (513, 16), (63, 128), (65, 128), (8192, 1), (8193, 1)])
def test_both_sides_of_the_bound_between_few_and_many_tokens(dtype, tokens, rank):
    ids = np.random.default_rng(tokens).integers(-1, 4, tokens)
    dev, want = test_gpu_adapters._case(dtype, tokens, [70, 33], 270, rank, 4, ids, rank, pad=1)
    test_gpu_adapters._check(test_gpu_adapters._run(dev)[0], want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ntop", [0, 2, 32])
def test_exceptional_rows_over_several_workgroups(dtype, ntop):
    """Few rows of a large vocabulary: every row has several parts, joined by a
    second kernel."""
    import ctypes
    from ring_all_reduce_channelmask_amd import _lib
    widths = [60000, 40000, 0, 31075]
    vocab, low = sum(widths), LOWEST[dtype]
    need = ctypes.c_size_t()
    _lib.check(_lib.load().rar_logprobs_workspace((ctypes.c_int64 * 4)(*widths), 4, 14, _lib.DTYPE[dtype], ntop, ctypes.byref(need)))
    assert need.value > 0  # several parts
    x = _normal(14, vocab, 31)
    x[0] = -np.inf                               # nothing left
    x[1] = low                                   # masked by the lowest value: uniform
    x[2] = -np.inf
    x[2, 90000] = 2.0                            # one token left
    x[3, 1::2] = -np.inf
    x[4, 17] = np.nan
    x[5, 130000] = np.inf
    x[6] = np.nan
    x[7, :vocab - 5] = low                       # the last part alone
    x[8] = 0.0
    x[8, ::3] = -0.0                             # equal to 0
    x[9, :100000] = -np.inf                      # two ranks masked entirely
    x[10] = -1e30
    x[11] = 200.0
    x[11, 3] = -low                              # the largest value, in the first part
    x[12] = -np.inf
    x[12, -1] = low
    x[13, 64:] = -np.inf                         # the first part alone
    ids = [0, 1, 90000, 2, 3, 130000, 5, vocab - 1, 8, 100001, 10, 3, vocab - 1, -1]
    test_gpu_logprobs._check(x, widths, dtype, ids, ntop)
    at = [0, 1, 2, 3, 7, 8, 9, 12, 13]
    test_gpu_logprobs._check(x[at], widths, dtype, [3] * len(at), ntop, scale=0.5)
