"""Logits whose scaled value leaves the range of fp32: they count as the
infinity that the product rounds to, in every output and in the gradient."""
import numpy as np
import pytest

from oracle import model_ops

from .test_gpu_logprobs import LOWEST, _close, _ids, _normal, _shards

pytestmark = pytest.mark.gpu

# rows of the first are one workgroup's, of the second split and joined
WIDTHS = [[5000, 4000, 1001], [70000, 0, 61075]]


def _rounded(exact, scale):
    """The logits, infinite where scale * logit is in fp32."""
    with np.errstate(over="ignore"):
        z = (exact * float(np.float32(scale))).astype(np.float32)
    return np.where(np.isinf(z), z, exact).astype(np.float64)


def _rows(vocab, dtype):
    low = LOWEST[dtype]
    x = _normal(8, vocab, 21)
    x[0] = low                                   # the mask leaves nothing
    x[1] = low
    x[1, 7] = -1e38                              # the one whose scaled value is finite
    x[2] = low
    x[2, [9, 4000, vocab - 1]] = [1.0, 2.0, 3.0]
    x[3] = low
    x[3, ::2] = -np.inf
    x[4, ::3] = low
    x[5] = -np.inf
    x[5, 2] = low
    x[6] = low / 2
    x[7, 17] = -low                              # overflows upwards
    return x


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("widths", WIDTHS, ids=["whole", "split"])
@pytest.mark.parametrize("scale", [1.25, 2.0, 3.0, 0.75])
def test_scaled_logits_beyond_fp32(dtype, widths, scale):
    import torch
    import ring_all_reduce_channelmask_amd as rar
    vocab = sum(widths)
    shards, exact = _shards(_rows(vocab, dtype), widths, dtype)
    seen = _rounded(exact, scale)
    ids = [0, 7, 9, 3, 3, 2, 11, 17]
    for ntop in (0, 5, 32):
        got = rar.logprobs(shards, _ids(ids), ntop=ntop, scale=scale)
        want = model_ops.logprobs(seen, ids, scale, ntop)
        for name in ("lse", "entropy", "logprob"):
            _close(getattr(got, name), want[name], want[name + "_bound"], name)
        assert np.array_equal(got.top_ids.cpu().numpy(), want["top_ids"])
        _close(got.top_logprobs, want["top_logprobs"], want["top_bound"], "top_logprobs")
    r = np.random.default_rng(3)
    g, h, l = (r.standard_normal(8).astype(np.float32) for _ in range(3))
    grads = rar.logprobs_backward(shards, _ids(ids), got.lse, got.entropy, *[torch.from_numpy(v).cuda() for v in (g, h, l)], scale=scale)
    # rows whose lse fp32 holds to a small absolute error, and those masked entirely
    lse = got.lse.double().cpu().numpy()
    at = [i for i in range(8) if lse[i] == -np.inf or abs(lse[i]) < 1e30]
    assert {2, 4} <= set(at) and (scale < 1 or {0, 3, 5} <= set(at))
    want, bound = model_ops.logprobs_backward(seen[at], [ids[i] for i in at], lse[at], got.entropy[at].double().cpu().numpy(),
                                              *[v[at].astype(float) for v in (g, h, l)], scale, dtype)
    _close(torch.cat(grads, 1)[at], want, bound, "gradient")
    if scale > 1:
        assert (torch.cat(grads, 1)[0] == 0).all()
