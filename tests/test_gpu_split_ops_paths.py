"""Paths of the embedding gradient and of the 8-bit projection on both sides of
the sizes where another one is taken."""
import numpy as np
import pytest

from oracle import model_ops

from .test_gpu_embedding import _backward
from .test_gpu_projection8 import _run

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "bfloat16"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [8127, 8128, 8191, 8192, 8193])
def test_gradient_ordered_by_pairs_and_by_digits(dtype, tokens):
    """Up to 8192 tokens are ordered by comparing pairs (the last list fills
    the workgroup's memory), more by their digits."""
    r = np.random.default_rng(tokens)
    ids = np.minimum(np.exp(r.random(tokens) * np.log(500)).astype(int) - 1, 499)
    ids = np.where(r.random(tokens) < 0.05, -1, (ids * 7 + 3) % 500)
    ids[[0, -1]] = 499, 0
    _backward(dtype, [70, 0, 300, 130], 5, ids, copies=2)
    _backward(dtype, [70, 0, 300, 130], 5, ids, table_dtype="float32", accumulate=True, scale=0.5, pad=1)


# the digits that a vocabulary's size has (it stands for padding): 1 to 2 passes
# of 9 bits each, 2 to 3, 3 to 4
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [511, 512, 262143, 262144, 300001, (1 << 27) - 1, 1 << 27])
def test_gradient_at_every_number_of_digits(dtype, vocab):
    """Tokens of the first and the last rows, and of each digit's largest
    values.  A large table is added to, so that only its rows that occur
    matter."""
    import torch
    import ring_all_reduce_channelmask_amd as rar
    tokens, width = 9001, 3
    r = np.random.default_rng(vocab)
    some = np.unique(np.concatenate([r.integers(0, vocab, 300), [0, 1, vocab - 1, vocab - 2, vocab // 2, 511 % vocab, 512 % vocab, 0x3FFFF % vocab, 0x40000 % vocab]]))
    ids = some[r.integers(0, len(some), tokens)]
    ids[r.random(tokens) < 0.03] = -1
    ids[r.random(tokens) < 0.03] = vocab
    grads = torch.from_numpy(r.integers(-8, 9, (tokens, width)).astype(np.float32)).cuda().to(getattr(torch, dtype))
    if vocab <= 300001:
        _backward(dtype, [vocab // 3, vocab - vocab // 3], width, ids)
    table = torch.ones(vocab, width, dtype=torch.float32, device="cuda")
    rar.embedding_allreduce_backward([grads], torch.from_numpy(ids).cuda(), [table[:vocab - 7], table[vocab - 7:]], scale=0.5, accumulate=True)
    # sums of whole numbers times a half: exact
    sums = np.zeros((len(some) + 1, width))
    there = (ids >= 0) & (ids < vocab)
    np.add.at(sums, np.searchsorted(some, ids[there]), grads.double().cpu().numpy()[there])
    rows = torch.from_numpy(some).cuda()
    assert np.array_equal(table[rows].cpu().numpy(), 1 + 0.5 * sums[:-1])
    table[rows] = 1
    assert bool((table == 1).all())


# 16 rows of tiles: 16 columns of 256 channels and 16 of 192 behind them; 32: 8 and 5
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,widths,outer", [(4000, [70, 33, 160], 7100), (4096, [64], 7168), (8100, [96], 2900)])
def test_both_widths_of_large_tiles_in_one_launch(dtype, tokens, widths, outer):
    import torch
    g = torch.Generator(device="cuda").manual_seed(tokens)
    xs, ws = ([torch.randint(-128, 128, (n, w), generator=g, device="cuda").to(torch.int8) for w in widths] for n in (tokens, outer))
    sx, sw = torch.rand(tokens, generator=g, device="cuda"), torch.rand(outer, generator=g, device="cuda")
    res = torch.randn(tokens, outer, generator=g, device="cuda").to(getattr(torch, dtype))
    got = _run(dict(xs=xs, weights=ws, x_scales=sx, weight_scales=sw, residual=res), tokens, outer, dtype, copies=2)
    # below 2^53: exact
    prod = sum(x.double() @ w.double().T for x, w in zip(xs, ws)) * sx.double()[:, None] * sw.double()
    want = prod + res.double()
    bound = prod.abs() * 3 * model_ops.U + want.abs() * 2 * model_ops.U
    bound = bound + (want.abs() + bound) * model_ops.ROUND[dtype]
    for y in got:
        assert ((y.double() - want).abs() <= bound).all()
