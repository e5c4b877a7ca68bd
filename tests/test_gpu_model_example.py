"""The tensor-parallel example: its gradients against torch's own on the
unsplit model in 64 bits, its training, its serving path."""
import os
import sys

import numpy as np
import pytest

from oracle import model_ops

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_training_step_gradients():
    """fp32: every sum here has at most 301 terms of order one, so each result
    is within 301 u = 2e-5 of its size, and five of them follow each other."""
    import torch
    import tensor_parallel as ex
    block = ex.Block(3, 64, 48, 301, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(20, 64, generator=g, device="cuda")
    residual = torch.randn(20, 48, generator=g, device="cuda")
    ids = torch.randint(0, 301, (20,), generator=g, device="cuda")
    ids[3] = -1
    rng = torch.tensor([7, 9], device="cuda")
    loss, dproj, dvocab, dres = ex.train_step(block, x, residual, ids, rng, call=2, p=0.25, entropy_bonus=0.1)

    factor = torch.from_numpy(model_ops.keep_factor(7, 11, 20 * 48, 0.25)).view(20, 48)
    w = torch.cat(block.proj, 1).double().cpu().requires_grad_()
    v = torch.cat(block.vocab, 0).double().cpu().requires_grad_()
    r = residual.double().cpu().requires_grad_()
    logp = torch.log_softmax((r + factor * (x.double().cpu() @ w.T)) @ v.T, 1)
    own = ids.cpu()
    given = logp[torch.arange(20), own.clamp(min=0)] * (own >= 0)
    want = -(given.sum() + 0.1 * -(logp.exp() * logp).sum()) / 20
    want.backward()
    assert abs(loss.item() - want.item()) < 1e-4
    for got, ref in ((torch.cat(dproj, 1), w.grad), (torch.cat(dvocab, 0), v.grad), (dres, r.grad)):
        assert (got.double().cpu() - ref).abs().max() < 1e-4 * ref.abs().max()


def test_training_lowers_the_loss_and_serving_runs(capsys):
    import tensor_parallel as ex
    ex.main()
    lines = capsys.readouterr().out.splitlines()
    losses = [float(l.split()[-1]) for l in lines if l.startswith("step")]
    assert len(losses) == 10 and losses[-1] < losses[0] - 0.5 and np.isfinite(losses).all()
    assert sum(l.startswith("adapter") for l in lines) == 4


def test_serving_matches_the_unsplit_model():
    import torch
    import tensor_parallel as ex
    block = ex.Block(4, 96, 40, 500, rank=8, adapters=3, dtype=torch.float32)
    x = torch.randn(9, 96, device="cuda")
    ids = torch.tensor([0, 0, 2, 1, -1, 2, 2, 0, 5], device="cuda")
    out = ex.serve(block, x, ids, ntop=4, temperature=0.5)
    hidden = x.double() @ torch.cat(block.proj, 1).double().T
    down = torch.cat(block.downs, 2).double()
    for t, a in enumerate(ids.tolist()):
        if 0 <= a < 3:
            hidden[t] += block.up[a].double() @ (down[a] @ x[t].double())
    logp = torch.log_softmax(hidden @ torch.cat(block.vocab, 0).double().T / 0.5, 1)
    top, at = logp.sort(dim=1, descending=True, stable=True)
    # fp32 sums of up to 96 terms twice over: far below the gaps of 500 random logits
    assert torch.equal(out.top_ids.long(), at[:, :4])
    assert (out.top_logprobs.double() - top[:, :4]).abs().max() < 1e-4
