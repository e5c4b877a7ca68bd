"""Embedding, norms, 8-bit projections and log probabilities together, as a
split model uses them: the example's gradients against torch's own on the
unsplit model in 64 bits, its serving path against the same quantisation in 64
bits, its run, and a training step captured and replayed."""
import os
import sys

import pytest

from oracle import model_ops

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _unsplit(model):
    """The weights in 64 bits on the host, whole, as leaves."""
    import torch

    def whole(ts, dim):
        return torch.cat(list(ts), dim).double().cpu().requires_grad_()

    def one(t):
        return t.double().cpu().requires_grad_()
    return dict(tables=whole(model.tables, 0), vocab=whole(model.vocab, 0), first_norm=one(model.first_norm),
                blocks=[dict(up=whole(b["up"], 0), down=whole(b["down"], 1), post=one(b["post"]), gate=one(b["gate"]), pre=one(b["pre"])) for b in model.blocks])


def _rms(x):
    return x / (x * x).mean(1, keepdim=True).add(1e-6).sqrt()


def _forward(model, w, ids, project):
    import torch
    there = (ids >= 0)[:, None]
    h = torch.where(there, w["tables"][ids.clamp(min=0)] * model.embedding_scale, torch.zeros((), dtype=torch.float64))
    x = _rms(h) * w["first_norm"]
    for b in w["blocks"]:
        total = project(torch.relu(project(x, b["up"])), b["down"])
        h = model.residual_scale * h + b["gate"] * (_rms(total) * b["post"])
        x = _rms(h) * b["pre"]
    return x @ w["vocab"].T


def test_training_step_gradients():
    """fp32: sums of at most 160 terms of order one (160 u = 1e-5 of their
    size), some ten of them in a row; the embedding's padding has a gradient of
    zero."""
    import torch
    import split_model as ex
    model = ex.Model(ranks=3, vocab=101, width=48, inner=160, layers=2, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(0, 101, (40,), generator=g, device="cuda")
    ids[5], ids[6:9] = -1, ids[0]
    targets = torch.randint(0, 101, (40,), generator=g, device="cuda")
    loss, grads = ex.train_step(model, ids, targets)
    w = _unsplit(model)
    logp = torch.log_softmax(_forward(model, w, ids.cpu(), lambda x, m: x @ m.T), 1)
    want = -logp[torch.arange(40), targets.cpu()].mean()
    want.backward()
    assert abs(loss.item() - want.item()) < 1e-4

    def near(got, ref):
        assert (got.double().cpu() - ref).abs().max() < 2e-4 * ref.abs().max()
    near(torch.cat(grads["tables"], 0), w["tables"].grad)
    near(torch.cat(grads["vocab"], 0), w["vocab"].grad)
    near(grads["first_norm"], w["first_norm"].grad)
    for d, b in zip(grads["blocks"], w["blocks"]):
        near(torch.cat(d["up"], 0), b["up"].grad)
        near(torch.cat(d["down"], 1), b["down"].grad)
        for k in ("post", "gate", "pre"):
            near(d[k], b[k].grad)


def test_serving_matches_the_same_quantisation():
    """In 64 bits with the same quantised weights; an activation next to the
    middle of two integers may fall to the other one, which moves a sum of 160
    terms by one step of 1/127."""
    import numpy as np
    import torch
    import split_model as ex
    model = ex.Model(ranks=3, vocab=101, width=48, inner=160, layers=2, dtype=torch.float32)
    ex.quantize(model)
    ids = torch.arange(0, 90, 7, device="cuda")
    out = ex.serve(model, ids)

    def project(x, m):
        (qx,), sx, _ = model_ops.quantize_rows([x.detach().numpy()])
        (qm,), sm, _ = model_ops.quantize_rows([m.detach().numpy()])
        return torch.from_numpy((qx @ qm.T) * sx[:, None] * sm[None, :])
    logp = torch.log_softmax(_forward(model, _unsplit(model), ids.cpu(), project), 1)
    top = logp.sort(dim=1, descending=True, stable=True)[0][:, :4]
    assert np.abs(out.top_logprobs.double().cpu().numpy() - top.detach().numpy()).max() < 0.02


def test_the_example_runs(capsys):
    import split_model as ex
    ex.main()
    lines = capsys.readouterr().out.splitlines()
    assert sum(l.startswith("step") for l in lines) == 8 and sum(l.startswith("after") for l in lines) == 3


def test_a_step_captured_and_replayed():
    """The operators of a layer, both ways, in one graph: workspaces of its
    own, while eager calls of the same shapes go on between the replays."""
    import torch
    import ring_all_reduce_channelmask_amd as rar
    rows, width, ranks = 130, 320, 3
    g = torch.Generator(device="cuda").manual_seed(4)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()
    tables, ids = [rand(50, width) for _ in range(ranks)], torch.randint(-1, 150, (rows,), generator=g, device="cuda")
    weights, w_scales = rar.quantize_rows([rand(width, 64) for _ in range(ranks)])
    post, gate, pre = rand(width), rand(width), rand(width)
    acts, dout = [rand(rows, 64) for _ in range(ranks)], rand(rows, width)

    def buffers():
        return dict(emb=rand(rows, width), y=rand(rows, width), hidden=rand(rows, width), out=rand(rows, width), total=rand(rows, width),
                    dpartial=rand(rows, width), dres=rand(rows, width), dpost=rand(width), dgate=rand(width), dpre=rand(width),
                    tables=[rand(50, width) for _ in range(ranks)])

    def layer(b):
        rar.embedding_allreduce(tables, ids, [b["emb"]], scale=3.0)
        q, s = rar.quantize_rows(acts)
        rar.int8_projection_allreduce(q, s, weights, w_scales, [b["y"]])
        cfg = dict(post_weight=post, gate=gate, pre_weight=pre)
        rar.norm_allreduce([b["y"]], [b["hidden"]], [b["out"]], residual=b["emb"], total=b["total"], **cfg)
        rar.norm_allreduce_backward([], [dout], [b["dpartial"]], total=b["total"], hidden=b["hidden"], dresidual=b["dres"], dpost_weight=b["dpost"],
                                    dgate=b["dgate"], dpre_weight=b["dpre"], **cfg)
        rar.embedding_allreduce_backward([b["dres"]], ids, b["tables"], scale=3.0)
    a, b = buffers(), buffers()
    layer(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(a)
    for step in range(4):
        ids.copy_(torch.randint(-1, 150, (rows,), device="cuda"))
        for t in acts + [dout]:
            t.copy_(torch.randn(t.shape, device="cuda"))
        graph.replay()
        layer(b)
        torch.cuda.synchronize()
        for k in a:
            for x, y in zip(a[k] if k == "tables" else [a[k]], b[k] if k == "tables" else [b[k]]):
                assert torch.equal(x, y), (step, k)
