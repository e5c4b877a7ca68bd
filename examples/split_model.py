"""A small model split over N virtual ranks of one GPU, from token ids to the
loss, with every reduction over the ranks in an operator.

    x = norm(E[ids]), and in each layer, rank r having the columns W1_r of the
    first projection and the rows W2_r of the second:
      P_r = relu(x W1_r^T) W2_r^T
      h  <- a h + g (rms(sum_r P_r) w_post)      the block's norm, gate, residual
      x  <- rms(h) w_pre                         the next layer's input
    logits = x V_r^T over the ranks' parts of the vocabulary

Training: the forward pass, the log probabilities' gradient and the way back
through the same places.  Serving: the projections in 8-bit integers, their
inputs quantised a token at a time.

    python examples/split_model.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import ring_all_reduce_channelmask_amd as rar  # noqa: E402


class Model:
    """Weights of `layers` blocks of `width` with `inner` hidden columns, cut
    over the ranks."""

    def __init__(self, ranks, vocab, width, inner, layers, dtype=torch.bfloat16, seed=3):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def make(*shape, size=1.0, around=0.0):
            return (around + torch.randn(*shape, generator=g, device="cuda") * size).to(dtype)
        self.ranks, self.width, self.layers = ranks, width, layers
        self.residual_scale, self.embedding_scale = 0.9, width ** 0.5
        self.tables = list(make(vocab, width, size=width ** -0.5).tensor_split(ranks, 0))
        self.vocab = [w.contiguous() for w in make(vocab, width, size=width ** -0.5).tensor_split(ranks, 0)]
        self.first_norm = make(width, size=0.1, around=1.0)
        self.blocks = []
        for _ in range(layers):
            self.blocks.append(dict(
                up=[w.contiguous() for w in make(inner, width, size=width ** -0.5).tensor_split(ranks, 0)],
                down=[w.contiguous() for w in make(width, inner, size=inner ** -0.5).tensor_split(ranks, 1)],
                post=make(width, size=0.1, around=1.0), gate=make(width, size=0.1, around=0.7), pre=make(width, size=0.1, around=1.0)))
        self.quantized = None

    def embed(self, ids):
        """The residual stream and the first layer's input."""
        like = self.tables[0]
        hidden = torch.empty(len(ids), self.width, dtype=like.dtype, device="cuda")
        rar.embedding_allreduce(self.tables, ids, [hidden], scale=self.embedding_scale)
        out = torch.empty_like(hidden)
        rar.norm_allreduce([hidden], [], [out], pre_weight=self.first_norm)
        return hidden, out


def train_step(model, ids, targets):
    """The mean loss of the targets and the gradients of all weights, in the
    weights' structure."""
    stream, x = model.embed(ids)
    kept, embedded = [], stream
    for b in model.blocks:
        acts = [torch.relu(x @ w.T) for w in b["up"]]
        partials = [a @ w.T for a, w in zip(acts, b["down"])]
        hidden, out, total = (torch.empty_like(stream) for _ in range(3))
        rar.norm_allreduce(partials, [hidden], [out], residual=stream, residual_scale=model.residual_scale, post_weight=b["post"], gate=b["gate"],
                           pre_weight=b["pre"], total=total)
        kept.append((x, acts, total, hidden))
        stream, x = hidden, out
    logits = [x @ w.T for w in model.vocab]
    out = rar.logprobs(logits, targets)
    rows = len(ids)
    loss = -out.logprob.mean()
    # the way back
    dlogits = rar.logprobs_backward(logits, targets, out.lse, None, torch.full((rows,), -1.0 / rows, device="cuda"), grads=logits)
    grads = dict(vocab=[d.T @ x for d in dlogits], blocks=[])
    dxs = [d @ w for d, w in zip(dlogits, model.vocab)]  # of each rank's copy of x
    dstream = []
    for b, (x, acts, total, hidden) in zip(reversed(model.blocks), reversed(kept)):
        dpartial, dresidual = torch.empty_like(hidden), torch.empty_like(hidden)
        dpost, dgate, dpre = (torch.empty_like(b[k]) for k in ("post", "gate", "pre"))
        rar.norm_allreduce_backward(dstream, dxs, [dpartial], total=total, hidden=hidden, residual_scale=model.residual_scale, post_weight=b["post"],
                                    gate=b["gate"], pre_weight=b["pre"], dresidual=dresidual, dpost_weight=dpost, dgate=dgate, dpre_weight=dpre)
        dacts = [(dpartial @ w) * (a > 0) for w, a in zip(b["down"], acts)]
        grads["blocks"].insert(0, dict(down=[dpartial.T @ a for a in acts], up=[d.T @ x for d in dacts], post=dpost, gate=dgate, pre=dpre))
        dxs = [d @ w for d, w in zip(dacts, b["up"])]
        dstream = [dresidual]
    dembedded, grads["first_norm"] = torch.empty_like(embedded), torch.empty_like(model.first_norm)
    # the first norm has the embedding for its hidden stream
    rar.norm_allreduce_backward(dstream, dxs, [dembedded], hidden=embedded, pre_weight=model.first_norm, dpre_weight=grads["first_norm"])
    grads["tables"] = [torch.empty_like(t) for t in model.tables]
    rar.embedding_allreduce_backward([dembedded], ids, grads["tables"], scale=model.embedding_scale)
    return loss, grads


def quantize(model):
    """The projections' weights in 8-bit integers, a scale a channel."""
    model.quantized = [dict(up=[rar.quantize_rows([w]) for w in b["up"]], down=rar.quantize_rows(b["down"])) for b in model.blocks]


def serve(model, ids, ntop=4):
    """The most probable next token of each position, through the 8-bit
    projections.  Positions do not see each other in this model."""
    stream, x = model.embed(ids)
    for b, q in zip(model.blocks, model.quantized):
        (qx,), sx = rar.quantize_rows([x])
        acts = []
        for weights, scales in q["up"]:  # each rank's columns: no reduction
            y = torch.empty(len(ids), weights[0].shape[0], dtype=x.dtype, device="cuda")
            rar.int8_projection_allreduce([qx], sx, weights, scales, [y])
            acts.append(torch.relu_(y))
        qa, sa = rar.quantize_rows(acts)
        total, hidden, out = (torch.empty_like(stream) for _ in range(3))
        rar.int8_projection_allreduce(qa, sa, *q["down"], [total])
        rar.norm_allreduce([total], [hidden], [out], residual=stream, residual_scale=model.residual_scale, post_weight=b["post"], gate=b["gate"], pre_weight=b["pre"])
        stream, x = hidden, out
    none = torch.full((len(ids),), -1, dtype=torch.int64, device="cuda")
    return rar.logprobs([x @ w.T for w in model.vocab], none, ntop=ntop)


def main():
    model = Model(ranks=4, vocab=4003, width=512, inner=2048, layers=2)
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, 4003, (512,), generator=g, device="cuda")
    targets = (ids * 7 + 11) % 4003  # what follows a token in this language
    for step in range(8):
        loss, grads = train_step(model, ids, targets)
        for w, d in zip(model.tables + model.vocab, grads["tables"] + grads["vocab"]):
            w -= 2.0 * d
        for b, d in zip(model.blocks, grads["blocks"]):
            for k in ("up", "down"):
                for w, dw in zip(b[k], d[k]):
                    w -= 0.5 * dw
        print(f"step {step}: loss {loss.item():.4f}", flush=True)
    quantize(model)
    out = serve(model, ids[:3])
    for row in range(3):
        print(f"after {ids[row].item()}: tokens {out.top_ids[row].tolist()}", flush=True)


if __name__ == "__main__":
    main()
