"""A tensor-parallel block and its loss over N virtual ranks of one GPU.

Training: each rank multiplies its columns of the input by its part of a
row-parallel projection; the partial products meet in one AllReduce with
dropout and a residual; each rank forms the logits of its part of the
vocabulary; the log probabilities of the given tokens come from all parts at
once.  The way back takes the same places: the gradient of the logits, the
AllReduce of the ranks' gradients of the block's output with the dropout
undone, the weights' gradients.

Serving: the same projection with low-rank adapters of several requests, then
each token's most probable continuations.

    python examples/tensor_parallel.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import ring_all_reduce_channelmask_amd as rar  # noqa: E402


class Block:
    """A row-parallel projection [outer, inner] and output embedding
    [vocab, outer], each cut over the ranks, with `adapters` low-rank adapters
    of the projection."""

    def __init__(self, ranks, inner, outer, vocab, rank=16, adapters=4, dtype=torch.bfloat16, seed=17):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def make(*shape, size):
            return (torch.randn(*shape, generator=g, device="cuda") * size).to(dtype)
        # cut, as the ranks hold them
        self.proj = [w.contiguous() for w in make(outer, inner, size=inner ** -0.5).tensor_split(ranks, 1)]
        self.vocab = [w.contiguous() for w in make(vocab, outer, size=outer ** -0.5).tensor_split(ranks, 0)]
        self.downs = [w.contiguous() for w in make(adapters, rank, inner, size=inner ** -0.5).tensor_split(ranks, 2)]
        self.up = make(adapters, outer, rank, size=rank ** -0.5)
        self.scales = torch.ones(adapters, device="cuda")

    def split(self, x):
        return list(x.tensor_split(len(self.proj), 1))


def train_step(block, x, residual, ids, rng, call=0, p=0.1, entropy_bonus=0.01):
    """The loss of a batch and the gradients of both weights (by rank) and of
    the residual.  `rng` is the dropout's [seed, offset]."""
    xs, ranks, rows = block.split(x), len(block.proj), x.shape[0]
    # forward
    partials = [a @ w.T for a, w in zip(xs, block.proj)]
    hidden = [torch.empty_like(residual) for _ in range(ranks)]  # every rank's copy
    rar.dropout_allreduce([t.view(-1) for t in partials], [t.view(-1) for t in hidden], p, rng, call=call,
                          residual=residual.contiguous().view(-1))
    logits = [h @ v.T for h, v in zip(hidden, block.vocab)]
    out = rar.logprobs(logits, ids)
    loss = -(out.logprob.sum() + entropy_bonus * out.entropy.sum()) / rows
    # backward; the logits give way to their gradients
    grad = torch.full((rows,), -1.0 / rows, device="cuda")
    dlogits = rar.logprobs_backward(logits, ids, out.lse, out.entropy, grad, grad_entropy=grad * entropy_bonus, grads=logits)
    dvocab = [d.T @ h for d, h in zip(dlogits, hidden)]
    dhidden = [d @ v for d, v in zip(dlogits, block.vocab)]  # of each rank's copy
    dresidual = torch.empty_like(residual)
    dpartial = torch.empty_like(residual)                    # the same for every rank's partial product
    rar.dropout_allreduce_backward([t.view(-1) for t in dhidden], [dpartial.view(-1)], p, rng, call=call,
                                   dresidual=dresidual.view(-1))
    dproj = [dpartial.T @ a for a in xs]
    return loss, dproj, dvocab, dresidual


def serve(block, x, adapter_ids, ntop=5, temperature=1.0):
    """The most probable next tokens of each row of x, whose request uses the
    adapter `adapter_ids[row]` (-1: none)."""
    xs = block.split(x)
    partials = [a @ w.T for a, w in zip(xs, block.proj)]
    hidden = [torch.empty_like(t) for t in partials]
    rar.adapter_allreduce(xs, partials, hidden, block.downs, block.up, adapter_ids, block.scales)
    logits = [h @ v.T for h, v in zip(hidden, block.vocab)]
    none = torch.full((x.shape[0],), -1, dtype=torch.int64, device="cuda")
    return rar.logprobs(logits, none, ntop=ntop, scale=1.0 / temperature)


def main():
    torch.manual_seed(0)
    ranks, inner, outer, vocab, rows = 4, 1024, 512, 8003, 256
    block = Block(ranks, inner, outer, vocab)
    x = torch.randn(rows, inner, device="cuda").bfloat16()
    residual = torch.randn(rows, outer, device="cuda").bfloat16()
    ids = torch.randint(0, vocab, (rows,), device="cuda")
    rng = torch.tensor([1234, 0], device="cuda")
    for step in range(10):
        loss, dproj, dvocab, _ = train_step(block, x, residual, ids, rng, call=step)
        for w, d in zip(block.proj + block.vocab, dproj + dvocab):
            w -= 1.0 * d
        print(f"step {step}: loss {loss.item():.4f}", flush=True)
    requests = torch.tensor([0] * 7 + [2] * 5 + [-1] + [3] * 3, device="cuda")
    out = serve(block, x[:len(requests)], requests, temperature=0.8)
    for row in (0, 7, 12, 13):
        print(f"adapter {requests[row].item():2d}: tokens {out.top_ids[row].tolist()}, "
              f"log probabilities {[round(v, 2) for v in out.top_logprobs[row].tolist()]}")


if __name__ == "__main__":
    main()
