"""The operators around an AllReduce in a model split over N virtual ranks, as
cases to be measured: token log probabilities over a vocabulary split over the
ranks (and their gradient), the AllReduce with dropout and a residual (and its
gradient), and the AllReduce of a row-parallel projection with low-rank
adapters of many requests.

``run`` computes each in plain torch operations in 32 bits, or through
``ring_all_reduce_channelmask_amd`` where ``own`` is true; ``exact`` computes
the definition in 64 bits.
"""
import numpy as np
import torch

own = False

TYPES = {"bfloat16": torch.bfloat16, "float32": torch.float32}


def listed():
    return [
        # one request's next token: the most probable 20 of a small vocabulary
        dict(name="logprobs 1 row top 20", op="logprobs", dtype="bfloat16", ranks=4, rows=1, vocab=32003, pad=0, ntop=20, masked=False, scale=1.0),
        # a batch of decoding requests under a grammar that masks half the vocabulary, at a temperature
        dict(name="logprobs 104 rows masked top 5", op="logprobs", dtype="bfloat16", ranks=8, rows=104, vocab=131075, pad=5, ntop=5, masked=True, scale=1.25),
        # a training batch's loss
        dict(name="logprobs 4096 rows", op="logprobs", dtype="bfloat16", ranks=4, rows=4096, vocab=131072, pad=0, ntop=0, masked=False, scale=1.0),
        # a policy's update with an entropy bonus, logits kept in 32 bits
        dict(name="logprobs gradient 333 rows fp32", op="logprobs_backward", dtype="float32", ranks=4, rows=333, vocab=32003, pad=0, masked=False, scale=1.25, bonus=True),
        # the training batch's gradient
        dict(name="logprobs gradient 4096 rows", op="logprobs_backward", dtype="bfloat16", ranks=8, rows=4096, vocab=131072, pad=0, masked=False, scale=1.0, bonus=False),
        # 104 tokens of 7168 after a row-parallel projection
        dict(name="dropout 104x7168", op="dropout", dtype="bfloat16", ranks=4, copies=4, count=104 * 7168, p=0.1, residual=True),
        # 64 MiB a rank, the AllReduce benchmark's size
        dict(name="dropout 16M fp32", op="dropout", dtype="float32", ranks=4, copies=4, count=1 << 24, p=0.1, residual=True),
        # one token's gradient, one copy of it going back to 4 ranks
        dict(name="dropout gradient 7168", op="dropout_backward", dtype="bfloat16", ranks=4, copies=1, count=7168, p=0.1, residual=True),
        # 8 ranks of 64 MiB, the bf16 benchmark's size
        dict(name="dropout gradient 32M", op="dropout_backward", dtype="bfloat16", ranks=8, copies=8, count=1 << 25, p=0.25, residual=False),
        # one request decoding with its adapter
        dict(name="adapters 1 token", op="adapters", dtype="bfloat16", ranks=4, copies=4, tokens=1, requests=1, inner=7168, outer=7168, rank=16, adapters=8),
        # 104 requests decoding, each with one of 64 adapters
        dict(name="adapters 104 tokens", op="adapters", dtype="bfloat16", ranks=4, copies=4, tokens=104, requests=104, inner=7168, outer=7168, rank=16, adapters=64),
        # a prompt batch: 4096 tokens of 7 requests
        dict(name="adapters 4096 tokens", op="adapters", dtype="bfloat16", ranks=4, copies=4, tokens=4096, requests=7, inner=7168, outer=7168, rank=64, adapters=8),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even in its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_backward", "dropout", "dropout_backward", "adapters"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    size = 2 if dtype == "bfloat16" else 4
    ranks = rng.choice([1, 2, 3, 4, 8])
    if op in ("logprobs", "logprobs_backward"):
        vocab = _log(rng, 1000, 150000)
        most = (1 << 29) * 2 // size // vocab  # as many bytes as the largest listed case
        case = dict(op=op, dtype=dtype, ranks=ranks, rows=_log(rng, 1, min(4096, most)), vocab=vocab, pad=rng.choice([0, 0, 3, 8]),
                    masked=rng.random() < 0.3, scale=rng.choice([1.0, 0.7, 1.25]))
        if op == "logprobs":
            case["ntop"] = rng.choice([0, 0, 1, 5, 20, 32])
        else:
            case["bonus"] = rng.random() < 0.5
        return case
    if op in ("dropout", "dropout_backward"):
        copies = rng.choice([1, ranks])
        most = (1 << 25) * 2 // size * 16 // (ranks + copies + 1)
        return dict(op=op, dtype=dtype, ranks=ranks, copies=copies, count=_log(rng, 2000, min(1 << 25, most)), p=rng.choice([0.05, 0.1, 0.25, 0.5]),
                    residual=rng.random() < 0.6)
    tokens = _log(rng, 1, 4096)
    adapters = _log(rng, 1, 64)
    return dict(op=op, dtype=dtype, ranks=min(ranks, 4), copies=rng.choice([1, min(ranks, 4)]), tokens=tokens, requests=_log(rng, 1, min(tokens, 200)),
                inner=_log(rng, 500, 7168) * size // 4, outer=_log(rng, 500, 7168) * size // 4, rank=rng.choice([8, 16, 32, 64, 12]), adapters=adapters)


def _parts(total, ranks):
    """`total` cut into near-equal parts, one a rank."""
    return [total // ranks + (r < total % ranks) for r in range(ranks)]


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi, (n,), generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t, s = TYPES[case["dtype"]], dict(case)
    if case["op"] in ("logprobs", "logprobs_backward"):
        rows, vocab = case["rows"], case["vocab"]
        # logits of a trained model: most of them moderate, a few tokens of each row far above
        x = _randn(g, rows, vocab).mul_(2.0)
        for _ in range(4):
            x.scatter_(1, torch.randint(0, vocab, (rows, 1), generator=g, device="cuda"), 6 + 3 * _randn(g, rows, 1))
        if case["masked"]:
            x.masked_fill_(torch.rand(rows, vocab, generator=g, device="cuda") < 0.5, float("-inf"))
            x[:, vocab // 2] = 1.0
        s["ids"] = _ints(g, 0, vocab, rows)
        if rows > 8:
            s["ids"][3] = -1  # a padded position
        if case["masked"]:
            s["ids"] = torch.where(s["ids"] < 0, s["ids"], torch.full_like(s["ids"], vocab // 2))
        s["shards"] = []
        for part in x.split(_parts(vocab, case["ranks"]), 1):
            held = torch.empty(rows, part.shape[1] + case["pad"], dtype=t, device="cuda")[:, : part.shape[1]]
            s["shards"].append(held.copy_(part))
        if case["op"] == "logprobs_backward":
            # what the forward pass kept
            lse, entropy = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
            for r0 in range(0, rows, 512):
                z = torch.cat([h[r0:r0 + 512] for h in s["shards"]], 1).double() * case["scale"]
                l = torch.logsumexp(z, 1)
                lse[r0:r0 + 512] = l
                entropy[r0:r0 + 512] = l - (torch.exp(z - l[:, None]) * z.clamp(min=-1e30)).sum(1)
            s["lse"], s["entropy"] = lse, entropy
            s["grad_logprob"] = _randn(g, rows)
            s["grad_entropy"] = 0.1 * _randn(g, rows) if case["bonus"] else None
            s["grads"] = [torch.empty_like(h, memory_format=torch.contiguous_format) for h in s["shards"]]
        return s
    if case["op"] in ("dropout", "dropout_backward"):
        # (seed, offset) of the generator, as a training program keeps them
        s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device="cuda")
        back = case["op"] == "dropout_backward"
        n_in, n_out = (case["copies"], case["ranks"]) if back else (case["ranks"], case["copies"])
        s["inputs"] = [_randn(g, case["count"]).to(t) for _ in range(n_in)]
        s["outputs"] = [torch.empty(case["count"], dtype=t, device="cuda") for _ in range(n_out)]
        s["resid"] = None
        if case["residual"]:
            s["resid"] = torch.empty(case["count"], dtype=t, device="cuda") if back else _randn(g, case["count"]).to(t)
        return s
    T, K, D, R, A = (case[k] for k in ("tokens", "inner", "outer", "rank", "adapters"))
    s["xs"] = [_randn(g, T, k).to(t) for k in _parts(K, case["ranks"])]
    s["partials"] = [_randn(g, T, D).to(t) for _ in range(case["ranks"])]
    s["downs"] = [(_randn(g, A, R, k) / K ** 0.5).to(t) for k in _parts(K, case["ranks"])]
    s["up"] = (_randn(g, A, D, R) / R ** 0.5).to(t)
    s["scales"] = 0.5 + torch.rand(A, generator=g, device="cuda")
    # a request's tokens stand together; one request in nine or so has no adapter
    of = _ints(g, -1 if case["requests"] > 8 else 0, A, case["requests"])
    cuts = torch.sort(_ints(g, 0, T, case["requests"] - 1))[0]
    where = torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)
    s["ids"] = of[where] if case["requests"] < T else of[torch.arange(T, device="cuda")]
    s["recvs"] = [torch.empty(T, D, dtype=t, device="cuda") for _ in range(case["copies"])]
    return s


def _keep(rng, count, p):
    """Dropout's factor of every element: 0, or 1 / (1 - p) with p in steps of
    2^-16.  Philox4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw, 2011),
    key = seed, counter = (element // 8, offset), 16 bits an element."""
    low = 0xFFFFFFFF
    n = torch.arange((count + 7) // 8, dtype=torch.int64, device=rng.device)
    a, b, c, d = n & low, n >> 32, (rng[1] & low).expand_as(n), ((rng[1] >> 32) & low).expand_as(n)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    for _ in range(7):
        u, v = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = ((v >> 32) & low) ^ b ^ k0, v & low, ((u >> 32) & low) ^ d ^ k1, u & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    fields = torch.stack([a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16, c & 0xFFFF, c >> 16, d & 0xFFFF, d >> 16], 1).reshape(-1)[:count]
    cut = int(round(p * 65536))
    return (fields >= cut).float() * (65536.0 / (65536.0 - cut))


def _plain_logprobs(s):
    x = torch.cat([h.float() for h in s["shards"]], 1)
    z = x * s["scale"]
    m = z.max(1, keepdim=True)[0]
    d = z - m
    e = torch.exp(d)
    total = e.sum(1)
    lse = m[:, 0] + torch.log(total)
    entropy = torch.log(total) - (e * d.clamp(min=-1e30)).sum(1) / total
    given = z.gather(1, s["ids"].clamp(min=0)[:, None])[:, 0] - lse
    out = {"logprob": torch.where(s["ids"] < 0, torch.zeros_like(given), given), "entropy": entropy, "lse": lse}
    if s["ntop"]:
        # the order of the logits, equal ones by the lower id: one whole number for both
        bits = (x + 0.0).view(torch.int32).long()  # -0 and 0 are equal
        order = torch.where(bits < 0, -0x80000000 - bits - 1, bits)
        key = (order << 32) + (0xFFFFFFFF - torch.arange(x.shape[1], device=x.device))
        ids = 0xFFFFFFFF - (torch.topk(key, s["ntop"], 1)[0] & 0xFFFFFFFF)
        out["top_ids"], out["top_logprobs"] = ids.int(), z.gather(1, ids) - lse[:, None]
    return out


def _plain_logprobs_backward(s):
    z = torch.cat([h.float() for h in s["shards"]], 1) * s["scale"]
    logp = z - s["lse"][:, None]
    ours = torch.where(s["ids"] < 0, torch.zeros_like(s["grad_logprob"]), s["grad_logprob"])
    w = -ours[:, None]
    if s["grad_entropy"] is not None:
        w = w - s["grad_entropy"][:, None] * (logp.clamp(min=-1e30) + s["entropy"][:, None])
    grad = torch.exp(logp) * w
    grad.scatter_add_(1, s["ids"].clamp(min=0)[:, None], ours[:, None])
    return [part.contiguous() for part in (grad * s["scale"]).to(s["shards"][0].dtype).split([h.shape[1] for h in s["shards"]], 1)]


def _plain_dropout(s, back):
    total = torch.stack(s["inputs"]).float().sum(0)
    kept = total * _keep(s["rng"], s["count"], s["p"])
    t = s["inputs"][0].dtype
    if back:
        given = kept.to(t)
        return {"dsends": [given.clone() for _ in s["outputs"]], "dresidual": total.to(t) if s["residual"] else None}
    given = (kept + s["resid"].float() if s["residual"] else kept).to(t)
    return {"recvs": [given.clone() for _ in s["outputs"]]}


def _plain_adapters(s):
    A, D, R = s["up"].shape
    x = torch.cat([v.float() for v in s["xs"]], 1)
    down = torch.cat([w.float() for w in s["downs"]], 2).reshape(A * R, -1)
    mine = (s["ids"][:, None] == torch.arange(A, device=x.device)).float() * s["scales"]
    h = (x @ down.T).reshape(-1, A, R) * mine[:, :, None]
    delta = h.reshape(-1, A * R) @ s["up"].float().transpose(1, 2).reshape(A * R, D)
    y = (torch.stack(s["partials"]).float().sum(0) + delta).to(s["up"].dtype)
    return [y.clone() for _ in s["recvs"]]


def run(state):
    s, op = state, state["op"]
    if not own:
        if op == "logprobs":
            return _plain_logprobs(s)
        if op == "logprobs_backward":
            return _plain_logprobs_backward(s)
        if op in ("dropout", "dropout_backward"):
            return _plain_dropout(s, op == "dropout_backward")
        return _plain_adapters(s)
    import ring_all_reduce_channelmask_amd as rar
    if op == "logprobs":
        r = rar.logprobs(s["shards"], s["ids"], ntop=s["ntop"], scale=s["scale"])
        out = {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse}
        if s["ntop"]:
            out["top_ids"], out["top_logprobs"] = r.top_ids, r.top_logprobs
        return out
    if op == "logprobs_backward":
        return rar.logprobs_backward(s["shards"], s["ids"], s["lse"], s["entropy"], s["grad_logprob"], grad_entropy=s["grad_entropy"],
                                     scale=s["scale"], grads=s["grads"])
    if op == "dropout":
        rar.dropout_allreduce(s["inputs"], s["outputs"], s["p"], s["rng"], residual=s["resid"])
        return {"recvs": s["outputs"]}
    if op == "dropout_backward":
        rar.dropout_allreduce_backward(s["inputs"], s["outputs"], s["p"], s["rng"], dresidual=s["resid"])
        return {"dsends": s["outputs"], "dresidual": s["resid"]}
    rar.adapter_allreduce(s["xs"], s["partials"], s["recvs"], s["downs"], s["up"], s["ids"], s["scales"])
    return s["recvs"]


def work(case):
    size = 2 if case["dtype"] == "bfloat16" else 4
    if case["op"] in ("logprobs", "logprobs_backward"):
        n = case["rows"] * case["vocab"]
        if case["op"] == "logprobs":
            return {"bytes": n * size + case["rows"] * (20 + 8 * case["ntop"]), "flops": 5 * n}
        return {"bytes": 2 * n * size + case["rows"] * (24 if case["bonus"] else 16), "flops": (8 if case["bonus"] else 5) * n}
    if case["op"] in ("dropout", "dropout_backward"):
        return {"bytes": case["count"] * size * (case["ranks"] + case["copies"] + case["residual"]), "flops": case["count"] * (case["ranks"] + 2)}
    T, K, D, R = (case[k] for k in ("tokens", "inner", "outer", "rank"))
    used = min(case["adapters"], case["requests"])
    data = T * K + T * D * (case["ranks"] + case["copies"]) + used * R * (K + D)
    return {"bytes": data * size + 8 * T, "flops": 2 * T * R * (K + D) + T * D * case["ranks"]}


def _philox_fields(seed, offset, count):
    """Every element's 16 bits, on the host."""
    m = np.uint64(0xFFFFFFFF)
    sh = np.uint64(32)
    n = np.arange((count + 7) // 8, dtype=np.uint64)
    ctr = [n & m, n >> sh, np.full_like(n, offset & 0xFFFFFFFF), np.full_like(n, (offset >> 32) & 0xFFFFFFFF)]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(7):
        lo0, lo1 = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(lo1 >> sh) ^ ctr[1] ^ np.uint64(key[0]), lo1 & m, (lo0 >> sh) ^ ctr[3] ^ np.uint64(key[1]), lo0 & m]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    return np.stack(ctr, 1).astype("<u4").view("<u2").reshape(-1)[:count]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        out = {k: [] for k in ("logprob", "entropy", "lse", "top_ids", "top_logprobs")}
        for r0 in range(0, case["rows"], 256):
            z = torch.cat([h[r0:r0 + 256].double() for h in s["shards"]], 1)
            ids = s["ids"][r0:r0 + 256]
            logp = torch.log_softmax(z * case["scale"], 1)
            out["lse"].append(torch.logsumexp(z * case["scale"], 1))
            out["entropy"].append(-torch.xlogy(logp.exp(), logp.exp()).sum(1))
            out["logprob"].append(torch.where(ids < 0, 0.0, logp[torch.arange(len(ids)), ids.clamp(min=0)]))
            if case["ntop"]:
                best = torch.sort(z, dim=1, descending=True, stable=True)[1][:, : case["ntop"]]
                out["top_ids"].append(best.int())
                out["top_logprobs"].append(logp.gather(1, best))
        return {k: torch.cat(v) for k, v in out.items() if v}
    if case["op"] == "logprobs_backward":
        rows = []
        for r0 in range(0, case["rows"], 256):
            z = torch.cat([h[r0:r0 + 256].double() for h in s["shards"]], 1) * case["scale"]
            ids, lse, ent, g = (s[k][r0:r0 + 256] for k in ("ids", "lse", "entropy", "grad_logprob"))
            g = g.double() * (ids >= 0)
            logp = z - lse.double()[:, None]
            p = logp.exp()
            d = -g[:, None] * p
            d[torch.arange(len(ids)), ids.clamp(min=0)] += g
            if s["grad_entropy"] is not None:
                d -= s["grad_entropy"][r0:r0 + 256].double()[:, None] * (torch.xlogy(p, p) + p * ent.double()[:, None])
            rows.append((d * case["scale"]).float() if case["dtype"] == "bfloat16" else d * case["scale"])
        whole = torch.cat(rows)
        return [part.contiguous() for part in whole.split(_parts(case["vocab"], case["ranks"]), 1)]
    if case["op"] in ("dropout", "dropout_backward"):
        seed64, offset = (int(v) & (2 ** 64 - 1) for v in s["rng"].tolist())
        cut = int(round(case["p"] * 65536))
        keep = torch.from_numpy((_philox_fields(seed64, offset, case["count"]) >= cut).astype(np.float64)).cuda()
        total = torch.zeros(case["count"], dtype=torch.float64, device="cuda")
        for x in s["inputs"]:
            total += x.double()
        kept = total * keep * 65536 / (65536 - cut)
        if case["op"] == "dropout_backward":
            return {"dsends": [kept] * case["ranks"], "dresidual": total if case["residual"] else None}
        return {"recvs": [kept + s["resid"].double() if case["residual"] else kept] * case["copies"]}
    y = sum(p.double() for p in s["partials"])
    for a in range(case["adapters"]):
        at = (s["ids"] == a).nonzero()[:, 0]
        if len(at):
            h = sum(x[at].double() @ w[a].double().T for x, w in zip(s["xs"], s["downs"]))
            y[at] += s["scales"][a].double() * (h @ s["up"][a].double().T)
    return [y] * case["copies"]
