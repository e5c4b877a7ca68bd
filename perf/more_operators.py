"""What a model split over N virtual ranks computes around its other
AllReduces, as cases to be measured: the embedding of tokens from a table split
by vocabulary (and its gradient), the norms before and after a block with its
gate and residual scale (and their gradient), and a row-parallel projection in
8-bit integers with a scale for each token and channel.

``run`` computes each in plain torch operations in 32 bits, or through
``ring_all_reduce_channelmask_amd`` where ``own`` is true; ``exact`` computes
the definition in 64 bits.
"""
import torch

own = False

TYPES = {"bfloat16": torch.bfloat16, "float32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one request's next token enters the model
        dict(name="embedding 1 token", op="embedding", dtype="bfloat16", ranks=4, copies=4, tokens=1, vocab=32003, width=7168, scale=1.0),
        # a prompt batch
        dict(name="embedding 4096 tokens", op="embedding", dtype="bfloat16", ranks=4, copies=4, tokens=4096, vocab=131072, width=7168, scale=1.0),
        # a small batch in 32 bits, an odd width and a scaled embedding
        dict(name="embedding gradient 333 tokens fp32", op="embedding_backward", dtype="float32", ranks=3, copies=3, tokens=333, vocab=8003, width=1001, scale=31.6),
        # a training batch of many short words
        dict(name="embedding gradient 65536 tokens", op="embedding_backward", dtype="bfloat16", ranks=4, copies=1, tokens=65536, vocab=131072, width=2048, scale=1.0),
        # one token behind a block
        dict(name="norms 1 row", op="norms", dtype="bfloat16", ranks=4, copies=4, rows=1, width=7168, post=True, groups=1, pre=True, residual=True, save=False, scale=1.0),
        # a training batch: what the gradient needs is kept
        dict(name="norms 4096 rows", op="norms", dtype="bfloat16", ranks=4, copies=4, rows=4096, width=7168, post=True, groups=1, pre=True, residual=True, save=True, scale=0.8),
        # 8 sequences of 13 positions with a gate each, 32 bits, an odd width
        dict(name="norms gradient 104 rows fp32", op="norms_backward", dtype="float32", ranks=4, copies=1, rows=104, width=2051, post=True, groups=8, pre=True, residual=True, scale=1.0),
        # the training batch's gradient, four ranks' gradients of the normed copies
        dict(name="norms gradient 4096 rows", op="norms_backward", dtype="bfloat16", ranks=4, copies=1, rows=4096, width=7168, post=True, groups=1, pre=True, residual=True, scale=0.8),
        # one request's token through an 8-bit projection
        dict(name="projection 1 token", op="projection", dtype="bfloat16", ranks=4, copies=4, tokens=1, inner=7168, outer=7168, residual=True),
        # 104 requests decoding
        dict(name="projection 104 tokens", op="projection", dtype="bfloat16", ranks=4, copies=4, tokens=104, inner=7168, outer=7168, residual=True),
        # a ragged batch in 32 bits, odd sizes
        dict(name="projection 1000 tokens fp32", op="projection", dtype="float32", ranks=3, copies=3, tokens=1000, inner=5001, outer=2051, residual=False),
        # a prompt batch
        dict(name="projection 4096 tokens", op="projection", dtype="bfloat16", ranks=4, copies=4, tokens=4096, inner=7168, outer=7168, residual=False),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even in its logarithm."""
    hi = max(lo, hi)
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["embedding", "embedding_backward", "norms", "norms_backward", "projection", "projection"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    size = 2 if dtype == "bfloat16" else 4
    ranks = rng.choice([1, 2, 3, 4, 8])
    case = dict(op=op, dtype=dtype, ranks=ranks, copies=rng.choice([1, ranks]))
    if op == "embedding":
        width = _log(rng, 100, 7168)
        case.update(tokens=_log(rng, 1, min(65536, (1 << 28) // size // width)), vocab=_log(rng, 1000, 131072), width=width, scale=rng.choice([1.0, 22.6]))
    elif op == "embedding_backward":
        width = _log(rng, 100, 7168)
        case.update(tokens=_log(rng, 1, min(65536, (1 << 28) // size // width // case["copies"])), vocab=_log(rng, 1000, min(131072, (1 << 28) // width)), width=width,
                    scale=rng.choice([1.0, 22.6]))
    elif op in ("norms", "norms_backward"):
        width = _log(rng, 100, 8192)
        rows = _log(rng, 1, (1 << 28) // size // width // (ranks + case["copies"] + 1))
        groups = rng.choice([0, 1, 1, max(d for d in range(1, 17) if rows % d == 0), rows])
        case.update(rows=rows, width=width, groups=groups, post=rng.random() < 0.6, pre=rng.random() < 0.8, residual=rng.random() < 0.9, scale=rng.choice([1.0, 0.8]))
        if op == "norms":
            case["save"] = rng.random() < 0.5
    else:
        inner, outer = _log(rng, 500, 7168), _log(rng, 500, 7168)
        case.update(ranks=min(ranks, 4), copies=min(case["copies"], 4), tokens=_log(rng, 1, 4096 * 2 // size), inner=inner, outer=outer, residual=rng.random() < 0.5)
    return case


def _parts(total, ranks):
    """`total` cut into near-equal parts, one a rank."""
    return [total // ranks + (r < total % ranks) for r in range(ranks)]


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _tokens(g, n, vocab):
    """Ids as a text has them: the n-th most frequent with a frequency of 1/n,
    in no order of the vocabulary; one position in 50 is padding."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    ids = torch.randperm(vocab, generator=g, device="cuda")[(torch.pow(float(vocab), u).long() - 1).clamp(0, vocab - 1)]
    pad = torch.rand(n, generator=g, device="cuda") < 0.02
    return torch.where(pad, torch.full_like(ids, -1), ids) if n > 8 else ids


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t, s, op = TYPES[case["dtype"]], dict(case), case["op"]
    if op in ("embedding", "embedding_backward"):
        T, V, D = case["tokens"], case["vocab"], case["width"]
        s["ids"] = _tokens(g, T, V)
        if op == "embedding":
            s["tables"] = [_randn(g, v, D).to(t) for v in _parts(V, case["ranks"])]
            s["recvs"] = [torch.empty(T, D, dtype=t, device="cuda") for _ in range(case["copies"])]
        else:
            s["grads"] = [(_randn(g, T, D) * 0.1).to(t) for _ in range(case["copies"])]
            s["dtables"] = [torch.empty(v, D, dtype=t, device="cuda") for v in _parts(V, case["ranks"])]
        return s
    if op in ("norms", "norms_backward"):
        R, D, G = case["rows"], case["width"], case["groups"]
        partials = [_randn(g, R, D).to(t) for _ in range(case["ranks"])]
        s["resid"] = (2 * _randn(g, R, D)).to(t) if case["residual"] else None
        s["post_w"] = (1 + 0.2 * _randn(g, D)).to(t) if case["post"] else None
        s["pre_w"] = (1 + 0.2 * _randn(g, D)).to(t) if case["pre"] else None
        s["gate"] = (0.5 + 0.3 * _randn(g, G, D)).to(t) if G else None
        empty = torch.empty(R, D, dtype=t, device="cuda")
        if op == "norms":
            s["partials"] = partials
            s["hidden"] = torch.empty_like(empty)
            s["outs"] = [torch.empty_like(empty) for _ in range(case["copies"])] if case["pre"] else []
            s["total"] = torch.empty_like(empty) if case["save"] else None
            return s
        # what the forward pass kept
        s["partials"] = partials
        total, hidden, _ = _plain_norms(s)
        s["total"], s["hidden"] = total.to(t), hidden.to(t)
        del s["partials"], s["resid"]
        s["grad_hidden"] = (0.1 * _randn(g, R, D)).to(t)
        s["grad_outs"] = [(0.1 * _randn(g, R, D)).to(t) for _ in range(case["ranks"])] if case["pre"] else []
        s["dpartials"] = [torch.empty_like(empty) for _ in range(case["copies"])]
        s["dresid"] = torch.empty_like(empty) if case["residual"] else None
        for w, d in (("post_w", "dpost_w"), ("pre_w", "dpre_w"), ("gate", "dgate")):
            s[d] = None if s[w] is None else torch.empty_like(s[w])
        return s
    T, K, D = case["tokens"], case["inner"], case["outer"]
    s["xs"] = [_randn(g, T, k).to(t) for k in _parts(K, case["ranks"])]
    for x in s["xs"]:  # a few channels far above the others
        x[:, torch.randint(0, x.shape[1], (4,), generator=g, device="cuda")] *= 8
    w = _randn(g, D, K) / K ** 0.5
    most = w.abs().amax(1)
    w = torch.round(w * (127 / most)[:, None]).to(torch.int8)
    s["weights"] = [part.contiguous() for part in w.split(_parts(K, case["ranks"]), 1)]
    s["w_scales"] = most / 127
    s["resid"] = _randn(g, T, D).to(t) if case["residual"] else None
    s["recvs"] = [torch.empty(T, D, dtype=t, device="cuda") for _ in range(case["copies"])]
    return s


def _plain_embedding(s):
    out, lo = 0.0, 0
    for table in s["tables"]:
        mine = (s["ids"] >= lo) & (s["ids"] < lo + table.shape[0])
        rows = table[(s["ids"] - lo).clamp(0, table.shape[0] - 1)].float()
        out = out + torch.where(mine[:, None], rows, torch.zeros_like(rows))
        lo += table.shape[0]
    out = (out * s["scale"]).to(s["tables"][0].dtype)
    return [out.clone() for _ in s["recvs"]]


def _plain_embedding_backward(s):
    total = s["grads"][0].float()
    for d in s["grads"][1:]:
        total = total + d.float()
    given = s["ids"] >= 0
    sizes = [d.shape[0] for d in s["dtables"]]
    dense = torch.zeros(sum(sizes), total.shape[1], device=total.device)
    dense.index_add_(0, s["ids"].clamp(min=0), total * given[:, None])
    return [part.contiguous() for part in (dense * s["scale"]).to(s["grads"][0].dtype).split(sizes)]


def _spread(gate, rows):
    """The gate of every row: row i has that of group i // (rows / groups)."""
    return gate.float().repeat_interleave(rows // gate.shape[0], 0)


def _rstd(x):
    return torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)


def _plain_norms(s):
    """The sum of the partials, the residual stream and its norm, in 32 bits."""
    total = s["partials"][0].float()
    for p in s["partials"][1:]:
        total = total + p.float()
    u = total if s["post_w"] is None else total * _rstd(total) * s["post_w"].float()
    if s["gate"] is not None:
        u = u * _spread(s["gate"], total.shape[0])
    hidden = u if s["resid"] is None else s["scale"] * s["resid"].float() + u
    return total, hidden, None if s["pre_w"] is None else hidden * _rstd(hidden) * s["pre_w"].float()


def _plain_norms_backward(s):
    t, out = s["total"].dtype, {}
    d = s["grad_hidden"].float()
    if s["pre_w"] is not None:
        h = s["hidden"].float()
        dn = s["grad_outs"][0].float()
        for g in s["grad_outs"][1:]:
            dn = dn + g.float()
        r = _rstd(h)
        out["dpre_w"] = (dn * h * r).sum(0).to(t)
        dn = dn * s["pre_w"].float()
        d = d + r * (dn - h * (r * r) * (dn * h).mean(1, keepdim=True))
    if s["residual"]:
        out["dresid"] = (s["scale"] * d).to(t)
    total, v = s["total"].float(), d
    q = 1.0 if s["post_w"] is None else _rstd(total)
    if s["gate"] is not None:
        u = total if s["post_w"] is None else total * q * s["post_w"].float()
        out["dgate"] = (d * u).reshape(s["gate"].shape[0], -1, total.shape[1]).sum(1).to(t)
        v = d * _spread(s["gate"], total.shape[0])
    if s["post_w"] is not None:
        out["dpost_w"] = (v * total * q).sum(0).to(t)
        v = v * s["post_w"].float()
        v = q * (v - total * (q * q) * (v * total).mean(1, keepdim=True))
    v = v.to(t)
    out["dpartials"] = [v.clone() for _ in s["dpartials"]]
    return out


def _plain_projection(s):
    y = 0.0
    most = torch.stack([x.abs().amax(1, keepdim=True).float() for x in s["xs"]]).amax(0)
    for x, w in zip(s["xs"], s["weights"]):
        # 64 bits: a value next to the middle of two whole numbers
        q = torch.round(x.double() * 127 / most.double()) if x.dtype == torch.float32 else torch.round(x.float() * 127 / most)
        y = y + q.float() @ w.float().T
    y = y * (most / 127 * s["w_scales"])
    if s["resid"] is not None:
        y = s["resid"].float() + y
    y = y.to(s["xs"][0].dtype)
    return [y.clone() for _ in s["recvs"]]


def run(state):
    s, op = state, state["op"]
    if not own:
        if op == "embedding":
            return _plain_embedding(s)
        if op == "embedding_backward":
            return _plain_embedding_backward(s)
        if op == "norms":
            total, hidden, y = _plain_norms(s)
            t = s["partials"][0].dtype
            y = None if y is None else y.to(t)
            return {"hidden": hidden.to(t), "outs": [y.clone() for _ in s["outs"]], "total": total.to(t) if s["save"] else None}
        if op == "norms_backward":
            return _plain_norms_backward(s)
        return _plain_projection(s)
    import ring_all_reduce_channelmask_amd as rar
    if op == "embedding":
        rar.embedding_allreduce(s["tables"], s["ids"], s["recvs"], scale=s["scale"])
        return s["recvs"]
    if op == "embedding_backward":
        rar.embedding_allreduce_backward(s["grads"], s["ids"], s["dtables"], scale=s["scale"])
        return s["dtables"]
    if op == "norms":
        rar.norm_allreduce(s["partials"], [s["hidden"]], s["outs"], residual=s["resid"], residual_scale=s["scale"], post_weight=s["post_w"], gate=s["gate"],
                           pre_weight=s["pre_w"], eps=EPS, total=s["total"])
        return {"hidden": s["hidden"], "outs": s["outs"], "total": s["total"]}
    if op == "norms_backward":
        rar.norm_allreduce_backward([s["grad_hidden"]], s["grad_outs"], s["dpartials"], total=s["total"], hidden=s["hidden"], residual_scale=s["scale"],
                                    post_weight=s["post_w"], gate=s["gate"], pre_weight=s["pre_w"], eps=EPS, dresidual=s["dresid"], dpost_weight=s["dpost_w"],
                                    dgate=s["dgate"], dpre_weight=s["dpre_w"])
        return {k: s[k] for k in ("dpre_w", "dresid", "dgate", "dpost_w") if s[k] is not None} | {"dpartials": s["dpartials"]}
    quantized, scales = rar.quantize_rows(s["xs"])
    rar.int8_projection_allreduce(quantized, scales, s["weights"], s["w_scales"], s["recvs"], residual=s["resid"])
    return s["recvs"]


def work(case):
    size, op = 2 if case["dtype"] == "bfloat16" else 4, case["op"]
    N, C = case["ranks"], case["copies"]
    if op == "embedding":
        n = case["tokens"] * case["width"]
        return {"bytes": 8 * case["tokens"] + n * size * (1 + C), "flops": n}
    if op == "embedding_backward":
        n = case["tokens"] * case["width"]
        return {"bytes": 8 * case["tokens"] + size * (n * C + case["vocab"] * case["width"]), "flops": n * (C + 1)}
    if op in ("norms", "norms_backward"):
        n, vectors = case["rows"] * case["width"], case["width"] * (case["post"] + case["pre"] + case["groups"])
        if op == "norms":
            moved = N + case["residual"] + 1 + C * case["pre"] + case["save"]
            return {"bytes": size * (n * moved + vectors), "flops": n * (N + 10)}
        moved = 1 + (N + 1) * case["pre"] + (case["post"] or case["groups"] > 0) + C + case["residual"]
        return {"bytes": size * (n * moved + 2 * vectors), "flops": n * (N + 25)}
    T, K, D = case["tokens"], case["inner"], case["outer"]
    return {"bytes": T * K * size + K * D + 4 * D + T * D * size * (C + case["residual"]), "flops": 2 * T * K * D}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "embedding":
        whole = torch.cat(s["tables"])
        rows = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device="cuda")
        at = torch.nonzero(s["ids"] >= 0)[:, 0]
        rows[at] = whole[s["ids"][at]].double() * case["scale"]
        return [rows] * case["copies"]
    if op == "embedding_backward":
        V, D = case["vocab"], case["width"]
        at = torch.nonzero(s["ids"] >= 0)[:, 0]
        total = torch.zeros(V, D, dtype=torch.float64, device="cuda")
        for d in s["grads"]:
            total.index_put_((s["ids"][at],), d[at].double(), accumulate=True)
        total *= case["scale"]
        return list(total.split(_parts(V, case["ranks"])))
    if op in ("norms", "norms_backward"):
        R, D, G = case["rows"], case["width"], case["groups"]

        def leaf(k):
            return None if s[k] is None else s[k].double().requires_grad_()

        def norm(x, w):
            return torch.nn.functional.normalize(x, dim=1, eps=0.0) * D ** 0.5 * w / (1 + EPS / (x * x).mean(1, keepdim=True)).sqrt()
        post_w, pre_w, gate = leaf("post_w"), leaf("pre_w"), leaf("gate")

        def stream(total, resid):
            u = total if post_w is None else norm(total, post_w)
            if gate is not None:
                u = (u.view(G, R // G, D) * gate[:, None]).view(R, D)
            return u if resid is None else u + case["scale"] * resid
        if op == "norms":
            with torch.no_grad():
                total = torch.stack([p.double() for p in s["partials"]]).sum(0)
                hidden = stream(total, None if s["resid"] is None else s["resid"].double())
                y = norm(hidden, pre_w) if case["pre"] else None
            return {"hidden": hidden, "outs": [y] * len(s["outs"]), "total": total if case["save"] else None}
        d, out = s["grad_hidden"].double(), {}
        if case["pre"]:
            h = s["hidden"].double().requires_grad_()
            dn = torch.stack([x.double() for x in s["grad_outs"]]).sum(0)
            more, out["dpre_w"] = torch.autograd.grad(norm(h, pre_w), (h, pre_w), dn)
            d = d + more
        total = s["total"].double().requires_grad_()
        resid = torch.zeros(R, D, dtype=torch.float64, device="cuda", requires_grad=True) if case["residual"] else None
        of = {"total": total, "dresid": resid, "dgate": gate, "dpost_w": post_w}
        of = {k: v for k, v in of.items() if v is not None}
        got = dict(zip(of, torch.autograd.grad(stream(total, resid), list(of.values()), d)))
        out.update({k: got[k] for k in ("dresid", "dgate", "dpost_w") if k in got})
        out["dpartials"] = [got["total"]] * case["copies"]
        return out
    y = torch.zeros(case["tokens"], case["outer"], dtype=torch.float64, device="cuda")
    most = torch.cat(s["xs"], 1).double().abs().max(1)[0]
    for x, w in zip(s["xs"], s["weights"]):
        y += (x.double() * 127 / most[:, None]).round() @ w.double().T
    y *= (most / 127)[:, None] * s["w_scales"].double()
    if case["residual"]:
        y += s["resid"].double()
    return [y] * case["copies"]
