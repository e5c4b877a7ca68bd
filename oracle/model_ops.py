"""The operators around an AllReduce in 64 bits, from their definitions, with
bounds on what fp32 arithmetic may add.

numpy only; shares no code with the GPU path.  Inputs are the payload's exact
values as float64 arrays.  Each function returns its results and, for the
computed numbers, a bound on the absolute error of an evaluation that keeps
sums in fp32 and rounds the result to the payload type once: u = 2^-24 is
fp32's unit roundoff, and a sum of n terms errs by at most n u times the sum
of their magnitudes.
"""
import numpy as np

U = 2.0 ** -24
# half a unit in the last place, relative, of the payload types: 2^-p for p
# significant bits, 24 and 8
ROUND = {"float32": U, "bfloat16": 2.0 ** -8}


def philox_fields(seed, offset, count, start=0):
    """16 random bits of the elements from `start` (a multiple of 8) on: Philox4x32 with 7 rounds (Salmon,
    Moraes, Dror and Shaw, 2011), key = seed, counter = (element // 8, offset)."""
    out = []
    for n in range(start // 8, start // 8 + (count + 7) // 8):
        c = [n & 0xFFFFFFFF, n >> 32, offset & 0xFFFFFFFF, (offset >> 32) & 0xFFFFFFFF]
        k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
        for _ in range(7):
            a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
            k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
        for w in c:
            out += [w & 0xFFFF, w >> 16]
    return np.array(out[:count], dtype=np.int64)


def keep_factor(seed, offset, count, p):
    """Dropout's factor of every element: 0 or 65536 / (65536 - cut)."""
    cut = int(np.rint(p * 65536))
    if cut == 65536:
        return np.zeros(count)
    return (philox_fields(seed, offset, count) >= cut) * (65536.0 / (65536.0 - cut))


def dropout(xs, residual, factor, dtype):
    """(y, bound): residual + factor * sum of xs."""
    total, size = xs.sum(axis=0), np.abs(xs).sum(axis=0)
    y = np.where(factor > 0, total * factor, 0.0)
    err = factor * size * (len(xs) + 2) * U
    if residual is not None:
        y = y + residual
        err = err + (np.abs(residual) + np.abs(y)) * U
    return y, err + (np.abs(y) + err) * ROUND[dtype]


def logprobs(x, ids, scale, ntop):
    """Of logits [rows, vocabulary]: a dict of logprob, entropy, lse, top_ids,
    top_logprobs and of bounds "<name>_bound".  NaN where the definition says so."""
    rows, vocab = x.shape
    scale = float(np.float32(scale))
    out = {k: np.zeros(rows) for k in ("logprob", "entropy", "lse", "logprob_bound", "entropy_bound", "lse_bound")}
    out["top_ids"] = np.full((rows, ntop), -1, dtype=np.int64)
    out["top_logprobs"] = np.full((rows, ntop), -np.inf)
    out["top_bound"] = np.zeros((rows, ntop))
    for i in range(rows):
        z = x[i] * scale
        with np.errstate(invalid="ignore"):
            m = np.max(z)
            if m == -np.inf:
                lse, ent, logp, mean = -np.inf, 0.0, np.full(vocab, -np.inf), 0.0
            else:
                e = np.exp(z - m)
                lse = m + np.log(e.sum())
                logp = (z - m) - np.log(e.sum())
                p = np.exp(logp)
                ent = -np.sum(np.where(p > 0, p * np.where(p > 0, logp, 0.0), 0.0)) if np.isfinite(m) else np.nan
                mean = float(np.sum(np.where(p > 0, p * np.abs(np.where(p > 0, z - m, 0.0)), 0.0)))
        if np.isnan(x[i]).any():
            lse = ent = np.nan
            logp = np.full(vocab, np.nan)
        near = np.abs(z[np.isfinite(z)])
        near = near[near < 1e30]
        big = near.max() if near.size else 0.0
        # z and its distance from the maximum: 3 roundings of numbers up to
        # 2 |z|; exp2 and log2 to 2 units; a thread adds every 256th token (and
        # the partial sums of 64 lanes, 4 waves and the parts of a row)
        rel = (vocab / 256 + 300) * U + 8 * U * (1 + 2 * big)
        last = 4 * U * (abs(lse) if np.isfinite(lse) else 0.0)
        out["lse"][i], out["entropy"][i] = lse, ent
        out["lse_bound"][i] = rel + last
        out["entropy_bound"][i] = 4 * rel * (1 + mean)
        ok = 0 <= ids[i] < vocab
        out["logprob"][i] = logp[ids[i]] if ok else 0.0
        out["logprob_bound"][i] = (rel + 4 * U * abs(logp[ids[i]]) if ok and np.isfinite(logp[ids[i]]) else 0.0)
        order = np.lexsort((np.arange(vocab), -np.where(np.isnan(x[i]), -np.inf, x[i])))
        order = [j for j in order if x[i, j] > -np.inf][:ntop]
        for k, j in enumerate(order):
            out["top_ids"][i, k] = j
            out["top_logprobs"][i, k] = logp[j]
            out["top_bound"][i, k] = rel + 4 * U * abs(logp[j]) if np.isfinite(logp[j]) else 0.0
    return out


def logprobs_backward(x, ids, lse, entropy, g, h, l, scale, dtype):
    """(gradient [rows, vocabulary], bound) for the fp32 lse and entropy given."""
    scale = float(np.float32(scale))
    rows, vocab = x.shape
    grad, bound = np.zeros_like(x), np.zeros_like(x)
    for i in range(rows):
        if lse[i] == -np.inf:
            continue
        z = x[i] * scale
        logp = z - lse[i]
        p = np.exp(logp)
        gi = g[i] if 0 <= ids[i] < vocab else 0.0
        finite = np.where(p > 0, logp, 0.0)
        d = p * (l[i] - gi - h[i] * (finite + entropy[i]))
        # logp errs by the roundings of z, its own and that of its product with
        # log2 e; the weight by three roundings of its terms
        off = p * U * (16 + 8 * np.abs(finite) + 4 * np.where(p > 0, np.abs(z), 0.0)) * (abs(l[i]) + abs(gi) + abs(h[i]) * (np.abs(finite) + abs(entropy[i])))
        if 0 <= ids[i] < vocab:
            d[ids[i]] += gi
            off[ids[i]] += abs(gi) * 4 * U
        grad[i] = d * scale
        bound[i] = off * scale + (np.abs(grad[i]) + off * scale) * ROUND[dtype] + 1e-37
    return grad, bound


def adapters(xs, partials, downs, up, ids, scales, dtype):
    """(y, bound): sum of partials + scale * B (sum of A x) of each token's adapter."""
    y = partials.sum(axis=0)
    bound = np.abs(partials).sum(axis=0) * len(partials) * U
    inner = sum(x.shape[1] for x in xs)
    n, rank = up.shape[0], up.shape[2]
    for t, a in enumerate(ids):
        if not 0 <= a < n:
            continue
        h, size = np.zeros(rank), np.zeros(rank)
        for x, w in zip(xs, downs):
            h += w[a] @ x[t]
            size += np.abs(w[a]) @ np.abs(x[t])
        s = abs(scales[a])
        y[t] += scales[a] * (up[a] @ h)
        # the matrix units' sums may truncate: 2 u a term; h enters the second
        # product with 16 bits of its mantissa at least
        off_h = size * (inner + 64) * 2 * U + np.abs(h) * (2.0 ** -16 + (rank + 8) * 2 * U)
        bound[t] += s * (np.abs(up[a]) @ off_h)
    bound = bound + np.abs(y) * 4 * U
    return y, bound + (np.abs(y) + bound) * ROUND[dtype]
