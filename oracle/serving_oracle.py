"""float64 CPU oracle of the operators around the sparse-MoE layer in a decode
step: paged cache append, one-token attention, eviction by accumulated weight,
token log probabilities.  Test infrastructure only; plain numpy, token by token
where that is clearest, sharing nothing with the CUDA code.

Arrays are float64 unless named otherwise.  The cache is an array
[pages][heads][slots][dim]; token t of sequence b lies in page
table[b, t // slots], slot t % slots.
"""
import numpy as np


def cached(pool, table_row, head, n):
    """Tokens 0..n-1 of one sequence and head: [n][dim]."""
    slots = pool.shape[2]
    return np.array([pool[table_row[t // slots], head, t % slots] for t in range(n)]).reshape(n, pool.shape[3])


def append(pool_k, pool_v, table, k, v, seq, slot):
    """The pools after the tokens (k, v)[i] were written at index slot[i] of sequence seq[i]."""
    pool_k, pool_v = pool_k.copy(), pool_v.copy()
    size = pool_k.shape[2]
    for i in range(len(seq)):
        page, at = table[seq[i], slot[i] // size], slot[i] % size
        pool_k[page, :, at] = k[i]
        pool_v[page, :, at] = v[i]
    return pool_k, pool_v


def softmax_rows(s):
    """exp(s - lse) and lse of each row; a row without any score above -inf: zeros and -inf."""
    m = s.max(axis=1, initial=-np.inf, keepdims=True)
    e = np.exp(s - np.where(np.isneginf(m), 0, m))
    total = e.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (np.where(np.isneginf(m), 0, m) + np.log(total))[:, 0]
    return e / np.where(total == 0, 1, total), lse


def attend(q, pool_k, pool_v, table, lens, scale):
    """Returns a list per (sequence, kv head) of dicts: out [group][dim], lse [group], drawn [n] (probabilities
    summed over the group), and what bounds rounding: absv [group][dim] = sum p |v|, absqk = max sum |q k|,
    vsum [dim] = sum |v|, floor = the smallest sum of exp(s - max)."""
    heads = pool_k.shape[1]
    group = q.shape[1] // heads
    got = []
    for b, n in enumerate(lens):
        for h in range(heads):
            qs = q[b, h * group:(h + 1) * group]
            k, v = cached(pool_k, table[b], h, n), cached(pool_v, table[b], h, n)
            s = (qs @ k.T) * scale
            p, lse = softmax_rows(s)
            live = n > 0 and not np.any(np.isneginf(lse))
            got.append(dict(out=p @ v, lse=lse, drawn=p.sum(axis=0), absv=p @ np.abs(v), vsum=np.abs(v).sum(axis=0),
                            absqk=float((np.abs(qs) @ np.abs(k).T).max() * abs(scale)) if live else 0.0,
                            floor=float(np.exp(lse - s.max(axis=1)).min()) if live else 1.0))
    return got


def kept_tokens(weight, pos, seen, budget, sink, recent):
    """Token indexes kept of one sequence and head, ascending: kept by position first, then the larger weight (NaN
    last), then the lower index."""
    def rank(j):
        always = pos[j] < sink or pos[j] >= seen - recent
        nan = np.isnan(weight[j])
        return (0 if always else 2 if nan else 1, 0.0 if always or nan else -float(weight[j]), j)
    return sorted(sorted(range(len(weight)), key=rank)[:budget])


def evict(pool_k, pool_v, table, lens, weight, pos, seen, budget, sink, recent):
    """Pools, weights, positions and lengths after the cut; weights and positions past a length are untouched."""
    pool_k, pool_v, weight, pos = pool_k.copy(), pool_v.copy(), weight.copy(), pos.copy()
    size = pool_k.shape[2]
    for b, n in enumerate(lens):
        if n <= budget:
            continue
        for h in range(pool_k.shape[1]):
            kept = kept_tokens(weight[b, h, :n], pos[b, h, :n], seen[b], budget, sink, recent)
            stay = set(kept)
            holes = [j for j in range(budget) if j not in stay]
            movers = [j for j in kept if j >= budget]
            for to, frm in zip(holes, movers):
                for pool in (pool_k, pool_v):
                    pool[table[b, to // size], h, to % size] = pool[table[b, frm // size], h, frm % size]
                weight[b, h, to], pos[b, h, to] = weight[b, h, frm], pos[b, h, frm]
    return pool_k, pool_v, weight, pos, [min(n, budget) for n in lens]


def token_logprobs(x, targets, top):
    """logprob, entropy, top indexes and their log probabilities, and spread = sum p |x - max|, of rows of logits."""
    logprob, entropy, index, value, spread = [], [], [], [], []
    for row, t in zip(x, targets):
        nan = np.isnan(row)
        order = np.lexsort((np.arange(len(row)), -np.where(nan, 0.0, row), nan))[:top]
        m = row.max()
        if not np.isfinite(m):   # a NaN, +inf, or nothing but -inf
            lse = h = s = np.nan
        else:
            e = np.exp(row - m)
            lse = m + np.log(e.sum())
            p, d = e / e.sum(), np.where(e > 0, row - m, 0.0)
            h, s = np.log(e.sum()) - (p * d).sum(), (p * np.abs(d)).sum()
        logprob.append(0.0 if t == -1 else row[t] - lse if 0 <= t < len(row) else np.nan)
        entropy.append(h)
        spread.append(s)
        index.append(order)
        value.append([row[i] - lse for i in order])
    return (np.array(logprob), np.array(entropy), np.array(index, dtype=np.int64).reshape(len(x), top),
            np.array(value).reshape(len(x), top), np.array(spread))
