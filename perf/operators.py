"""The operators of a decode step around the sparse-MoE layer, measured case by case.

Four operators: writing new keys and values into a paged cache (append), the
attention of one new token per sequence over that cache (attend), dropping
tokens from it by accumulated attention weight (evict), and the log
probabilities of given tokens with entropy and the top alternatives (logprobs).
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    bf = dict(type="bf16")
    return [
        # one new token for each of 16 sequences of a decode batch
        dict(op="append", name="append_decode_16", seqs=16, tokens=16, start=4096, kv_heads=2, dim=256, page=16,
             layout="head", **bf),
        # the last 4096-token chunk of a 16384-token prompt
        dict(op="append", name="append_chunk_4096", seqs=1, tokens=4096, start=12288, kv_heads=2, dim=256, page=64,
             layout="slot", **bf),
        # a chat turn just begun: the latency of one short sequence
        dict(op="attend", name="attend_1x300", seqs=1, len=300, ragged=False, q_heads=16, kv_heads=2, dim=256,
             page=16, layout="head", track=False, **bf),
        # one user at a very long context
        dict(op="attend", name="attend_1x131072", seqs=1, len=131072, ragged=False, q_heads=16, kv_heads=2, dim=256,
             page=64, layout="head", track=False, **bf),
        # a serving batch of mixed lengths, one slot idle
        dict(op="attend", name="attend_16xmixed", seqs=16, len=32768, ragged=True, q_heads=32, kv_heads=8, dim=128,
             page=32, layout="slot", track=False, type="fp16"),
        # a batch whose cache is pruned: the attention also adds up each token's weight
        dict(op="attend", name="attend_8x4097_track", seqs=8, len=4097, ragged=False, q_heads=16, kv_heads=2, dim=256,
             page=16, layout="head", track=True, **bf),
        # every query head with keys of its own, short odd lengths
        dict(op="attend", name="attend_64x1000_mha", seqs=64, len=1000, ragged=True, q_heads=12, kv_heads=12, dim=64,
             page=128, layout="slot", track=False, **bf),
        # steady state: the cache is one page over its budget
        dict(op="evict", name="evict_16x4112", seqs=16, len=4112, ragged=False, budget=4096, sink=4, recent=256,
             kv_heads=2, dim=256, page=16, layout="head", **bf),
        # long prompts cut to a budget after their prefill
        dict(op="evict", name="evict_4x32768", seqs=4, len=32768, ragged=True, budget=8192, sink=4, recent=1024,
             kv_heads=8, dim=128, page=32, layout="slot", type="fp16"),
        # the sampled token of one sequence, with five alternatives
        dict(op="logprobs", name="logprobs_1x32000", rows=1, vocab=32000, top=5, type="fp32"),
        # a decode batch with the twenty alternatives that an API returns
        dict(op="logprobs", name="logprobs_16x131072", rows=16, vocab=131072, top=20, **bf),
        # scoring a 4096-token prompt chunk; rows of odd length are not aligned
        dict(op="logprobs", name="logprobs_4096x49999", rows=4096, vocab=49999, top=5, type="fp16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "evict", "logprobs"])
    if op == "logprobs":
        typ = rng.choice(["bf16", "fp16", "fp32"])
        vocab = _log(rng, 1000, 262144)
        rows = _log(rng, 1, max(1, min(4096, 400_000_000 // (vocab * (4 if typ == "fp32" else 2)))))
        return dict(op=op, rows=rows, vocab=vocab, top=rng.randint(0, 20), type=typ)
    c = dict(op=op, type=rng.choice(["bf16", "fp16"]), layout=rng.choice(["head", "slot"]),
             page=rng.choice([8, 16, 32, 64, 128]), dim=rng.choice([64, 128, 256]), kv_heads=rng.choice([1, 2, 4, 8]))
    row = c["kv_heads"] * c["dim"] * 4   # bytes of a token's keys and values
    if op == "append":
        tokens = _log(rng, 1, 16384)
        c.update(tokens=tokens, seqs=rng.randint(1, min(tokens, 64)), start=_log(rng, 1, 8192))
        return c
    if op == "attend":
        n = _log(rng, 1, 131072)
        seqs = _log(rng, 1, max(1, min(128, 500_000_000 // (n * row))))
        c.update(len=n, seqs=seqs, ragged=rng.random() < 0.6, track=rng.random() < 0.3)
        c["q_heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 5, 8, 12, 16, 24])
        return c
    n = _log(rng, 64, 32768)
    budget = max(8, min(n, int(n * rng.uniform(0.2, 1.0))))
    c.update(len=n, seqs=_log(rng, 1, max(1, min(16, 250_000_000 // (n * row)))), ragged=rng.random() < 0.6,
             budget=budget, sink=rng.randint(0, 4), recent=rng.randint(0, budget // 2))
    return c


def _lens(case):
    """The sequences' lengths: the longest first; mixed ones spread over their logarithm, from eight up one idle."""
    n, seqs = case["len"], case["seqs"]
    if not case["ragged"]:
        return [n] * seqs
    rng = random.Random("%d %d" % (n, seqs))
    lens = [n] + [_log(rng, 1, n) for _ in range(seqs - 1)]
    if seqs >= 8 and case["op"] == "attend":
        lens[seqs // 2] = 0
    return lens


def _pool(case, pages, g):
    """Keys and values of `pages` pages, as [page][head][slot][dim] views of either order in memory."""
    dt = TYPES[case["type"]]
    h, s, d = case["kv_heads"], case["page"], case["dim"]
    shape = (pages, h, s, d) if case["layout"] == "head" else (pages, s, h, d)
    kv = [torch.randn(shape, dtype=dt, device="cuda", generator=g) for _ in range(2)]
    return [t if case["layout"] == "head" else t.permute(0, 2, 1, 3) for t in kv]


def _table(lens, page, g):
    """Pages handed out in random order; entries past a sequence's end are -1."""
    need = [-(-n // page) for n in lens]
    width, total = max(1, max(need)), sum(need)
    order = torch.randperm(total + 1, device="cuda", generator=g).to(torch.int32)
    t = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = order[at:at + n]
        at += n
    return t, total + 1


def _append_split(case):
    """Tokens of each sequence in this call."""
    n, seqs = case["tokens"], case["seqs"]
    return [n // seqs + (1 if i < n % seqs else 0) for i in range(seqs)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    dt, dev = TYPES[case["type"]], "cuda"
    s = dict(case=case)
    if case["op"] == "logprobs":
        n, v = case["rows"], case["vocab"]
        x = torch.randn((n, v), dtype=torch.float32, device=dev, generator=g) * 2.5
        s["logits"] = x.to(dt)
        s["targets"] = torch.randint(0, v, (n,), device=dev, generator=g).to(torch.int32)
        del x
        # every fourth target is a token that the model finds likely, as most are when a prompt is scored
        s["targets"][::4] = s["logits"][::4].argmax(1).to(torch.int32)
    else:
        if case["op"] == "append":
            new = _append_split(case)
            lens = [case["start"] + t for t in new]
        else:
            lens = _lens(case)
        s["table"], pages = _table(lens, case["page"], g)
        s["k"], s["v"] = _pool(case, pages, g)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        h, d, seqs = case["kv_heads"], case["dim"], case["seqs"]
        width = s["table"].shape[1] * case["page"]
        if case["op"] == "append":
            s["seq"] = torch.cat([torch.full((t,), i, dtype=torch.int32) for i, t in enumerate(new)]).to(dev)
            s["slot"] = torch.cat([torch.arange(t, dtype=torch.int32) for t in new]).to(dev) + case["start"]
            # keys and values as they leave one projection: a token's keys, then its values
            kv = torch.randn((case["tokens"], 2, h, d), dtype=dt, device=dev, generator=g)
            s["k_new"], s["v_new"] = kv[:, 0], kv[:, 1]
        elif case["op"] == "attend":
            q = torch.randn((seqs, case["q_heads"], d), dtype=torch.float32, device=dev, generator=g)
            s["q"] = (q * 1.5).to(dt)
            s["scale"] = 1 / math.sqrt(d)
            if case["track"]:
                s["weight"] = torch.rand((seqs, h, width), device=dev, generator=g) * 4
                s["weight_out"] = torch.zeros_like(s["weight"])
        else:
            # weights as attention leaves them: a few large, a tail, and the newest tokens still without any
            w = torch.exp(2 * torch.randn((seqs, h, width), device=dev, generator=g))
            w[:, :, case["len"] - case["len"] // 32:case["len"]] = 0
            s["weight"] = w
            # positions after earlier evictions: half of the tokens seen are left, in no order
            seen = 2 * width
            s["pos"] = torch.rand((seqs, h, seen), device=dev, generator=g).argsort(2)[:, :, :width].to(torch.int32)
            s["seen"] = torch.full((seqs,), seen, dtype=torch.int32, device=dev)
            s["weight_out"], s["pos_out"] = torch.zeros_like(w), torch.zeros_like(s["pos"])
            s["lens_out"] = torch.zeros_like(s["lens"])
    if own:
        from bit_quantized_sparse_gb300 import serving
        s["api"] = serving
        if case["op"] != "logprobs":
            s["cache"] = serving.PagedKVCache(s["k"], s["v"], s["table"], s["lens"], weight=s.get("weight"),
                                              pos=s.get("pos"))
    return s


def run(state):
    return _CALLS[state["case"]["op"]][1 if own else 0](state)


# ---- append -----------------------------------------------------------------
def _append_plain(s):
    page = s["case"]["page"]
    seq, slot = s["seq"].long(), s["slot"].long()
    pages = s["table"][seq, slot // page].long()
    heads = torch.arange(s["case"]["kv_heads"], device="cuda")
    at = (pages[:, None], heads[None, :], (slot % page)[:, None])
    s["k"][at] = s["k_new"]
    s["v"][at] = s["v_new"]
    return dict(k=s["k"], v=s["v"])


def _append_own(s):
    s["api"].kv_append(s["cache"], s["k_new"], s["v_new"], seq=s["seq"], slot=s["slot"])
    return dict(k=s["k"], v=s["v"])


# ---- attend -----------------------------------------------------------------
def _gathered(pool, table):
    """[sequence][head][token][dim] in 32 bits, by the table; pages of entries without one are page 0."""
    x = pool[table.clamp(min=0).long()]
    b, p, h, t, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(b, h, p * t, d).float()


def _attend_plain(s):
    c = s["case"]
    b, h, group = c["seqs"], c["kv_heads"], c["q_heads"] // c["kv_heads"]
    k = _gathered(s["k"], s["table"])
    scores = torch.matmul(s["q"].float().view(b, h, group, c["dim"]), k.transpose(2, 3)) * s["scale"]
    del k
    there = torch.arange(scores.shape[3], device="cuda")[None, :] < s["lens"][:, None]
    scores = scores.masked_fill(~there[:, None, None, :], -math.inf)
    top = scores.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(3, keepdim=True)
    lse = (top + torch.log(total)).squeeze(3)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    v = _gathered(s["v"], s["table"]).masked_fill(~there[:, None, :, None], 0)
    out = torch.matmul(p, v).to(s["q"].dtype)
    got = dict(out=out.view(b, c["q_heads"], c["dim"]), lse=lse.reshape(b, c["q_heads"]))
    if c["track"]:
        more = s["weight"] + p.sum(2)
        s["weight_out"].copy_(torch.where(there[:, None, :], more, s["weight_out"]))
        got["weight"] = s["weight_out"]
    return got


def _attend_own(s):
    got = s["api"].attend_decode(s["cache"], s["q"], scale=s["scale"], return_lse=True, max_len=s["case"]["len"],
                                 weight_out=s.get("weight_out"))
    r = dict(out=got[0], lse=got[1])
    if s["case"]["track"]:
        r["weight"] = s["weight_out"]
    return r


# ---- evict ------------------------------------------------------------------
def _evict_plain(s):
    c = s["case"]
    n, budget, page, h = c["len"], c["budget"], c["page"], c["kv_heads"]
    lens = s["lens"].long()
    w, pos = s["weight"][:, :, :n], s["pos"][:, :, :n]
    slots = torch.arange(n, device="cuda")
    there = slots[None, None, :] < lens[:, None, None]
    kept_always = (pos < c["sink"]) | (pos >= s["seen"][:, None, None] - c["recent"])
    nan = torch.isnan(w)
    rank = torch.where(kept_always, 3, torch.where(nan, 1, 2)) * there
    value = torch.where(nan | kept_always, torch.zeros_like(w), w)
    order = value.sort(dim=2, descending=True, stable=True).indices
    order = order.gather(2, rank.gather(2, order).sort(dim=2, descending=True, stable=True).indices)
    keep = torch.zeros_like(there.expand_as(w))
    keep.scatter_(2, order[:, :, :budget], True)
    over = (lens > budget)[:, None, None]
    hole = ~keep[:, :, :budget] & over
    moved = keep & (slots >= budget) & over
    m = min(budget, n)
    movers = torch.where(moved, slots, n).sort(dim=2).values[:, :, :m]
    here = slots[:m].expand(c["seqs"], h, m)
    src = torch.where(hole[:, :, :m], movers.gather(2, (hole[:, :, :m].cumsum(2) - 1).clamp(min=0)), here)
    new = lens.clamp(max=budget)
    # slots past the end repeat slot 0's move, which changes nothing
    live = here < new[:, None, None]
    src, dst = torch.where(live, src, src[:, :, :1]), torch.where(live, here, here[:, :, :1])
    table = s["table"].long()
    b_at = torch.arange(c["seqs"], device="cuda")[:, None, None]
    h_at = torch.arange(h, device="cuda")[None, :, None]
    for x in (s["k"], s["v"]):
        x[table[b_at, dst // page], h_at, dst % page] = x[table[b_at, src // page], h_at, src % page]
    for x, y in ((s["weight"], s["weight_out"]), (s["pos"], s["pos_out"])):
        y[:, :, :m] = torch.where(live, x.gather(2, src), y[:, :, :m])
    s["lens_out"].copy_(new)
    return dict(k=s["k"], v=s["v"], weight=s["weight_out"], pos=s["pos_out"], lens=s["lens_out"])


def _evict_own(s):
    c = s["case"]
    s["api"].kv_evict(s["cache"], s["seen"], c["budget"], sink=c["sink"], recent=c["recent"], max_len=c["len"],
                      lens_out=s["lens_out"], weight_out=s["weight_out"], pos_out=s["pos_out"])
    return dict(k=s["k"], v=s["v"], weight=s["weight_out"], pos=s["pos_out"], lens=s["lens_out"])


# ---- logprobs ---------------------------------------------------------------
def _logprobs_plain(s):
    x, top = s["logits"].float(), s["case"]["top"]
    most = x.amax(1, keepdim=True)
    e = torch.exp(x - most)
    total = e.sum(1, keepdim=True, dtype=torch.float64)
    lse = most.double() + torch.log(total)
    got = dict(logprob=(x.gather(1, s["targets"].long()[:, None]).double() - lse).float().squeeze(1),
               entropy=(torch.log(total) - (e * (x - most)).sum(1, keepdim=True, dtype=torch.float64) / total)
               .float().squeeze(1))
    if top:
        best = x.sort(dim=1, descending=True, stable=True).indices[:, :top]
        got["top_index"] = best.to(torch.int32)
        got["top_logprob"] = (x.gather(1, best).double() - lse).float()
    return got


def _logprobs_own(s):
    r = s["api"].token_logprobs(s["logits"], s["targets"], top=s["case"]["top"])
    got = dict(logprob=r.logprob, entropy=r.entropy)
    if s["case"]["top"]:
        got["top_index"], got["top_logprob"] = r.top_index, r.top_logprob
    return got


_CALLS = dict(append=(_append_plain, _append_own), attend=(_attend_plain, _attend_own),
              evict=(_evict_plain, _evict_own), logprobs=(_logprobs_plain, _logprobs_own))


# ---- what each has to read, write and compute ---------------------------------
def work(case):
    size = 4 if case["type"] == "fp32" else 2
    if case["op"] == "logprobs":
        n, v, k = case["rows"], case["vocab"], case["top"]
        return dict(bytes=n * (v * size + 12 + 8 * k), flops=n * v * 6)
    row = case["kv_heads"] * case["dim"] * size * 2
    if case["op"] == "append":
        return dict(bytes=case["tokens"] * (2 * row + 12), flops=0)
    lens = _lens(case)
    tokens, pages = sum(lens), sum(-(-n // case["page"]) for n in lens)
    if case["op"] == "attend":
        heads = case["seqs"] * case["q_heads"]
        extra = tokens * case["kv_heads"] * 8 if case["track"] else 0
        return dict(bytes=tokens * row + 2 * heads * case["dim"] * size + heads * 4 + 4 * pages + 4 * len(lens) + extra,
                    flops=4 * tokens * case["q_heads"] * case["dim"])
    # every weight and position is read, those kept are written; the rows that move, at the share
    # that tokens kept by chance alone would have, are read and written
    kept = sum(min(n, case["budget"]) for n in lens)
    moves = sum(b * (1 - b / n) for n in lens for b in [min(n, case["budget"])])
    return dict(bytes=8 * case["kv_heads"] * (tokens + kept) + int(moves * 2 * row) + 4 * pages, flops=0)


# ---- the definitions in 64 bits -----------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return dict(append=_append_exact, attend=_attend_exact, evict=_evict_exact, logprobs=_logprobs_exact)[case["op"]](s)


def _append_exact(s):
    c = s["case"]
    k, v = s["k"].double(), s["v"].double()
    table, seq, slot = s["table"].cpu().numpy(), s["seq"].cpu().numpy(), s["slot"].cpu().numpy()
    pages = torch.from_numpy(table[seq, slot // c["page"]].astype(np.int64)).cuda()
    inside = torch.from_numpy((slot % c["page"]).astype(np.int64)).cuda()
    for h in range(c["kv_heads"]):
        k[pages, h, inside] = s["k_new"][:, h].double()
        v[pages, h, inside] = s["v_new"][:, h].double()
    return dict(k=k, v=v)


def _attend_exact(s):
    c = s["case"]
    group = c["q_heads"] // c["kv_heads"]
    out = torch.zeros((c["seqs"], c["q_heads"], c["dim"]), dtype=torch.float64, device="cuda")
    lse = torch.full((c["seqs"], c["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
    weight = s["weight_out"].double() if c["track"] else None
    for b, n in enumerate(s["lens"].tolist()):
        if not n:
            continue
        pages = s["table"][b, :-(-n // c["page"])].long()
        for h in range(c["kv_heads"]):
            k = s["k"][pages, h].reshape(-1, c["dim"])[:n].double()
            v = s["v"][pages, h].reshape(-1, c["dim"])[:n].double()
            mine = slice(h * group, (h + 1) * group)
            scores = (s["q"][b, mine].double() @ k.T) * s["scale"]
            p = torch.softmax(scores, 1)
            out[b, mine] = p @ v
            lse[b, mine] = torch.logsumexp(scores, 1)
            if c["track"]:
                weight[b, h, :n] = s["weight"][b, h, :n].double() + p.sum(0)
    got = dict(out=out, lse=lse)
    if c["track"]:
        got["weight"] = weight
    return got


def _evict_exact(s):
    c = s["case"]
    k, v = s["k"].double(), s["v"].double()
    w, pos, table = s["weight"].cpu().numpy(), s["pos"].cpu().numpy(), s["table"].cpu().numpy()
    w_out, pos_out = s["weight_out"].cpu().numpy().astype(np.float64), s["pos_out"].cpu().numpy()
    budget, page = c["budget"], c["page"]
    lens = s["lens"].tolist()
    for b, n in enumerate(lens):
        seen = int(s["seen"][b])
        for h in range(c["kv_heads"]):
            src = np.arange(min(n, budget))
            if n > budget:
                p, x = pos[b, h, :n], w[b, h, :n].astype(np.float64)
                always = (p < c["sink"]) | (p >= seen - c["recent"])
                kept = np.sort(np.lexsort((np.arange(n), -np.where(always, np.inf, x)))[:budget])
                src[np.setdiff1d(np.arange(budget), kept)] = kept[kept >= budget]
            w_out[b, h, :len(src)], pos_out[b, h, :len(src)] = w[b, h, src], pos[b, h, src]
            to = np.nonzero(src != np.arange(len(src)))[0]
            if len(to):
                a = [torch.from_numpy(i.astype(np.int64)).cuda() for i in
                     (table[b, to // page], to % page, table[b, src[to] // page], src[to] % page)]
                for x in (k, v):
                    x[a[0], h, a[1]] = x[a[2], h, a[3]].clone()
    return dict(k=k, v=v, weight=torch.from_numpy(w_out), pos=torch.from_numpy(pos_out),
                lens=torch.tensor([min(n, budget) for n in lens], dtype=torch.int32))


def _logprobs_exact(s):
    n, top = s["case"]["rows"], s["case"]["top"]
    got = dict(logprob=[], entropy=[], top_index=[], top_logprob=[])
    for at in range(0, n, 256):
        x = s["logits"][at:at + 256].double()
        logp = x - torch.logsumexp(x, 1, keepdim=True)
        got["logprob"].append(logp.gather(1, s["targets"][at:at + 256].long()[:, None]).squeeze(1))
        got["entropy"].append(-(torch.exp(logp) * logp).sum(1))
        if top:
            # the t-th best: the largest value left, the lowest index that has it
            left = x.clone()
            best = []
            for _ in range(top):
                most = left.amax(1, keepdim=True)
                best.append((left == most).to(torch.int8).argmax(1, keepdim=True))
                left.scatter_(1, best[-1], -math.inf)
            best = torch.cat(best, 1)
            got["top_index"].append(best.to(torch.int32))
            got["top_logprob"].append(logp.gather(1, best))
    return {name: torch.cat(v) for name, v in got.items() if v}
