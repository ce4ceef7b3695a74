"""A small decoder that generates tokens with the library's operators.

One block: attention over a paged key-value cache, then the sparse-MoE layer,
then logits over a small vocabulary.  Weights are seeded random numbers; the
projections are plain matrix products.  Every step, for a batch of sequences:

    kv_append       the new token's keys and values into the cache
    attend_decode   attention over it, adding up the weight each token draws
    forward_decode  the sparse-MoE layer
    token_logprobs  the next token (the likeliest), its log probability, the
                    entropy and the runners-up
    kv_evict        every `page` steps, once the cache is past its budget

Run it on a GPU with the library built:

    python examples/decode_loop.py --steps 64 --budget 32
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_quantized_sparse_gb300 import moe_w4 as mw, serving as sv, synthetic as S  # noqa: E402


class Decoder:
    """The block's weights and the cache of `seqs` sequences, at most `budget + page` tokens each."""

    def __init__(self, seqs=4, q_heads=8, kv_heads=2, head_dim=64, vocab=1000, page=8, budget=32, seed=0):
        layer, _ = S.draw_config("tiny_T4")
        self.layer = mw.DeviceLayer(layer, "cuda")
        hidden = layer.H
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            w = torch.randn(shape, device="cuda", generator=g) * shape[0] ** -0.5
            return w.to(torch.bfloat16)
        self.embed = weight(vocab, hidden) * vocab ** 0.5
        self.qkv = weight(hidden, (q_heads + 2 * kv_heads) * head_dim)
        self.proj = weight(q_heads * head_dim, hidden)
        self.unembed = weight(hidden, vocab) * 4
        self.heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.budget, self.page, self.seen = budget, page, 0
        # pages handed out once: a sequence keeps its own, eviction frees places inside them
        pages = -(-(budget + page) // page)
        table = torch.arange(seqs * pages, dtype=torch.int32, device="cuda").view(seqs, pages)
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.cache = sv.PagedKVCache.allocate(seqs * pages, page, kv_heads, head_dim, table, self.lens, track=True)
        self.positions = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.length = 0   # of every sequence: known here without asking the GPU

    @staticmethod
    def _normed(x):
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def step(self, tokens, top=3):
        """Feeds one int32 token per sequence; returns the next tokens and their TokenLogprobs."""
        if self.length == self.budget + self.page:   # room for the new token
            sv.kv_evict(self.cache, self.positions, self.budget, sink=2, recent=self.budget // 4)
            self.length = self.budget
        x = self.embed[tokens.long()]
        qkv = (self._normed(x) @ self.qkv).view(len(tokens), -1, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
        self.lens += 1
        sv.kv_append(self.cache, k, v, pos=self.positions)
        self.positions += 1
        self.length += 1
        att = sv.attend_decode(self.cache, q, max_len=self.length, weight_out=self.cache.weight)
        x = x + att.reshape(len(tokens), -1) @ self.proj
        x = x + mw.forward_decode(self.layer, self._normed(x).contiguous())
        logits = self._normed(x) @ self.unembed
        best = sv.token_logprobs(logits, top=top)
        following = best.top_index[:, 0].contiguous()
        return following, best


def generate(steps, **kw):
    """Tokens [steps][sequences], their log probabilities and entropies, and the decoder."""
    dec = Decoder(**kw)
    tokens = torch.arange(dec.lens.shape[0], dtype=torch.int32, device="cuda")
    said = []
    for _ in range(steps):
        tokens, best = dec.step(tokens)
        said.append((tokens, best.top_logprob[:, 0], best.entropy))
    return [torch.stack(x) for x in zip(*said)], dec


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--budget", type=int, default=32)
    a = ap.parse_args()
    (tokens, logprob, entropy), dec = generate(a.steps, seqs=a.seqs, budget=a.budget)
    for b in range(a.seqs):
        print("sequence %d: %s" % (b, " ".join(str(t) for t in tokens[:, b].tolist())))
        print("  mean log probability %.3f, mean entropy %.3f nats" % (logprob[:, b].mean(), entropy[:, b].mean()))
    n = int(dec.lens[0])
    held = dec.cache.pos[0, 0, :n].sort().values.tolist()
    print("tokens fed %d, held %d; positions that head 0 of sequence 0 holds: %s" % (a.steps, n, held))
    print("device status: cache %d, layer %d, log probabilities %d" % (dec.cache.status(), dec.layer.status(), sv.logprobs_status()))


if __name__ == "__main__":
    main()
