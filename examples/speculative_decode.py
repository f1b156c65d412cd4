"""Drafted tokens from end to end: a small model with one int8 scale per token, a drafter's guesses as a tree or
as drawn chains, their verification, and a cache whose pages are taken, forked and freed on the device.

One decoder layer and a head with random int8 weights:

    hidden -> q8ta_norm_quantize -> q8ta_linear_per_token (queries, keys and values) -> q8ta_rope_append (into
    the cache) -> q8ta_tree_attention -> q8ta_quantize_per_token -> q8ta_linear_per_token -> q8ta_norm_quantize
    (added to hidden, scaled by a gate) -> q8ta_gated_linear -> q8ta_quantize_per_token -> q8ta_linear_per_token
    -> q8ta_norm_quantize -> q8ta_linear_per_token (logits)

and around it, a step of every request:

    q8ta_pages_take (room for the drafts) -> the model over the drafts -> q8ta_verify_drafts ->
    q8ta_cache_compact (the kept tokens' rows) -> q8ta_pages_release (the pages of the others)

Run as ``python examples/speculative_decode.py`` on a machine with the GPU.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import int8_quantized_amd as q8  # noqa: E402

EPS = 1e-6


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


class Model:
    """Up to `requests` requests; the drafter is a table of what tends to follow each token, which the logits
    hold too."""

    def __init__(self, requests=4, hidden=256, heads=8, kv_heads=2, dim=32, ffn=688, vocab=400, page=16, pages=64,
                 table_pages=12, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        def weight(n, k, std=1.0):
            codes = normal(n, k).mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)
            return codes, torch.full((n,), std / 36.0 / math.sqrt(k), device="cuda")
        self.heads, self.kv_heads, self.dim, self.vocab, self.page = heads, kv_heads, dim, vocab, page
        self.embedding = normal(vocab, hidden).bfloat16()
        self.qkv, self.out = weight((heads + 2 * kv_heads) * dim, hidden), weight(hidden, heads * dim)
        self.gate, self.up, self.down = weight(ffn, hidden), weight(ffn, hidden), weight(hidden, ffn)
        self.head = weight(vocab, hidden)
        self.norms = [normal(hidden).mul_(0.1).add_(1.0) for _ in range(3)]
        self.gain = torch.full((1, hidden), 0.5, dtype=torch.bfloat16, device="cuda")   # of what a block adds
        self.follow = normal(vocab, vocab).mul_(2.0)
        self.inv_freq = 10000.0 ** (-torch.arange(0, dim, 2, device="cuda").double() / dim)
        self.cache = torch.zeros((pages, 2, kv_heads, page, dim), dtype=torch.int8, device="cuda")
        self.scales = torch.zeros((pages, 2, kv_heads, page), device="cuda")
        self.table, self.lens, self.refs = ints(requests, table_pages).fill_(-1), ints(requests), ints(pages)

    def linear(self, codes, scales, weight, dtype=torch.bfloat16):
        out = torch.empty((codes.shape[0], weight[0].shape[0]), dtype=dtype, device="cuda")
        return q8.q8ta_linear_per_token(codes, scales, weight[0], weight[1], None, "none", out)

    def codes(self, x):
        codes, scales = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(x.shape[0], device="cuda")
        q8.q8ta_quantize_per_token(x, codes, scales)
        return codes, scales

    def norm(self, x, residual, weight):
        """The sum of the block's output and the residual, and the codes of its norm."""
        total, codes = torch.empty_like(x), torch.empty(x.shape, dtype=torch.int8, device="cuda")
        scales = torch.empty(x.shape[0], device="cuda")
        q8.q8ta_norm_quantize(x, residual, None, None if residual is None else self.gain, 1.0, weight, EPS, total, codes,
                              scales)
        return total, codes, scales

    def take(self, more):
        """Pages for `more` rows behind each request's own."""
        granted = ints(self.lens.numel())
        q8.q8ta_pages_take(self.table, self.lens, self.page, more, self.refs, granted)
        return granted

    def forward(self, rows, tokens, mask=None):
        """Logits [len(rows), T, vocab] of T new tokens of the requests `rows`, appended behind their rows; mask as for
        q8ta_tree_attention (None: a chain).  The requests' pages have to be there."""
        B, T = tokens.shape
        table, lens = self.table[rows].contiguous(), self.lens[rows].contiguous()
        at = torch.arange(T, device="cuda")
        place = lens.long().unsqueeze(1) + at
        slots = table.gather(1, place // self.page).long() * self.page + place % self.page
        # a token's depth: its ancestors
        depth = at.expand(B, T) if mask is None else ((mask.unsqueeze(2) >> at) & 1).sum(2) - 1
        positions = (lens.unsqueeze(1) + depth).int()
        x = self.embedding[tokens.reshape(-1).long()]
        x, codes, scales = self.norm(x, None, self.norms[0])
        hq, hk, d = self.heads, self.kv_heads, self.dim
        q, k, v = (p.unflatten(1, (-1, d)) for p in self.linear(codes, scales, self.qkv).split([hq * d, hk * d, hk * d], 1))
        turned, seen = (torch.empty((B * T, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q8.q8ta_rope_append(q, k, v, positions.reshape(-1).contiguous(), slots.reshape(-1).contiguous(), self.inv_freq, 1.0,
                            False, turned, self.cache, self.scales)
        q8.q8ta_tree_attention(turned.view(B, T, hq, d), self.cache, self.scales, table, lens, None, mask,
                               1.0 / math.sqrt(d), seen.view(B, T, hq, d))
        y = self.linear(*self.codes(seen.view(B * T, hq * d)), self.out)
        x, codes, scales = self.norm(y, x, self.norms[1])
        mid = torch.empty((B * T, self.gate[0].shape[0]), dtype=torch.bfloat16, device="cuda")
        q8.q8ta_gated_linear(codes, scales, self.gate[0], self.gate[1], None, self.up[0], self.up[1], None, "silu", mid)
        y = self.linear(*self.codes(mid), self.down)
        x, codes, scales = self.norm(y, x, self.norms[2])
        logits = self.linear(codes, scales, self.head, torch.float32).view(B, T, self.vocab)
        return logits + self.follow[tokens.long()]

    def prompt(self, rows, tokens):
        """Appends prompts [len(rows), T] but their last tokens, which the first step takes up.  Returns those."""
        more = ints(self.lens.numel())
        more[rows] = tokens.shape[1] - 1
        self.take(more)
        self.forward(rows, tokens[:, :-1])
        self.lens[rows] += tokens.shape[1] - 1
        return tokens[:, -1]

    def step(self, rows, known, u, temperature=1.0, drawn=True, depth=3):
        """One step of the requests `rows`, whose last known tokens are `known`: drafts, the model over them, and
        what it keeps.  u [len(rows), tokens]: random numbers, as q8ta_verify_drafts takes them (and one more for each
        drawn draft).  Returns the new tokens [len(rows), depth + 1] and how many they are."""
        B = len(rows)
        heat = torch.full((B,), temperature, device="cuda")
        if drawn:       # a chain, each token drawn by its last
            T, mask, ids = depth + 1, None, [known.int()]
            draft = torch.empty((B, depth, self.vocab), device="cuda")
            for i in range(depth):
                draft[:, i] = self.follow[ids[-1].long()]
                ids.append(q8.q8ta_sample(draft[:, i], heat, None, None, None, u[:, T + i].contiguous(), ints(B)))
            ids = torch.stack(ids, 1)
        else:           # a tree: the two that most often follow, and the two after each
            T, draft = 7, None
            first = self.follow[known.long()].topk(2, -1).indices
            second = self.follow[first].topk(2, -1).indices.view(B, 4)
            ids = torch.cat((known.unsqueeze(1), first, second), 1).int()
            mask = torch.tensor([1, 3, 5, 11, 19, 37, 69], device="cuda").expand(B, -1).contiguous()
        more = ints(self.lens.numel())
        more[rows] = T
        self.take(more)
        logits = self.forward(rows, ids, mask)
        path, accepted, following = ints(B, T), ints(B), ints(B)
        q8.q8ta_verify_drafts(logits, draft, ids.contiguous(), None, mask, heat, None, u[:, :T].contiguous(), path, accepted,
                              following)
        q8.q8ta_cache_compact(self.cache, self.scales, self.table[rows].contiguous(), self.lens[rows].contiguous(), path,
                              accepted)
        self.lens[rows] += accepted
        q8.q8ta_pages_release(self.table, self.lens, self.page, rows.int(), self.lens[rows].contiguous(), self.refs)
        # the kept drafts, then the token after them
        at = torch.arange(depth + 1 if drawn else 3, device="cuda")
        kept = ids.gather(1, path[:, 1:1 + at.numel()].long().clamp(min=0))
        kept = torch.cat((kept, kept[:, -1:]), 1)[:, :at.numel()]
        return torch.where(at == (accepted - 1).unsqueeze(1), following.unsqueeze(1), kept), accepted

    def fork(self, src, dst):
        """Requests dst become copies of requests src (int32)."""
        out = [ints(src.numel()) for _ in range(4)]
        q8.q8ta_pages_fork(self.table, self.lens, self.page, src, dst, self.refs, *out)
        q8.q8ta_pages_copy(self.cache, self.scales, *out[1:])
        return out[0]

    def free(self, rows):
        q8.q8ta_pages_release(self.table, self.lens, self.page, rows, None, self.refs)


def generate(model, rows, known, steps, g, **kw):
    """Tokens of each request, step by step."""
    said = [[] for _ in rows]
    for _ in range(steps):
        new, count = model.step(rows, known, torch.rand((len(rows), 16), generator=g, device="cuda"), **kw)
        known = new.gather(1, (count - 1).long().unsqueeze(1)).squeeze(1)
        for text, row, n in zip(said, new.tolist(), count.tolist()):
            text += row[:n]
    return said


def main():
    model = Model()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rows = torch.arange(2, device="cuda")
    known = model.prompt(rows, torch.randint(0, model.vocab, (2, 21), generator=g, device="cuda"))
    # two samples of each prompt
    model.fork(rows.int(), (rows + 2).int())
    rows, known = torch.arange(4, device="cuda"), known.repeat(2)
    for kind, kw in (("drawn chains", dict(drawn=True)), ("trees, greedy", dict(drawn=False, temperature=0.0))):
        said = generate(model, rows, known, 4, g, **kw)
        for r, text in enumerate(said):
            print(f"{kind}, request {r}: {text}")
        known = torch.tensor([text[-1] for text in said], device="cuda")
    model.free(rows.int())
    print("pages in use:", int((model.refs > 0).sum()))


if __name__ == "__main__":
    main()
