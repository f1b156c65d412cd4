"""The decode-step operators together: prompt, single tokens and a drafted tree of a small model.

One decoder layer and a head with random int8 weights, a paged int8 cache and low-rank adapters of
several requests:

    hidden -> q8ta_quantize_per_tensor -> q8ta_linear_lora (queries, keys and values; an adapter a
    request) -> q8ta_rope_append (into the cache) -> q8ta_tree_attention -> q8ta_quantize_per_tensor
    -> q8ta_linear_dq, added to hidden -> q8ta_quantize_per_tensor -> q8ta_linear_lora (logits, no
    adapter) -> q8ta_sample

Run as ``python examples/decode_step.py`` on a machine with the GPU.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import int8_quantized_amd as q8  # noqa: E402


class Decoder:
    """Requests 0 .. batch - 1, each with its pages of the cache and its adapter (request 0: none)."""

    def __init__(self, batch=3, hidden=512, heads=8, kv_heads=2, dim=64, vocab=2000, page=16, pages=16,
                 rank=8, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        def codes(*shape):
            return normal(*shape).mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)
        self.batch, self.heads, self.kv_heads, self.dim, self.vocab, self.page = \
            batch, heads, kv_heads, dim, vocab, page
        wide = (heads + 2 * kv_heads) * dim
        self.embedding = normal(vocab, hidden)
        self.w_qkv, self.w_out, self.w_head = codes(wide, hidden), codes(hidden, heads * dim), codes(vocab, hidden)
        self.s_qkv, self.s_out, self.s_head = (torch.full((n,), s / 36.0 / math.sqrt(k), device="cuda")
                                               for n, k, s in ((wide, hidden, 1.0), (hidden, heads * dim, 1.0),
                                                               (vocab, hidden, 3.0)))
        self.lora_a = (normal(batch, rank, hidden) / math.sqrt(hidden)).bfloat16()
        self.lora_b = (normal(batch, wide, rank) / math.sqrt(rank) * 0.3).bfloat16()
        # the head has no adapter of its own: one of zeros, which no row names
        self.head_a = torch.zeros((1, 1, hidden), dtype=torch.bfloat16, device="cuda")
        self.head_b = torch.zeros((1, vocab, 1), dtype=torch.bfloat16, device="cuda")
        self.x_scale, self.o_scale = 4.0 / 127, 3.0 / 127
        self.inv_freq = 10000.0 ** (-torch.arange(0, dim, 2, device="cuda").double() / dim)
        total = batch * pages
        self.cache = torch.zeros((total, 2, kv_heads, page, dim), dtype=torch.int8, device="cuda")
        self.scales = torch.zeros((total, 2, kv_heads, page), device="cuda")
        self.table = torch.randperm(total, generator=g, device="cuda").reshape(batch, pages).int()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def step(self, tokens, depth=None, mask=None):
        """Logits [batch, T, vocab] of T new tokens a request, appended to the cache behind its
        context.  depth [batch, T]: a drafted token's place behind the context (None: a chain);
        mask [batch, T]: as for q8ta_tree_attention.  `accept` moves the context on."""
        B, T = tokens.shape
        at = torch.arange(T, device="cuda").expand(B, T)
        rows = self.lens.unsqueeze(1).long() + at                        # cache rows
        slots = self.table.gather(1, rows // self.page).long() * self.page + rows % self.page
        positions = (self.lens.unsqueeze(1) + (at if depth is None else depth)).int()
        x = self.embedding[tokens.reshape(-1).long()]
        xq = torch.empty(x.shape, dtype=torch.int8, device="cuda")
        q8.q8ta_quantize_per_tensor(x, xq, self.x_scale, 0)
        qkv = torch.empty((B * T, self.w_qkv.shape[0]), dtype=torch.bfloat16, device="cuda")
        request = torch.arange(B, dtype=torch.int32, device="cuda").repeat_interleave(T)
        q8.q8ta_linear_lora(xq, self.x_scale, 0, self.w_qkv, self.s_qkv, None, self.lora_a, self.lora_b,
                            None, None, request - (request == 0).int(), "none", qkv)
        hq, hk, d = self.heads, self.kv_heads, self.dim
        q, k, v = (part.unflatten(1, (-1, d)) for part in qkv.split([hq * d, hk * d, hk * d], 1))
        turned = torch.empty((B * T, hq, d), dtype=torch.bfloat16, device="cuda")
        q8.q8ta_rope_append(q, k, v, positions.reshape(-1).contiguous(), slots.reshape(-1).contiguous(),
                            self.inv_freq, 1.0, False, turned, self.cache, self.scales)
        out = torch.empty((B, T, hq, d), dtype=torch.bfloat16, device="cuda")
        q8.q8ta_tree_attention(turned.view(B, T, hq, d), self.cache, self.scales, self.table, self.lens,
                               None, mask, 1.0 / math.sqrt(d), out)
        oq = torch.empty((B * T, hq * d), dtype=torch.int8, device="cuda")
        q8.q8ta_quantize_per_tensor(out.float().view(B * T, hq * d), oq, self.o_scale, 0)
        y = torch.empty_like(x)
        q8.q8ta_linear_dq(oq, self.o_scale, 0, self.w_out, None, self.s_out, None, self.x_scale, 0, "none", y)
        q8.q8ta_quantize_per_tensor(x + y, xq, self.x_scale, 0)
        logits = torch.empty((B * T, self.vocab), device="cuda")
        q8.q8ta_linear_lora(xq, self.x_scale, 0, self.w_head, self.s_head, None, self.head_a, self.head_b,
                            None, None, torch.full_like(request, -1), "none", logits)
        return logits.view(B, T, self.vocab)

    def accept(self, n):
        self.lens += n

    def sample(self, logits, u, temperature=0.8, top_k=50, top_p=0.95):
        """One token a row of logits [rows, vocab], by the numbers u."""
        rows = logits.shape[0]

        def full(value, dtype=torch.float32):
            return torch.full((rows,), value, dtype=dtype, device="cuda")
        tokens = torch.empty(rows, dtype=torch.int32, device="cuda")
        q8.q8ta_sample(logits, full(temperature), full(top_k, torch.int32), full(top_p), None, u, tokens)
        return tokens


def tree_of(chain, spare):
    """Drafts of `chain` [B, n] as a tree of 2n tokens a request: the chain at the even places and a
    wrong guess `spare` beside each.  Returns tokens, depths and ancestor masks."""
    B, n = chain.shape
    tokens = torch.stack((chain, spare), 2).reshape(B, 2 * n)
    depth = torch.arange(n, device="cuda").repeat_interleave(2).expand(B, -1)
    bits = []
    for i in range(n):
        above = sum(1 << (2 * j) for j in range(i))
        bits += [above | 1 << (2 * i), above | 1 << (2 * i + 1)]
    mask = torch.tensor(bits, dtype=torch.int64, device="cuda").expand(B, -1).contiguous()
    return tokens, depth, mask


def main():
    model = Decoder()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    prompt = torch.randint(0, model.vocab, (model.batch, 21), generator=g, device="cuda")
    logits = model.step(prompt)
    model.accept(prompt.shape[1])
    new = []
    for _ in range(8):
        token = model.sample(logits[:, -1], torch.rand(model.batch, generator=g, device="cuda"))
        new.append(token)
        logits = model.step(token.unsqueeze(1))
        model.accept(1)
    for b, row in enumerate(torch.stack(new, 1).tolist()):
        print(f"request {b}: {row}")


if __name__ == "__main__":
    main()
