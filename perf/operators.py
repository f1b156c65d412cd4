"""The decode-step operators around q8ta_linear: what is timed, and their plain forms.

Four operators of a quantized language model's step, which run one after the
other: ``q8ta_linear_lora`` (the shared int8 projection with low-rank adapters
of many requests), ``q8ta_rope_append`` (rotary positions, keys and values
quantized into the paged int8 cache), ``q8ta_tree_attention`` (single tokens
or a tree of drafted tokens over that cache) and ``q8ta_sample`` (temperature,
top-k, top-p and min-p from given random numbers).

``run`` makes the package's calls where ``own`` is true, and elementary torch
operations where it is not.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"fp32": 4, "fp16": 2, "bf16": 2}
DEV = "cuda"


def listed():
    return [
        # one new token of one request, as every step of a chat does: latency
        {"name": "rope_append 1 token", "op": "rope_append", "tokens": 1, "seqs": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "rot": 128, "layout": "half", "scaling": "none", "dtype": "bf16",
         "start": 611, "page": 16},
        # the prompts of five requests, projections in fp32 as q8ta_linear_dq
        # leaves them, part of the head rotated, positions far past the trained length
        {"name": "rope_append prompts", "op": "rope_append", "tokens": 8191, "seqs": 5, "heads": 32,
         "kv_heads": 8, "dim": 128, "rot": 64, "layout": "interleaved", "scaling": "yarn",
         "dtype": "fp32", "start": 120000, "page": 64},
        # one request, one token, a short context: latency
        {"name": "attention 1 x 700", "op": "attention", "batch": 1, "tokens": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "context": 700, "page": 16, "dtype": "bf16"},
        # verification of 24 drafted tokens for 16 requests of ragged length
        {"name": "attention tree 24 x 16 x 4k", "op": "attention", "batch": 16, "tokens": 24,
         "heads": 32, "kv_heads": 8, "dim": 128, "context": 4100, "page": 32, "dtype": "fp16"},
        # a busy server's decode step: single tokens over long contexts
        {"name": "attention 32 x 24k", "op": "attention", "batch": 32, "tokens": 1, "heads": 64,
         "kv_heads": 8, "dim": 128, "context": 24001, "page": 64, "dtype": "bf16"},
        # wide trees with narrow heads over long contexts: the arithmetic counts
        {"name": "attention tree 64 x 4 x 16k", "op": "attention", "batch": 4, "tokens": 64,
         "heads": 32, "kv_heads": 4, "dim": 64, "context": 16385, "page": 128, "dtype": "bf16"},
        # one token of one request with its own adapter: the weight stream
        {"name": "lora 1 row", "op": "lora", "rows": 1, "k": 4096, "n": 4096, "rank": 16,
         "adapters": 4, "runs": 1, "adapter_dtype": "bf16", "dtype": "fp32"},
        # single tokens of 50 requests over 24 adapters, in the order they came
        {"name": "lora 50 rows of 24 adapters", "op": "lora", "rows": 50, "k": 4096, "n": 11008,
         "rank": 32, "adapters": 24, "runs": 50, "adapter_dtype": "fp16", "dtype": "bf16"},
        # prompts of eight requests, each a run of rows with one adapter
        {"name": "lora 2048 rows", "op": "lora", "rows": 2048, "k": 4096, "n": 11008, "rank": 64,
         "adapters": 6, "runs": 8, "adapter_dtype": "bf16", "dtype": "bf16"},
        # one request's next token from a small vocabulary: latency
        {"name": "sample 1 x 32000", "op": "sample", "rows": 1, "vocab": 32000, "dtype": "fp32",
         "temperature": 0.7, "top_k": 50, "top_p": 0.9, "min_p": 0.0, "mixed": False},
        # a small batch, 16-bit logits with their many ties, nucleus only
        {"name": "sample 24 x 100003", "op": "sample", "rows": 24, "vocab": 100003, "dtype": "bf16",
         "temperature": 1.0, "top_k": 0, "top_p": 0.95, "min_p": 0.0, "mixed": False},
        # a full batch whose requests each have their own settings (greedy and unfiltered among them)
        {"name": "sample 256 x 131072", "op": "sample", "rows": 256, "vocab": 131072,
         "dtype": "fp32", "temperature": 0.8, "top_k": 100, "top_p": 0.9, "min_p": 0.02,
         "mixed": True},
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope_append", "attention", "lora", "sample"])
    if op == "rope_append":
        dim = rng.choice([64, 80, 96, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 4, 7, 8])
        tokens = _between(rng, 1, min(16384, 8191 * 48 * 128 // ((heads + 2 * kv_heads) * dim)))
        return {"op": op, "tokens": tokens, "seqs": rng.randint(1, min(tokens, 64)), "heads": heads,
                "kv_heads": kv_heads, "dim": dim, "rot": rng.choice([dim, dim // 2]),
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "ntk", "yarn"]),
                "dtype": rng.choice(["fp32", "fp16", "bf16"]), "start": _between(rng, 1, 1000000),
                "page": rng.choice([16, 32, 64, 128, 256])}
    if op == "attention":
        batch = _between(rng, 1, 64)
        tokens = rng.choice([1, _between(rng, 1, 64)])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 4, 7, 8])
        dim = rng.choice([64, 80, 128, 256])
        # no more cache than the busy server's case, no more arithmetic than the wide trees'
        most = min(32768, 32 * 16000 * 8 * 128 // (batch * kv_heads * dim),
                   4 * 64 * 32 * 64 * 12000 // (batch * tokens * heads * dim))
        return {"op": op, "batch": batch, "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
                "dim": dim, "context": _between(rng, 1, max(1, most)),
                "page": rng.choice([16, 32, 64, 128, 256]), "dtype": rng.choice(["fp16", "bf16"])}
    if op == "lora":
        rows = _between(rng, 1, 2048)
        k = 16 * _between(rng, 16, 688) - (rng.randint(1, 15) if rng.random() < 0.1 else 0)
        n = _between(rng, 256, 11008)
        most = 2048 * 4096 * 11008 // (k * n)
        rows = min(rows, max(1, most))
        return {"op": op, "rows": rows, "k": k, "n": n, "rank": rng.choice([4, 8, 16, 32, 64]),
                "adapters": _between(rng, 1, 32), "runs": _between(rng, 1, rows),
                "adapter_dtype": rng.choice(["fp16", "bf16"]),
                "dtype": rng.choice(["fp32", "fp16", "bf16"])}
    vocab = _between(rng, 1000, 262144)
    return {"op": op, "rows": _between(rng, 1, max(1, min(256, 256 * 131072 // vocab))),
            "vocab": vocab, "dtype": rng.choice(["fp32", "fp16", "bf16"]),
            "temperature": round(rng.uniform(0.3, 1.5), 2), "top_k": rng.choice([0, 1, 20, 50, 1000]),
            "top_p": rng.choice([1.0, 0.95, 0.9, 0.5]), "min_p": rng.choice([0.0, 0.02, 0.1]),
            "mixed": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# Sizes that follow from a case alone

def _lengths(case):
    """Ragged context lengths of the attention's requests; the first is the longest."""
    c = case["context"]
    return [max(1, c - (b * 7919) % (c // 2 + 1)) for b in range(case["batch"])]


def _pages(case):
    """Pages of each request's block table."""
    return -(-(case["context"] + case["tokens"]) // case["page"])


def _append_pages(case):
    """Token counts of the appended requests and the pages that hold them."""
    t, n = case["tokens"], case["seqs"]
    counts = [t // n + (1 if i < t % n else 0) for i in range(n)]
    return counts, sum(-(-c // case["page"]) for c in counts)


def _adapter_rows(case):
    """Adapter of each row: `runs` runs of rows; one run in nine has no adapter."""
    m, runs, n = case["rows"], min(case["runs"], case["rows"]), case["adapters"]
    run = np.arange(m) * runs // m
    return np.where((run % 9 == 8), -1, (run * 5 + 1) % n)


def _settings(case):
    """Per-row sampling settings: [temperature, top_k, top_p, min_p] columns."""
    b = case["rows"]
    t, k = np.full(b, case["temperature"]), np.full(b, case["top_k"])
    p, mp = np.full(b, case["top_p"]), np.full(b, case["min_p"])
    if case["mixed"]:
        r = np.arange(b) % 8
        t[r == 1] = 0.0                       # greedy
        k[(r == 2) | (r == 4)] = 0
        p[(r == 2) | (r == 3)] = 1.0
        mp[(r == 2) | (r == 5) | (r == 6)] = 0.0   # rows 2: unfiltered
        t[r == 6] = 1.0
    return t.astype(np.float32), k.astype(np.int32), p.astype(np.float32), mp.astype(np.float32)


def work(case):
    """Bytes and operations that one pass cannot do without."""
    op = case["op"]
    if op == "rope_append":
        t, d, hq, hk = case["tokens"], case["dim"], case["heads"], case["kv_heads"]
        es, slots = SIZES[case["dtype"]], _append_pages(case)[1] * case["page"]
        return {"bytes": t * (2 * hq + 2 * hk) * d * es + t * 2 * hk * (d + 4) + t * 12
                + slots * 2 * hk * (d * 5 + 4),
                "flops": 3 * t * (hq + hk) * case["rot"] + 4 * t * hk * d + slots * 2 * hk * d}
    if op == "attention":
        d, hq, hk, t = case["dim"], case["heads"], case["kv_heads"], case["tokens"]
        keys = sum(_lengths(case)) + case["batch"] * t
        return {"bytes": keys * hk * 2 * (d + 4)
                + case["batch"] * t * hq * (2 * d * SIZES[case["dtype"]] + 4),
                "flops": 4 * keys * t * hq * d}
    if op == "lora":
        m, k, n, r = case["rows"], case["k"], case["n"], case["rank"]
        rows = _adapter_rows(case)
        used = len(set(rows[rows >= 0].tolist()))
        return {"bytes": m * k + n * k + 8 * n + used * r * (k + n) * 2 + m * n * SIZES[case["dtype"]],
                "flops": 2 * m * n * k + 2 * int((rows >= 0).sum()) * r * (k + n)}
    return {"bytes": case["rows"] * (case["vocab"] * SIZES[case["dtype"]] + 28),
            "flops": case["rows"] * case["vocab"] * 4}


# ---------------------------------------------------------------------------
# Inputs

def _frequencies(case):
    """Angle per position of each rotated pair (float64) and the factor on cos and sin."""
    rot, theta, length = case["rot"], 10000.0, 4096
    i = np.arange(rot // 2, dtype=np.float64)
    f = theta ** (-2.0 * i / rot)
    s = 8.0
    if case["scaling"] == "linear":
        return f / s, 1.0
    if case["scaling"] == "ntk":
        return (theta * s ** (rot / max(rot - 2.0, 1.0))) ** (-2.0 * i / rot), 1.0
    if case["scaling"] == "yarn":
        def pair(turns):   # the pair that makes `turns` turns over the trained length
            return rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f / s * ramp + f * (1.0 - ramp), 0.1 * math.log(s) + 1.0
    return f, 1.0


def _tree(rng, batch, tokens):
    """Ancestor masks (bit j: token j is the token itself or an ancestor) and depths of random trees."""
    mask, depth = np.zeros((batch, tokens), np.uint64), np.zeros((batch, tokens), np.int64)
    mask[:, 0] = 1
    for t in range(1, tokens):
        parent = rng.integers(max(0, t - 4), t, batch)
        mask[:, t] = mask[np.arange(batch), parent] | (np.uint64(1) << np.uint64(t))
        depth[:, t] = depth[np.arange(batch), parent] + 1
    return mask.view(np.int64), depth


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def codes(*shape):
        out = torch.empty(shape, dtype=torch.int8, device=DEV)
        flat, step = out.view(-1), 1 << 28
        for at in range(0, flat.numel(), step):
            part = flat[at:at + step]
            part.copy_(normal(part.numel()).mul_(36.0).round_().clamp_(-127, 127))
        return out

    s = {"case": dict(case)}
    if case["op"] == "rope_append":
        t, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        dt = DTYPES[case["dtype"]]
        counts, pages = _append_pages(case)
        qkv = normal(t, (hq + 2 * hk) * d).to(dt)     # one fused projection's rows
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["v"] = qkv[:, (hq + hk) * d:].unflatten(1, (hk, d))
        order, slots, positions, at = rng.permutation(pages), [], [], 0
        for i, n in enumerate(counts):
            j, need = np.arange(n), -(-n // case["page"])
            slots.append(order[at + j // case["page"]] * case["page"] + j % case["page"])
            positions.append(case["start"] + 13 * i + j)
            at += need
        s["slots"] = dev(np.concatenate(slots).astype(np.int64))
        s["positions"] = dev(np.concatenate(positions).astype(np.int32))
        f, s["factor"] = _frequencies(case)
        s["inv_freq"] = dev(f)
        s["q_out"] = torch.empty((t, hq, d), dtype=dt, device=DEV)
        s["cache"] = torch.zeros((pages, 2, hk, case["page"], d), dtype=torch.int8, device=DEV)
        s["scales"] = torch.zeros((pages, 2, hk, case["page"]), dtype=torch.float32, device=DEV)
    elif case["op"] == "attention":
        b, t, hq, hk, d = (case[n] for n in ("batch", "tokens", "heads", "kv_heads", "dim"))
        pages, dt = _pages(case), DTYPES[case["dtype"]]
        s["q"] = normal(b, t, hq, d).mul_(1.5).to(dt)
        s["cache"] = codes(b * pages, 2, hk, case["page"], d)
        s["scales"] = normal(b * pages, 2, hk, case["page"]).mul_(0.3).exp_().mul_(0.03)
        s["table"] = dev(rng.permutation(b * pages).reshape(b, pages).astype(np.int32))
        s["lens"] = dev(np.array(_lengths(case), np.int32))
        s["mask"] = dev(_tree(rng, b, t)[0])
        s["softmax_scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.empty((b, t, hq, d), dtype=dt, device=DEV)
        s["lse"] = torch.empty((b, t, hq), dtype=torch.float32, device=DEV)
    elif case["op"] == "lora":
        m, k, n, r, na = (case[c] for c in ("rows", "k", "n", "rank", "adapters"))
        ad = DTYPES[case["adapter_dtype"]]
        s["x"], s["w"] = codes(m, k), codes(n, k)
        s["x_scale"], s["x_zp"] = 0.021, int(rng.integers(-20, 21))
        s["w_scales"] = normal(n).mul_(0.2).exp_().mul_(0.0009)
        s["bias"] = normal(n).mul_(0.1)
        s["a"] = normal(na, r, k).mul_(1.0 / math.sqrt(k)).to(ad)
        s["b"] = normal(na, n, r).mul_(1.0 / math.sqrt(r)).to(ad)
        s["ad_scales"] = dev(rng.uniform(0.5, 2.0, na).astype(np.float32))
        s["ids"] = dev(_adapter_rows(case).astype(np.int32))
        s["out"] = torch.empty((m, n), dtype=DTYPES[case["dtype"]], device=DEV)
    else:
        b, v = case["rows"], case["vocab"]
        # a bulk of unlikely tokens and some tens of likely ones a row
        x = normal(b, v).mul_(2.0)
        x += (torch.rand((b, v), generator=g, device=DEV) < 40.0 / v) * normal(b, v).mul_(3.0).add_(8.0)
        s["logits"] = x.to(DTYPES[case["dtype"]])
        for name, a in zip(("temperature", "top_k", "top_p", "min_p"), _settings(case)):
            s[name] = dev(a)
        s["u"] = torch.rand(b, generator=g, device=DEV)
        s["tokens"] = torch.empty(b, dtype=torch.int32, device=DEV)
        s["logprobs"] = torch.empty(b, dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# One pass

def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _own_rope_append(s):
    import int8_quantized_amd as q8
    q8.q8ta_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"],
                        s["factor"], s["case"]["layout"] == "interleaved", s["q_out"], s["cache"],
                        s["scales"])
    return {"q": s["q_out"], "values": s["cache"] * s["scales"].unsqueeze(-1)}


def _own_attention(s):
    import int8_quantized_amd as q8
    q8.q8ta_tree_attention(s["q"], s["cache"], s["scales"], s["table"], s["lens"], None, s["mask"],
                           s["softmax_scale"], s["out"], s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_lora(s):
    import int8_quantized_amd as q8
    return q8.q8ta_linear_lora(s["x"], s["x_scale"], s["x_zp"], s["w"], s["w_scales"], s["bias"],
                               s["a"], s["b"], s["ad_scales"], None, s["ids"], "none", s["out"])


def _own_sample(s):
    import int8_quantized_amd as q8
    q8.q8ta_sample(s["logits"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"],
                   s["tokens"], s["logprobs"])
    return {"tokens": s["tokens"], "logprobs": s["logprobs"]}


def _rotate(x, cos, sin, rot, layout):
    """Pairs of the first `rot` elements turned by their angles, in float64."""
    x = x.double()
    h = rot // 2
    if layout == "half":
        a, b = x[..., :h], x[..., h:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _quantize(x):
    """Codes and scales of the rows of x (float64, as ties are frequent and have to stay ties): amax / 127 a row."""
    top = x.abs().amax(-1, keepdim=True)
    code = (x * 127.0 / torch.where(top > 0, top, 1.0)).round().to(torch.int8)
    return code, (top / 127.0).float().squeeze(-1)


def _plain_rope_append(s):
    c = s["case"]
    angle = s["positions"].double().unsqueeze(1) * s["inv_freq"]
    cos = (angle.cos() * s["factor"]).unsqueeze(1)
    sin = (angle.sin() * s["factor"]).unsqueeze(1)
    q = _rotate(s["q"], cos, sin, c["rot"], c["layout"]).float().to(s["q"].dtype)
    kc, ks = _quantize(_rotate(s["k"], cos, sin, c["rot"], c["layout"]))
    vc, vs = _quantize(s["v"].double())
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    s["cache"][page, 0, :, at] = kc
    s["cache"][page, 1, :, at] = vc
    s["scales"][page, 0, :, at] = ks
    s["scales"][page, 1, :, at] = vs
    return {"q": q, "values": s["cache"] * s["scales"].unsqueeze(-1)}


def _plain_attention(s):
    c = s["case"]
    b, t, hq, hk, d = (c[n] for n in ("batch", "tokens", "heads", "kv_heads", "dim"))
    table = s["table"].long()
    kv = s["cache"][table].float() * s["scales"][table].unsqueeze(-1)   # [b, pages, 2, hk, page, d]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, b, hk, -1, d)
    q = s["q"].float().reshape(b, t, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d)
    scores = torch.matmul(q, kv[0].transpose(-1, -2)).mul_(s["softmax_scale"])
    at = torch.arange(kv.shape[3], device=q.device) - s["lens"].long().unsqueeze(1)   # [b, keys]
    bit = (s["mask"].unsqueeze(2) >> at.clamp(0, 63).unsqueeze(1)) & 1               # [b, t, keys]
    seen = (at < 0).unsqueeze(1) | ((at < t).unsqueeze(1) & (bit == 1))
    seen = seen.unsqueeze(2).expand(b, t, hq // hk, -1).reshape(b, 1, t * (hq // hk), -1)
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = (scores - torch.where(top > -math.inf, top, 0.0)).exp()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, kv[1]) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, top + total.log(), -math.inf)

    def back(x):
        return x.reshape(b, hk, t, hq // hk, -1).permute(0, 2, 1, 3, 4).reshape(b, t, hq, -1)
    return {"out": back(out).to(s["q"].dtype), "lse": back(lse).squeeze(-1)}


def _plain_lora(s):
    c = s["case"]
    x = (s["x"].float() - s["x_zp"]) * s["x_scale"]
    y = torch.matmul(x, s["w"].float().t()) * s["w_scales"] + s["bias"]
    na, r, k = s["a"].shape
    t = torch.matmul(x, s["a"].float().reshape(na * r, k).t()).reshape(-1, na, r)
    on = s["ids"].unsqueeze(1) == torch.arange(na, device=x.device)
    t = (t * (on * s["ad_scales"]).unsqueeze(2)).reshape(-1, na * r)
    y += torch.matmul(t, s["b"].float().permute(0, 2, 1).reshape(na * r, -1))
    return y.to(DTYPES[c["dtype"]])


def _plain_sample(s):
    x = s["logits"].double()
    values, order = torch.sort(x, dim=-1, descending=True, stable=True)
    t = s["temperature"].double().unsqueeze(1)
    greedy = t == 0
    z = (values - values[:, :1]) / torch.where(greedy, 1.0, t)
    rank = torch.arange(x.shape[1], device=x.device)
    k = s["top_k"].unsqueeze(1)
    keep = (rank < k) | (k <= 0)
    w = torch.where(keep, z.exp(), 0.0)
    before = w.cumsum(-1) - w
    keep &= before < s["top_p"].double().unsqueeze(1) * w.sum(-1, keepdim=True)
    keep &= w >= s["min_p"].double().unsqueeze(1)
    keep = torch.where(greedy, False, keep) | (rank == 0)
    w = torch.zeros_like(x).scatter_(1, order, torch.where(keep, w, 0.0))   # the vocabulary's order
    below = w.cumsum(-1)
    total = below[:, -1:]
    token = (below <= s["u"].double().unsqueeze(1) * total).sum(-1, keepdim=True)
    token = token.clamp(max=x.shape[1] - 1)
    return {"tokens": token.squeeze(1).int(),
            "logprobs": (w.gather(1, token) / total).log().squeeze(1).float()}


_OWN = {"rope_append": _own_rope_append, "attention": _own_attention, "lora": _own_lora,
        "sample": _own_sample}
_PLAIN = {"rope_append": _plain_rope_append, "attention": _plain_attention, "lora": _plain_lora,
          "sample": _plain_sample}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, written apart from the plain forms

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope_append": _exact_rope_append, "attention": _exact_attention, "lora": _exact_lora,
            "sample": _exact_sample}[case["op"]](case, s)


def _exact_rope_append(case, s):
    h, rot = case["rot"] // 2, case["rot"]
    # a pair is a complex number, its turn a product with factor * e^(i angle)
    angle = s["positions"].cpu().numpy().astype(np.float64)[:, None] * s["inv_freq"].cpu().numpy()
    turn = torch.from_numpy(s["factor"] * np.exp(1j * angle)).to(DEV)[:, None, :]

    def rows(x):
        y = x.double().clone()
        first = slice(0, h) if case["layout"] == "half" else slice(0, rot, 2)
        second = slice(h, rot) if case["layout"] == "half" else slice(1, rot, 2)
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def stored(x):
        top = x.abs().max(-1, keepdim=True).values
        return torch.where(top > 0, torch.round(x * 127 / top) * top / 127, 0.0)

    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    flat = torch.zeros((s["cache"].shape[0] * page, 2, hk, d), dtype=torch.float64, device=DEV)
    flat[s["slots"], 0] = stored(rows(s["k"]))
    flat[s["slots"], 1] = stored(s["v"].double())
    return {"q": rows(s["q"]), "values": flat.reshape(-1, page, 2, hk, d).permute(0, 2, 3, 1, 4)}


def _exact_attention(case, s):
    b, t, hq, hk, d = (case[n] for n in ("batch", "tokens", "heads", "kv_heads", "dim"))
    out = torch.zeros((b, t, hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((b, t, hq), -math.inf, dtype=torch.float64, device=DEV)
    for i, n in enumerate(_lengths(case)):
        pages = s["table"][i].long()
        part = s["cache"][pages].double() * s["scales"][pages].double()[..., None]
        bits = s["mask"][i]
        draft = ((bits[:, None] >> torch.arange(t, device=DEV)) & 1).bool()
        seen = torch.cat((torch.ones((t, n), dtype=torch.bool, device=DEV), draft), 1)
        for h in range(hk):
            k, v = (part[:, j, h].reshape(-1, d)[:n + t] for j in (0, 1))
            heads = slice(h * (hq // hk), (h + 1) * (hq // hk))
            z = torch.tensordot(s["q"][i, :, heads].double(), k, dims=([2], [1])) * s["softmax_scale"]
            z = torch.where(seen[:, None], z, -math.inf)
            lse[i, :, heads] = torch.logsumexp(z, -1)
            share = torch.exp(z - lse[i, :, heads].nan_to_num(neginf=0.0)[..., None])
            out[i, :, heads] = torch.tensordot(share, v, dims=([2], [0]))
    return {"out": out, "lse": lse}


def _exact_lora(case, s):
    x = (s["x"].double() - s["x_zp"]) * s["x_scale"]
    y = x @ s["w"].double().t() * s["w_scales"].double() + s["bias"].double()
    ids = _adapter_rows(case)
    for a in sorted(set(ids[ids >= 0].tolist())):
        rows = torch.from_numpy(np.nonzero(ids == a)[0]).to(DEV)
        low = x[rows] @ s["a"][a].double().t()
        y[rows] += s["ad_scales"][a].double() * (low @ s["b"][a].double().t())
    return y


def _exact_sample(case, s):
    x = s["logits"].double().cpu().numpy()
    u = s["u"].double().cpu().numpy()
    tokens, logprobs = [], []
    for row, t, k, p, mp, ui in zip(x, *(a.astype(np.float64) for a in _settings(case)), u):
        if t == 0:
            tokens.append(int(row.argmax()))
            logprobs.append(0.0)
            continue
        order = np.argsort(-row, kind="stable")[:int(k) if k > 0 else len(row)]
        w = np.exp((row[order] - row[order[0]]) / t)
        # the shortest prefix that reaches p of the mass, and of it what min-p leaves
        n = 1 + int(np.count_nonzero(np.cumsum(w)[:-1] < p * w.sum()))
        n = max(1, min(n, int(np.count_nonzero(w >= mp))))
        kept = np.sort(order[:n])
        w = np.exp((row[kept] - row[order[0]]) / t)
        at = min(int(np.searchsorted(np.cumsum(w), ui * w.sum(), side="right")), n - 1)
        tokens.append(int(kept[at]))
        logprobs.append(math.log(w[at] / w.sum()))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32),
            "logprobs": torch.tensor(logprobs, dtype=torch.float64)}
