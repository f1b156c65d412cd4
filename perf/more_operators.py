"""A decoder block with one scale per token, and what follows a step with drafted tokens: what is
timed, and the plain forms.

``q8ta_norm_quantize`` (norms before and after a block with its gate and residual, and the codes that
the next projection takes), ``q8ta_linear_per_token`` and ``q8ta_gated_linear`` (the int8 projections
with scales per token and channel), ``q8ta_verify_drafts`` (drafted tokens against the target's
probabilities), and the pages of the int8 cache: ``q8ta_pages_release`` / ``_fork`` / ``_take`` with
``q8ta_pages_copy``, and ``q8ta_cache_compact``.

``run`` makes the package's calls where ``own`` is true, and elementary torch operations where it is
not.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"fp32": 4, "fp16": 2, "bf16": 2}
DEV = "cuda"
EPS = 1e-6


def listed():
    return [
        # the codes of one new token, before a block's first projection: latency
        {"name": "norm 1 token", "op": "norm", "tokens": 1, "n": 4096, "dtype": "bf16", "post": False,
         "residual": True, "gate": "none"},
        # prompts between two blocks: norm of the block's output, its gate by channel, the scaled
        # residual, the next block's norm and codes
        {"name": "norm prompts", "op": "norm", "tokens": 8191, "n": 5120, "dtype": "bf16", "post": True,
         "residual": True, "gate": "channel"},
        # one token's projection: the weight stream
        {"name": "linear 1 row", "op": "linear", "rows": 1, "k": 4096, "n": 4096, "bias": False,
         "dtype": "bf16"},
        # single tokens of 50 requests
        {"name": "linear 50 rows", "op": "linear", "rows": 50, "k": 4096, "n": 11008, "bias": True,
         "dtype": "fp16"},
        # prompts: the matrix cores
        {"name": "linear 2048 rows", "op": "linear", "rows": 2048, "k": 4096, "n": 11008, "bias": False,
         "dtype": "bf16"},
        # one token's feed-forward block
        {"name": "gated 1 row", "op": "gated", "rows": 1, "k": 4096, "n": 11008, "act": "silu",
         "dtype": "bf16"},
        # prompts' feed-forward block
        {"name": "gated 2048 rows", "op": "gated", "rows": 2048, "k": 4096, "n": 11008, "act": "silu",
         "dtype": "bf16"},
        # one request, four tokens drawn from a drafter's distribution: latency
        {"name": "verify chain 1 x 5", "op": "verify", "batch": 1, "tokens": 5, "vocab": 32000,
         "dtype": "fp32", "draft": True, "temperature": 0.8},
        # trees of 24 nodes for 16 requests, some of them greedy
        {"name": "verify tree 16 x 24", "op": "verify", "batch": 16, "tokens": 24, "vocab": 131072,
         "dtype": "bf16", "draft": False, "temperature": 1.0},
        # after the verification: the accepted nodes' rows move up behind the context
        {"name": "compact trees", "op": "compact", "batch": 64, "context": 1000, "tokens": 24,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0},
        # requests that keep their first rows and a window of the newest: most of the bytes of a cache
        {"name": "compact windows", "op": "compact", "batch": 8, "context": 16384, "tokens": 4,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 6001},
        # 8 samples of each of 8 prompts: last step's samples freed, new ones forked, room for drafts
        {"name": "fork 8 x 8", "op": "fork", "prompts": 8, "samples": 8, "context": 4111, "more": 24,
         "kv_heads": 8, "dim": 128, "page": 64},
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "gated", "verify", "compact", "fork", "copy"])
    dtype = rng.choice(["fp32", "fp16", "bf16"])
    if op == "norm":
        n = _between(rng, 64, 20000)
        most = 8191 * 5120 * 2 // (n * SIZES[dtype])
        return {"op": op, "tokens": _between(rng, 1, max(1, min(16384, most))), "n": n, "dtype": dtype,
                "post": rng.random() < 0.5, "residual": rng.random() < 0.8,
                "gate": rng.choice(["none", "channel", "token"])}
    if op in ("linear", "gated"):
        k = 16 * _between(rng, 16, 688) - (rng.randint(1, 15) if rng.random() < 0.1 else 0)
        n = _between(rng, 256, 11008)
        rows = min(_between(rng, 1, 2048), max(1, 2048 * 4096 * 11008 // (k * n)))
        if op == "linear":
            return {"op": op, "rows": rows, "k": k, "n": n, "bias": rng.random() < 0.5, "dtype": dtype}
        return {"op": op, "rows": rows, "k": k, "n": n, "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu"]),
                "dtype": dtype}
    if op == "verify":
        vocab = _between(rng, 1000, 262144)
        batch = _between(rng, 1, 64)
        most = max(2, 16 * 24 * 131072 * 2 // (batch * vocab * SIZES[dtype]))
        draft = rng.random() < 0.5
        tokens = _between(rng, 2, min(64, max(2, most // 2) if draft else most))
        return {"op": op, "batch": batch, "tokens": tokens, "vocab": vocab, "dtype": dtype, "draft": draft,
                "temperature": round(rng.uniform(0.3, 1.5), 2)}
    kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 96, 128, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    row = 2 * kv_heads * (dim + 4)
    if op == "compact":
        batch = _between(rng, 1, 64)
        context = _between(rng, 8, max(8, min(32768, 8 * 16388 * 2112 // (batch * row))))
        wide = rng.random() < 0.5
        return {"op": op, "batch": batch, "context": context, "tokens": 4 if wide else _between(rng, 2, 64),
                "kv_heads": kv_heads, "dim": dim, "page": page,
                "window": rng.randint(1, max(1, context // 2 - 4)) if wide else 0}
    if op == "fork":
        prompts = _between(rng, 1, 32)
        samples = min(_between(rng, 1, 16), max(1, 8 * 16384 * 2112 // (prompts * (64 + 4 * page) * row)))
        # whole pages are shared, one a sample is copied
        most = min(16384, 8 * 16384 * 2112 // (prompts * row)) - 2 * samples * page
        return {"op": op, "prompts": prompts, "samples": samples, "context": _between(rng, 1, max(1, most)),
                "more": rng.randint(1, 64), "kv_heads": kv_heads, "dim": dim, "page": page}
    pages = _between(rng, 2, max(2, 8 * 16384 * 2112 // (page * row)))
    return {"op": op, "pages": pages, "kv_heads": kv_heads, "dim": dim, "page": page,
            "part": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# Sizes that follow from a case alone

def _contexts(case):
    """Ragged context lengths of the requests of a compaction; the first is the longest."""
    c = case["context"]
    return [max(1, c - (b * 7919) % (c // 8 + 1)) for b in range(case["batch"])]


def _paths(case):
    """First row of each request's path, and the rows kept from there on, as offsets in rising order.

    A row that moves comes from behind the rows that are kept, so that a pass leaves the same rows
    however often it has run."""
    base, paths = [], []
    for b, n in enumerate(_contexts(case)):
        if case["window"]:
            w = max(1, min(case["window"], n // 2 - 4))
            base.append(0)
            paths.append(np.concatenate((np.arange(4), np.arange(n - w, n)) if n >= 2 * w + 8 else (np.arange(4),)))
        else:
            rng = np.random.default_rng(b + 100 * case["tokens"])
            count = int(rng.integers(1, min(8, case["tokens"]) + 1))
            stay = int(rng.integers(1, count + 1))
            away = np.sort(rng.permutation(np.arange(count, case["tokens"]))[:count - stay])
            base.append(n)
            paths.append(np.concatenate((np.arange(stay), away)))
    return base, paths


def _fork_pages(case):
    """Pages of a prompt's context, pages of a request's table, pages of the pool."""
    full = -(-case["context"] // case["page"])
    row = -(-(case["context"] + case["more"]) // case["page"]) + 1
    pages = case["prompts"] * (full + 1) + case["prompts"] * case["samples"] * (row - full + 2) + 64
    return full, row, pages


def work(case):
    """Bytes and operations that one pass cannot do without."""
    op = case["op"]
    if op == "norm":
        t, n, es = case["tokens"], case["n"], SIZES[case["dtype"]]
        inputs = (2 if case["residual"] else 1) * t * n * es
        inputs += {"none": 0, "channel": n * es, "token": t * n * es}[case["gate"]]
        # written: the sum, the codes and scales; the codes read back as the values they stand for
        return {"bytes": inputs + 4 * n + (4 * n if case["post"] else 0) + t * n * es + t * (n + 4)
                + t * (5 * n + 4),
                "flops": t * n * (12 if case["post"] else 8)}
    if op in ("linear", "gated"):
        m, k, n, two = case["rows"], case["k"], case["n"], 2 if op == "gated" else 1
        return {"bytes": m * k + 4 * m + two * (n * k + 4 * n) + m * n * SIZES[case["dtype"]],
                "flops": 2 * two * m * n * k}
    if op == "verify":
        b, t, v = case["batch"], case["tokens"], case["vocab"]
        rows = 2 * t - 1 if case["draft"] else t
        return {"bytes": b * rows * v * SIZES[case["dtype"]] + b * t * 20 + b * 12, "flops": b * rows * v * 4}
    row = 2 * case["kv_heads"] * (case["dim"] + 4)
    if op == "compact":
        moved = sum(int((p != np.arange(len(p))).sum()) for p in _paths(case)[1])
        listed_rows = sum(len(p) for p in _paths(case)[1])
        return {"bytes": 2 * moved * row + 4 * listed_rows, "flops": 0}
    if op == "copy":
        moved = sum(_copy_rows(case)) if case["part"] else case["pages"] // 2 * case["page"]
        return {"bytes": 2 * moved * row + 8 * (case["pages"] // 2), "flops": 0}
    full, width, pages = _fork_pages(case)
    new, part = case["prompts"] * case["samples"], case["context"] % case["page"]
    return {"bytes": new * (2 * part * row + 3 * width * 4 + 2 * full * 4) + 2 * pages * 4, "flops": 0}


def _copy_rows(case):
    return [(i * 37) % (case["page"] + 1) for i in range(case["pages"] // 2)]


# ---------------------------------------------------------------------------
# Inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def codes(*shape):
        return normal(*shape).mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)

    def cache(pages):
        shape = (pages, 2, case["kv_heads"], case["page"])
        s["cache"] = torch.randint(-127, 128, shape + (case["dim"],), dtype=torch.int8, generator=g, device=DEV)
        s["scales"] = torch.rand(shape, generator=g, device=DEV).add_(0.5).mul_(0.03)

    s = {"case": dict(case)}
    op = case["op"]
    if op == "norm":
        t, n, dt = case["tokens"], case["n"], DTYPES[case["dtype"]]
        s["x"] = normal(t, n).to(dt)
        s["residual"] = normal(t, n).mul_(3.0).to(dt) if case["residual"] else None
        s["post"] = normal(n).mul_(0.2).add_(1.0) if case["post"] else None
        s["gate"] = (None if case["gate"] == "none" else
                     normal(1 if case["gate"] == "channel" else t, n).mul_(0.5).to(dt))
        s["weight"] = normal(n).mul_(0.2).add_(1.0)
        s["residual_scale"] = 0.875 if case["residual"] else 1.0
        s["out"] = torch.empty((t, n), dtype=dt, device=DEV)
        s["codes"] = torch.empty((t, n), dtype=torch.int8, device=DEV)
        s["code_scales"] = torch.empty(t, device=DEV)
    elif op in ("linear", "gated"):
        m, k, n = case["rows"], case["k"], case["n"]
        s["x"] = codes(m, k)
        s["x_scales"] = normal(m).mul_(0.3).exp_().mul_(0.02)
        for name in ("gate", "up") if op == "gated" else ("",):
            s["w" + name] = codes(n, k)
            s["s" + name] = normal(n).mul_(0.2).exp_().mul_(0.0009 if op == "linear" else 0.03 / math.sqrt(k))
        s["bias"] = normal(n).mul_(0.1) if case.get("bias") else None
        s["out"] = torch.empty((m, n), dtype=DTYPES[case["dtype"]], device=DEV)
    elif op == "verify":
        b, t, v, dt = case["batch"], case["tokens"], case["vocab"], DTYPES[case["dtype"]]
        # a bulk of unlikely tokens and some tens of likely ones a row
        x = normal(b, t, v).mul_(2.0)
        x += (torch.rand((b, t, v), generator=g, device=DEV) < 40.0 / v) * normal(b, t, v).mul_(3.0).add_(8.0)
        s["logits"] = x.to(dt)
        temp = np.full(b, case["temperature"], np.float32)
        if b > 4:
            temp[3::5] = 0.0          # greedy requests among them
        s["temperature"] = dev(temp)
        heat = s["temperature"].clamp(min=0.2).view(-1, 1, 1)
        parent = np.maximum(np.arange(t) - 1, 0) + np.zeros((b, 1), np.int64)
        if not case["draft"]:
            for i in range(1, t):
                parent[:, i] = rng.integers(max(0, i - 4), i, b)
        mask = np.zeros((b, t), np.uint64)
        mask[:, 0] = 1
        for i in range(1, t):
            mask[:, i] = mask[np.arange(b), parent[:, i]] | (np.uint64(1) << np.uint64(i))
        s["mask"] = dev(mask.view(np.int64)) if not case["draft"] else None
        s["parent"] = dev(parent)
        # the drafter: near the target; its tokens are drawn from it
        y = (x + normal(b, t, v).mul_(0.7)).to(dt)
        s["draft"] = y[:, :t - 1].contiguous() if case["draft"] else None
        noise = -torch.log(-torch.log(torch.rand((b, t, v), generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)))
        from_rows = torch.gather(y, 1, s["parent"].unsqueeze(2).expand(b, t, v)).float()
        s["tokens"] = (from_rows / heat + noise).argmax(-1).int()
        s["u"] = torch.rand((b, t), generator=g, device=DEV)
        s["path"] = torch.empty((b, t), dtype=torch.int32, device=DEV)
        s["accepted"] = torch.empty(b, dtype=torch.int32, device=DEV)
        s["next"] = torch.empty(b, dtype=torch.int32, device=DEV)
    elif op == "compact":
        base, paths = _paths(case)
        b, width = case["batch"], max(len(p) for p in paths)
        row = -(-(case["context"] + case["tokens"]) // case["page"])
        cache(b * row)
        s["table"] = dev(rng.permutation(b * row).reshape(b, row).astype(np.int32))
        s["base"] = dev(np.array(base, np.int32))
        s["counts"] = dev(np.array([len(p) for p in paths], np.int32))
        s["path"] = dev(np.stack([np.pad(p, (0, width - len(p)), constant_values=-1) for p in paths]).astype(np.int32))
    elif op == "copy":
        cache(case["pages"])
        half, order = case["pages"] // 2, rng.permutation(case["pages"])
        s["src"], s["dst"] = dev(order[:half].astype(np.int32)), dev(order[half:2 * half].astype(np.int32))
        s["rows"] = dev(np.array(_copy_rows(case), np.int32)) if case["part"] else None
    else:
        full, width, pages = _fork_pages(case)
        p, n = case["prompts"], case["samples"]
        cache(pages)
        table = np.full((p + p * n, width), -1, np.int32)
        refs = np.zeros(pages, np.int32)
        held = rng.permutation(pages)[:p * full].reshape(p, full)
        table[:p, :full] = held
        refs[held] = 1
        lens = np.zeros(p + p * n, np.int32)
        lens[:p] = case["context"]
        s["table"], s["refs"], s["lens"] = dev(table), dev(refs), dev(lens)
        s["src"] = dev(np.repeat(np.arange(p), n).astype(np.int32))
        s["dst"] = dev((p + np.arange(p * n)).astype(np.int32))
        s["more"] = dev(np.concatenate((np.zeros(p), np.full(p * n, case["more"]))).astype(np.int32))
        for name in ("granted", "copy_src", "copy_dst", "copy_rows"):
            s[name] = torch.empty(p * n, dtype=torch.int32, device=DEV)
        s["served"] = torch.empty(p + p * n, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# One pass

def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _own_norm(s):
    import int8_quantized_amd as q8
    q8.q8ta_norm_quantize(s["x"], s["residual"], s["post"], s["gate"], s["residual_scale"], s["weight"],
                          EPS, s["out"], s["codes"], s["code_scales"])
    return {"sum": s["out"], "values": s["codes"] * s["code_scales"].unsqueeze(-1)}


def _own_linear(s):
    import int8_quantized_amd as q8
    return q8.q8ta_linear_per_token(s["x"], s["x_scales"], s["w"], s["s"], s["bias"], "none", s["out"])


def _own_gated(s):
    import int8_quantized_amd as q8
    return q8.q8ta_gated_linear(s["x"], s["x_scales"], s["wgate"], s["sgate"], None, s["wup"], s["sup"], None,
                                s["case"]["act"], s["out"])


def _own_verify(s):
    import int8_quantized_amd as q8
    q8.q8ta_verify_drafts(s["logits"], s["draft"], s["tokens"], None, s["mask"], s["temperature"], None,
                          s["u"], s["path"], s["accepted"], s["next"])
    return {"path": s["path"], "accepted": s["accepted"], "next": s["next"]}


def _own_compact(s):
    import int8_quantized_amd as q8
    q8.q8ta_cache_compact(s["cache"], s["scales"], s["table"], s["base"], s["path"], s["counts"])
    return {"cache": s["cache"], "scales": s["scales"]}


def _own_copy(s):
    import int8_quantized_amd as q8
    q8.q8ta_pages_copy(s["cache"], s["scales"], s["src"], s["dst"], s["rows"])
    return {"cache": s["cache"], "scales": s["scales"]}


def _own_fork(s):
    import int8_quantized_amd as q8
    page = s["case"]["page"]
    q8.q8ta_pages_release(s["table"], s["lens"], page, s["dst"], None, s["refs"])
    q8.q8ta_pages_fork(s["table"], s["lens"], page, s["src"], s["dst"], s["refs"], s["granted"],
                       s["copy_src"], s["copy_dst"], s["copy_rows"])
    q8.q8ta_pages_copy(s["cache"], s["scales"], s["copy_src"], s["copy_dst"], s["copy_rows"])
    q8.q8ta_pages_take(s["table"], s["lens"], page, s["more"], s["refs"], s["served"])
    return {n: s[n] for n in ("table", "refs", "lens", "granted", "served", "cache", "scales")}


def _rms(x):
    return 1.0 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()


def _plain_norm(s):
    # in 64 bits: codes are whole numbers, and a value next to a border may not cross it
    b = s["x"].double()
    if s["post"] is not None:
        b = b * _rms(b) * s["post"].double()
    if s["gate"] is not None:
        b = b * s["gate"].double()
    if s["residual"] is not None:
        b = b + s["residual"].double() * s["residual_scale"]
    h = b.float().to(s["x"].dtype)
    z = h.double()
    z = z * _rms(z) * s["weight"].double()
    top = z.abs().amax(-1, keepdim=True)
    code = (z * 127.0 / torch.where(top > 0, top, 1.0)).round().to(torch.int8)
    return {"sum": h, "values": code * (top / 127.0).float()}


def _product(s, w, scales):
    return torch.matmul(s["x"].float(), w.float().t()) * s["x_scales"].unsqueeze(1) * scales


def _plain_linear(s):
    y = _product(s, s["w"], s["s"])
    return (y if s["bias"] is None else y + s["bias"]).to(s["out"].dtype)


def _plain_gated(s):
    g, act = _product(s, s["wgate"], s["sgate"]), s["case"]["act"]
    if act == "silu":
        g = g / (1.0 + torch.exp(-g))
    elif act == "gelu":
        g = g * 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        g = g * 0.5 * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))
    else:
        g = torch.maximum(g, torch.zeros_like(g))
    return (g * _product(s, s["wup"], s["sup"])).to(s["out"].dtype)


def _shares(logits, temperature):
    """Softmax in 64 bits over the vocabulary; the largest alone (the first of them) where T is 0."""
    x = logits.double()
    t = temperature.double().view(-1, 1, 1)
    top = x.amax(-1, keepdim=True)
    w = ((x - top) / torch.where(t > 0, t, 1.0)).exp()
    first = torch.arange(x.shape[-1], device=x.device) == x.argmax(-1, keepdim=True)
    w = torch.where(t > 0, w, first.double())
    return w / w.sum(-1, keepdim=True)


def _plain_verify(s):
    b, t = s["tokens"].shape
    p, token, u = _shares(s["logits"], s["temperature"]), s["tokens"].long(), s["u"].double()
    row = torch.arange(b, device=p.device)
    q = _shares(s["draft"], s["temperature"]) if s["draft"] is not None else None
    at, count = torch.zeros_like(row), torch.ones_like(row)
    path = torch.full((b, t), -1, dtype=torch.int64, device=p.device)
    path[:, 0] = 0
    left = p[:, 0].clone()                # of the current node: what is not rejected yet
    done = torch.zeros_like(row, dtype=torch.bool)
    for i in range(1, t):                 # a node's children follow it, and are tried in their order
        tried = (s["parent"][:, i] == at) & ~done
        mine = left[row, token[:, i]]
        if q is None:
            good = tried & (u[:, i] * left.sum(-1) < mine)
            less = left.clone()
            less[row, token[:, i]] = 0.0
        else:
            good = tried & (u[:, i] * q[row, i - 1, token[:, i]] < mine)
            greedy = s["temperature"] <= 0
            less = torch.where(greedy.unsqueeze(1), left, (left - q[:, i - 1]).clamp(min=0.0))
            done |= tried & ~good
        left = torch.where((tried & ~good).unsqueeze(1), less, left)
        left = torch.where(good.unsqueeze(1), p[:, i], left)
        # a greedy request's token is the largest of its node, whatever was drafted
        at = torch.where(good, i, at)
        path.scatter_(1, count.clamp(max=t - 1).unsqueeze(1), torch.where(
            good, i, path[row, count.clamp(max=t - 1)]).unsqueeze(1))
        count = count + good
    left = torch.where((s["temperature"] > 0).unsqueeze(1), left, p[row, at])
    below = left.cumsum(-1)
    next_token = (below <= u[:, :1] * below[:, -1:]).sum(-1).clamp(max=p.shape[-1] - 1)
    return {"path": path.int(), "accepted": count.int(), "next": next_token.int()}


def _plain_compact(s):
    page = s["case"]["page"]
    i = torch.arange(s["path"].shape[1], device=DEV)
    # (a row that stays where it is is written onto itself, in place of a list of those that move)
    on = (i < s["counts"].unsqueeze(1)) & (s["path"] >= 0)
    src = s["base"].long().unsqueeze(1) + torch.where(on, s["path"].long(), 0)
    dst = s["base"].long().unsqueeze(1) + torch.where(on, i, 0)
    from_page, to_page = (s["table"].long().gather(1, r // page) for r in (src, dst))
    for name in ("cache", "scales"):
        s[name][to_page, :, :, dst % page] = s[name][from_page, :, :, src % page]
    return {"cache": s["cache"], "scales": s["scales"]}


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    rows = torch.arange(s["case"]["page"], device=DEV)
    for name in ("cache", "scales"):
        new = s[name][src]
        if s["rows"] is not None:
            on = (rows < s["rows"].unsqueeze(1)).view((-1, 1, 1, rows.numel()) + (1,) * (new.dim() - 4))
            new = torch.where(on, new, s[name][dst])
        s[name][dst] = new
    return {"cache": s["cache"], "scales": s["scales"]}


def _plain_fork(s):
    page, table, refs, lens = s["case"]["page"], s["table"], s["refs"], s["lens"]
    src, dst, width = s["src"].long(), s["dst"].long(), s["table"].shape[1]
    j = torch.arange(width, device=DEV)
    # release
    held = table[dst]
    refs.index_add_(0, held.clamp(min=0).view(-1).long(), -(held >= 0).view(-1).int())
    table[dst] = -1
    lens[dst] = 0
    # fork: whole pages shared, the lowest free page for a part of one
    n = lens[src]
    part = n % page
    free = torch.argsort((refs > 0).int(), stable=True).int()
    rank = (part > 0).cumsum(0) - 1
    granted = (part == 0) | (rank < (refs <= 0).sum())
    fresh = torch.where((part > 0) & granted, free[rank.clamp(0, refs.numel() - 1)], -1)
    shared = granted.unsqueeze(1) & (j < (n // page).unsqueeze(1))
    rows = torch.where(shared, table[src], -1)
    refs.index_add_(0, rows.clamp(min=0).view(-1).long(), (rows >= 0).view(-1).int())
    refs.index_add_(0, fresh.clamp(min=0).long(), (fresh >= 0).int())
    old = torch.where(fresh >= 0, table[src, (n // page).clamp(max=width - 1).long()], -1)
    rows = torch.where((j == (n // page).unsqueeze(1)) & (fresh >= 0).unsqueeze(1), fresh.unsqueeze(1), rows)
    table[dst] = torch.where(granted.unsqueeze(1), rows, table[dst])
    lens[dst] = torch.where(granted, n, lens[dst])
    # copy
    to = torch.where(fresh >= 0, fresh, s["cache"].shape[0] - 1).long()
    on = (torch.arange(page, device=DEV) < part.unsqueeze(1)) & (fresh >= 0).unsqueeze(1)
    for name in ("cache", "scales"):
        new = s[name][old.clamp(min=0).long()]
        keep = on.view((-1, 1, 1, page) + (1,) * (new.dim() - 4))
        s[name][to] = torch.where(keep, new, s[name][to])
    # take
    first = (table >= 0).sum(1)
    want = torch.where(s["more"] > 0, (lens + s["more"] + page - 1) // page, 0)
    need = (want - first).clamp(min=0)
    before = need.cumsum(0) - need
    free = torch.argsort((refs > 0).int(), stable=True).int()
    served = (need == 0) | (before + need <= (refs <= 0).sum())
    at = j - first.unsqueeze(1)
    new = (at >= 0) & (at < need.unsqueeze(1)) & served.unsqueeze(1)
    picked = free[(before.unsqueeze(1) + at).clamp(0, refs.numel() - 1)]
    table.copy_(torch.where(new, picked, table))
    refs.index_add_(0, torch.where(new, picked, 0).view(-1).long(), new.view(-1).int())
    return {"table": table, "refs": refs, "lens": lens, "granted": granted.int(), "served": served.int(),
            "cache": s["cache"], "scales": s["scales"]}


_OWN = {"norm": _own_norm, "linear": _own_linear, "gated": _own_gated, "verify": _own_verify,
        "compact": _own_compact, "copy": _own_copy, "fork": _own_fork}
_PLAIN = {"norm": _plain_norm, "linear": _plain_linear, "gated": _plain_gated, "verify": _plain_verify,
          "compact": _plain_compact, "copy": _plain_copy, "fork": _plain_fork}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, written apart from the plain forms

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "gated": _exact_gated, "verify": _exact_verify,
            "compact": _exact_compact, "copy": _exact_copy, "fork": _exact_fork}[case["op"]](case, s)


def _exact_norm(case, s):
    def unit(v):
        return v * torch.rsqrt((v * v).sum(1, keepdim=True) / case["n"] + EPS)
    x = s["x"].to(torch.float64)
    if case["post"]:
        x = s["post"] * unit(x)
    if case["gate"] != "none":
        x = s["gate"].to(torch.float64) * x
    if case["residual"]:
        x = torch.add(x, s["residual"].to(torch.float64), alpha=s["residual_scale"])
    # the codes are those of the sum as it is stored
    z = s["weight"] * unit(x.to(torch.float32).to(DTYPES[case["dtype"]]).to(torch.float64))
    top = z.abs().max(1, keepdim=True).values
    return {"sum": x, "values": torch.where(top > 0, torch.round(z * 127 / top) * top / 127, 0.0)}


def _exact_linear(case, s):
    y = (s["x"].double() * s["x_scales"].double()[:, None]) @ (s["w"].double() * s["s"].double()[:, None]).t()
    return y + s["bias"].double() if case["bias"] else y


def _exact_gated(case, s):
    x = s["x"].double() * s["x_scales"].double()[:, None]
    g, u = (x @ (s["w" + n].double() * s["s" + n].double()[:, None]).t() for n in ("gate", "up"))
    if case["act"] == "silu":
        g = g * torch.sigmoid(g)
    elif case["act"] == "gelu":
        g = g * torch.special.ndtr(g)
    elif case["act"] == "gelu_tanh":
        # tanh by the logistic function: (1 + tanh z) / 2 = 1 / (1 + e^-2z)
        g = g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))
    else:
        g = g.clamp(min=0.0)
    return g * u


def _exact_verify(case, s):
    b, t = s["tokens"].shape
    token, u = s["tokens"].cpu().numpy(), s["u"].double().cpu().numpy()
    parent, temp = s["parent"].cpu().numpy(), s["temperature"].cpu().numpy().astype(np.float64)

    def shares(rows, r, i):
        x = rows[r, i].double().cpu().numpy()
        if temp[r] <= 0:
            return np.eye(1, len(x), int(x.argmax()))[0]
        w = np.exp((x - x.max()) / temp[r])
        return w / math.fsum(w)
    path, accepted, following = np.full((b, t), -1), [], []
    for r in range(b):
        node, kept = 0, [0]
        while True:
            p = shares(s["logits"], r, node)
            children = [i for i in range(node + 1, t) if parent[r, i] == node]
            step = None
            for c in children:
                if case["draft"]:
                    d = shares(s["draft"], r, node)
                    if u[r, c] * d[token[r, c]] < p[token[r, c]]:
                        step = c
                        break
                    p = np.maximum(p - d, 0.0) if temp[r] > 0 else p
                else:
                    if u[r, c] * math.fsum(p) < p[token[r, c]]:
                        step = c
                        break
                    if temp[r] > 0:
                        p[token[r, c]] = 0.0
            if step is None:
                break
            node = step
            kept.append(step)
        sums = np.cumsum(p)
        following.append(min(int(np.searchsorted(sums, u[r, 0] * sums[-1], side="right")), len(p) - 1))
        path[r, :len(kept)] = kept
        accepted.append(len(kept))
    return {n: torch.from_numpy(np.array(v, np.int32)) for n, v in
            (("path", path), ("accepted", accepted), ("next", following))}


def _exact_compact(case, s):
    page, table = case["page"], s["table"].cpu().numpy()
    base, paths = _paths(case)
    new = {n: s[n].clone() for n in ("cache", "scales")}
    for b, (first, path) in enumerate(zip(base, paths)):
        src, dst = first + path, first + np.arange(len(path))
        where = [torch.from_numpy(a.astype(np.int64)).to(DEV) for a in
                 (table[b, src // page], src % page, table[b, dst // page], dst % page)]
        for n in new:
            new[n][where[2], :, :, where[3]] = s[n][where[0], :, :, where[1]]
    return new


def _exact_copy(case, s):
    rows = _copy_rows(case) if case["part"] else [case["page"]] * (case["pages"] // 2)
    at = torch.arange(case["page"], device=DEV)
    n = torch.tensor(rows, device=DEV)
    pair, row = torch.nonzero(at < n[:, None], as_tuple=True)
    new = {k: s[k].clone() for k in ("cache", "scales")}
    for k in new:
        new[k][s["dst"].long()[pair], :, :, row] = s[k][s["src"].long()[pair], :, :, row]
    return new


def _exact_fork(case, s):
    page, table = case["page"], s["table"].cpu().numpy()
    refs, lens = s["refs"].cpu().numpy(), s["lens"].cpu().numpy()
    cache, scales = s["cache"].clone(), s["scales"].clone()
    src, dst = s["src"].cpu().numpy(), s["dst"].cpu().numpy()
    more = s["more"].cpu().numpy()
    for r in dst:
        for p in table[r][table[r] >= 0]:
            refs[p] -= 1
        table[r], lens[r] = -1, 0

    def lowest(n):
        return np.flatnonzero(refs <= 0)[:n]
    granted, spent = [], 0
    free = lowest(len(refs))
    for a, r in zip(src, dst):
        full, part = divmod(int(lens[a]), page)
        fine = spent + (part > 0) <= len(free)
        granted.append(int(fine))
        if part and fine:
            new, old = int(free[spent]), int(table[a, full])
            cache[new, :, :, :part], scales[new, :, :, :part] = cache[old, :, :, :part], scales[old, :, :, :part]
        if fine:
            table[r, :full], lens[r] = table[a, :full], lens[a]
            refs[table[a, :full]] += 1
            if part:
                table[r, full] = new
                refs[new] = 1
        spent += part > 0
    free, spent, served = lowest(len(refs)), 0, []
    for r in range(len(lens)):
        first = int((table[r] >= 0).sum())
        need = max(0, -(-int(lens[r] + more[r]) // page) - first) if more[r] > 0 else 0
        served.append(int(need == 0 or spent + need <= len(free)))
        if served[-1]:
            table[r, first:first + need] = free[spent:spent + need]
            refs[free[spent:spent + need]] = 1
        spent += need
    whole = {"table": table, "refs": refs, "lens": lens, "granted": granted, "served": served}
    return {**{n: torch.from_numpy(np.array(v, np.int32)) for n, v in whole.items()}, "cache": cache,
            "scales": scales}
