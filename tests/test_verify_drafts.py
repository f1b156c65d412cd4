"""q8ta_verify_drafts against its definition in 64 bits (numpy, one request at a time): chains drawn from a
drafter and trees, all types, strides, ragged counts, masks, infinite and NaN logits, random numbers at their
ends; that kept and following tokens are distributed as the target's; and the calls it refuses.

Whole numbers have to be equal.  A kept child is decided by comparing a random number with a share whose
sum is off by up to 1e-8 of itself, a next token by one with 64-bit sums: the definition says how near the
random numbers come to their borders, and a case nearer than 1e-6 (1e-10 for the next token) is no case.
"""
import math

import numpy as np
import pytest

import int8_quantized_amd as q8

torch = pytest.importorskip("torch")

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def shares(x, t):
    """softmax(x / t) in 64 bits: t <= 0 (or NaN) all on the first largest, infinite ones alone; None where all are -inf."""
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    if top == -np.inf:
        return None
    if not t > 0:
        return np.eye(1, len(x), int(x.argmax()))[0]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x == top, 1.0, np.exp((x - top) / t) if np.isfinite(top) else 0.0)
    return w / math.fsum(w)


def parents_of(T, mask):
    if mask is None:
        return [i - 1 for i in range(T)]
    out = []
    for i in range(T):
        above = int(np.uint64(mask[i])) & ((1 << i) - 1)
        out.append(above.bit_length() - 1)
    return out


def definition(c):
    x = c["logits"].double().numpy()
    d = None if c["draft"] is None else c["draft"].double().numpy()
    B, T, V = x.shape
    path, accepted, following, near = np.full((B, T), -1), [], [], []
    for b in range(B):
        count = T if c["counts"] is None else min(max(int(c["counts"][b]), 0), T)
        t = float(c["temperature"][b])
        td = t if c["draft_temperature"] is None else float(c["draft_temperature"][b])
        parent = parents_of(T, None if c["mask"] is None else c["mask"][b])
        margin, kept, token = math.inf, [], -1
        node = 0 if count > 0 else None
        while node is not None:
            kept.append(node)
            p = shares(x[b, node], t)
            if p is None:
                break
            left, step = p.copy(), None
            for i in range(node + 1, count):
                if parent[i] != node:
                    continue
                tok, u = int(c["ids"][b, i]), float(c["u"][b, i])
                u = 0.0 if u < 0 else u       # (a NaN stays, and is below nothing)
                good_id = 0 <= tok < V
                mine = left[tok] if good_id else 0.0
                if t > 0 and d is not None:
                    q = shares(d[b, node], td)
                    q = np.zeros(V) if q is None else q
                    share = q[tok] if good_id else 0.0
                    good = u * share < mine
                    margin = min(margin, abs(u * share - mine) if good_id else math.inf)
                    if not good:
                        left = np.maximum(left - q, 0.0)
                elif t > 0:
                    good = u * math.fsum(left) < mine
                    margin = min(margin, abs(u * math.fsum(left) - mine) / max(math.fsum(left), 1e-300) if mine > 0 else math.inf)
                    if not good and good_id:
                        left[tok] = 0.0
                else:
                    good = mine > 0
                if good:
                    step = i
                    break
                if d is not None:
                    break
            if step is None:
                if not math.fsum(left) > 0 or not t > 0:
                    left = p
                sums = np.cumsum(left)
                u = float(c["u"][b, 0])
                goal = (0.0 if u < 0 else u) * sums[-1]
                over = np.flatnonzero((sums > goal) & (left > 0))
                token = int(over[0]) if len(over) else int(np.flatnonzero(left > 0)[-1])
                if t > 0 and 0 <= u < 1:
                    margin = min(margin, 1e4 * np.abs(sums - goal).min() / sums[-1] if goal else math.inf)
            node = step
        path[b, :len(kept)] = kept
        accepted.append(len(kept))
        following.append(token)
        near.append(margin)
    return path, np.array(accepted), np.array(following), np.array(near)


def make(B, T, V, dtype="fp32", draft=True, tree=None, seed=0, temperature=0.8, counts=None, spread=2.0, near=0.7, pad=0,
         offset=0):
    g = np.random.default_rng(seed)
    tree = not draft if tree is None else tree
    rows = (g.standard_normal((B, T, V)) * spread).astype(np.float32)
    rows += (g.random((B, T, V)) < 4.0 / V) * 6.0
    other = rows + g.standard_normal(rows.shape).astype(np.float32) * near
    t = np.full(B, temperature, np.float32) if np.isscalar(temperature) else np.array(temperature, np.float32)

    def typed(a):
        whole = torch.zeros(a.shape[:2] + (V + pad + offset,), dtype=TYPES[dtype])
        part = whole[:, :, offset:offset + V]
        part.copy_(torch.from_numpy(a))
        return part
    mask = None
    if tree:
        m = np.zeros((B, T), np.uint64)
        m[:, 0] = 1
        for i in range(1, T):
            up = g.integers(max(0, i - 4), i, B)
            m[:, i] = m[np.arange(B), up] | (np.uint64(1) << np.uint64(i))
        mask = m.view(np.int64)
    ids = np.zeros((B, T), np.int32)
    for b in range(B):
        parent = parents_of(T, None if mask is None else mask[b])
        for i in range(1, T):
            src = other[b, max(parent[i], 0)] / max(t[b], 0.3)
            ids[b, i] = (src - np.log(-np.log(g.uniform(1e-7, 1 - 1e-7, V)))).argmax()
    return dict(logits=typed(rows), draft=typed(other[:, :T - 1]) if draft else None, ids=ids,
                counts=None if counts is None else np.array(counts, np.int32), mask=mask, temperature=t,
                draft_temperature=None, u=g.random((B, T)).astype(np.float32))


def gpu(t):
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return torch.from_numpy(np.ascontiguousarray(t)).cuda()
    if t.numel() == 0:
        return t.cuda()
    base = torch.as_strided(t, (t.untyped_storage().nbytes() // t.element_size(),), (1,), 0).cuda()
    return torch.as_strided(base, t.shape, t.stride(), t.storage_offset())


def run(c):
    B, T = c["ids"].shape
    path = torch.full((B, T), 77, dtype=torch.int32, device="cuda")
    accepted, following = (torch.full((B,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    q8.q8ta_verify_drafts(gpu(c["logits"]), gpu(c["draft"]), gpu(c["ids"]), gpu(c["counts"]), gpu(c["mask"]),
                          gpu(c["temperature"]), gpu(c["draft_temperature"]), gpu(c["u"]), path, accepted, following)
    return path.cpu().numpy(), accepted.cpu().numpy(), following.cpu().numpy()


def check(c):
    want = definition(c)
    got = run(c)
    clear = want[3] > 1e-6
    assert clear.mean() > 0.9 or len(clear) < 10, want[3]
    for name, a, b in zip(("path", "accepted", "next"), got, want):
        assert (a[clear] == b[clear]).all(), (name, a, b, want[3])
    return want


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (1, 2, 5), (3, 5, 64), (2, 4, 4095), (4, 7, 4096), (2, 6, 4097), (5, 64, 1000),
                                   (1, 5, 32000), (70, 3, 300), (2, 9, 50001), (1, 3, 140000)])
def test_verify(B, T, V, draft, dtype):
    check(make(B, T, V, dtype, draft, seed=B * T + V))


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
def test_verify_longest_vocabulary(draft):
    check(make(1, 2, 1 << 24, "bf16", draft, seed=3))


@pytest.mark.gpu
@pytest.mark.parametrize("pad,offset", [(0, 1), (5, 0), (8, 8), (4, 4)])
def test_verify_strides_and_alignment(pad, offset):
    for dtype in TYPES:
        check(make(3, 5, 5000, dtype, True, seed=1, pad=pad, offset=offset))
        check(make(3, 12, 5000, dtype, False, seed=2, pad=pad, offset=offset))


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("seed", range(4))
def test_verify_temperatures_and_counts(draft, seed):
    """Greedy requests, hot and cold ones, counts of none to more than all."""
    temps = [0.0, 0.8, -1.0, 5.0, 0.05, float("nan"), 1.0, 1e-30, 1e30]
    check(make(9, 8, 777, "fp32", draft, seed=seed, temperature=temps, counts=[8, 0, 3, 1, 99, 5, -4, 8, 2]))


@pytest.mark.gpu
@pytest.mark.parametrize("temps", [[0.5, 2.0, 1.0, 0.7], [0.0, -1.0, float("nan"), 0.0]])
def test_verify_a_drafter_at_its_own_temperature(temps):
    for seed in range(4):
        c = make(4, 6, 500, "fp16", True, seed=seed)
        c["draft_temperature"] = np.array(temps, np.float32)
        if not temps[0] > 0:     # a greedy drafter: its largest
            d = c["draft"].double().numpy()
            c["ids"][:, 1:] = d.argmax(2)
            c["ids"][0, 2] = 3
        check(c)


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
def test_verify_logits_that_are_not_finite(draft):
    for seed in range(6):
        c = make(6, 5, 300, "fp32", draft, seed=seed)
        x = c["logits"]
        x[0, :, ::2] = -math.inf                     # a filter
        x[1, 0] = -math.inf                          # nothing at the first token
        x[2, 1] = -math.inf                          # nothing at the second
        x[3, :, 7] = math.inf
        x[3, :, 9] = math.inf                        # infinite ones share the weight
        x[4, :, 5:200] = math.nan
        c["ids"][3, 1:] = 9
        if draft:
            c["draft"][5, 0] = -math.inf             # a drafter that gives nothing
            c["draft"][0, :, ::3] = -math.inf
            c["draft"][3, 1, 9] = math.inf
        check(c)


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
def test_verify_random_numbers_at_their_ends(draft):
    for value in (0.0, -3.0, 1.0, 2.0, math.nan, math.inf, -math.inf, 1.0 - 2.0 ** -24):
        for where in (slice(0, 1), slice(1, None), slice(None)):
            c = make(4, 6, 200, "fp32", draft, seed=5)
            c["u"][:, where] = value
            check(c)


@pytest.mark.gpu
def test_verify_ids_outside_the_vocabulary_and_doubled():
    for seed in range(6):
        for draft in (True, False):
            c = make(5, 7, 40, "bf16", draft, seed=seed)
            c["ids"][0, 1] = 40
            c["ids"][1, 1:3] = -1
            c["ids"][2, 2] = 1 << 30
            c["ids"][:, 0] = -99                     # the known token is not looked up
            check(c)
        c = make(6, 9, 12, "fp32", False, seed=seed)     # brothers with one id: kept once or never
        c["mask"] = np.full((6, 9), 1, np.uint64)
        c["mask"] = (c["mask"] | (np.uint64(1) << np.arange(9, dtype=np.uint64))).view(np.int64)
        c["ids"][:, 1:] = c["ids"][:, 1:] % 3
        check(c)


@pytest.mark.gpu
def test_verify_masks():
    """Forests, tokens without a parent, bits of later tokens, and the chain by its mask."""
    c = make(4, 10, 100, "fp32", False, seed=3)
    m = c["mask"].view(np.uint64)
    m[0] = np.uint64(0)                              # nobody has a parent
    m[1] |= ~np.uint64(0) << np.uint64(10)           # bits past the tokens
    m[2, 3:] &= ~np.uint64(7)                        # some have lost theirs
    check(c)
    chain = make(3, 8, 60, "fp32", False, tree=False, seed=4)
    plain = run(chain)
    chain["mask"] = np.tile(np.array([(2 << i) - 1 for i in range(8)], np.int64), (3, 1))
    assert all((a == b).all() for a, b in zip(plain, run(chain)))
    check(chain)


@pytest.mark.gpu
def test_verify_does_not_depend_on_the_batch():
    c = make(40, 6, 9000, "bf16", True, seed=8)
    whole = run(c)
    for b in (0, 17, 39):
        one = {k: v[b:b + 1] if v is not None else None for k, v in c.items()}
        assert all((a[b:b + 1] == o).all() for a, o in zip(whole, run(one)))


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,V,draft", [(40000, 64, 5, False), (65535, 33, 9, True)])
def test_verify_of_more_requests_than_one_launch(B, T, V, draft):
    g = torch.Generator(device="cuda").manual_seed(B)
    x = torch.randn(B, T, V, generator=g, device="cuda")
    y = torch.randn(B, T - 1, V, generator=g, device="cuda") if draft else None
    ids = torch.randint(0, V, (B, T), generator=g, dtype=torch.int32, device="cuda")
    u = torch.rand(B, T, generator=g, device="cuda") * 0.3
    heat = torch.rand(B, generator=g, device="cuda") + 0.5

    def run_rows(a, b):
        outs = [torch.full(s, -7, dtype=torch.int32, device="cuda") for s in ((b - a, T), (b - a,), (b - a,))]
        q8.q8ta_verify_drafts(x[a:b], None if y is None else y[a:b], ids[a:b], None, None, heat[a:b], None, u[a:b],
                              *outs)
        return outs

    whole, parts = run_rows(0, B), [run_rows(a, min(a + 9999, B)) for a in range(0, B, 9999)]
    for i, o in enumerate(whole):
        assert torch.equal(o, torch.cat([p[i] for p in parts]))
    assert (whole[1] > 1).any() and ((whole[2] >= 0) & (whole[2] < V)).all()


def frequencies_near(counts, p, n):
    # five standard deviations of a count
    assert (np.abs(counts - n * p) <= 5 * np.sqrt(n * p * (1 - p)) + 1).all(), (counts / n, p)


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
def test_tokens_are_distributed_as_the_targets(draft):
    """The first token after the known one, kept or drawn, over 40000 requests of the same logits."""
    n, V = 40000, 11
    g = np.random.default_rng(12)
    x, y = (g.standard_normal(V) * 1.5).astype(np.float32), (g.standard_normal(V) * 1.5).astype(np.float32)
    p, q = shares(x.astype(np.float64), 1.0), shares(y.astype(np.float64), 1.0)
    T = 3 if draft else 4
    logits = torch.from_numpy(np.broadcast_to(x, (n, T, V)).copy()).cuda()
    ids = np.zeros((n, T), np.int32)
    if draft:
        ids[:, 1:] = g.choice(V, (n, 2), p=q)
        mask, other = None, torch.from_numpy(np.broadcast_to(y, (n, T - 1, V)).copy()).cuda()
    else:
        ids[:, 1:] = np.argsort(-y)[:3]              # three brothers, the drafter's most likely
        mask, other = torch.tensor([[1, 3, 5, 9]]).repeat(n, 1).cuda(), None
    u = torch.from_numpy(g.random((n, T)).astype(np.float32)).cuda()
    path = torch.empty(n, T, dtype=torch.int32, device="cuda")
    accepted, following = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(2))
    q8.q8ta_verify_drafts(logits, other, torch.from_numpy(ids).cuda(), None, mask, torch.ones(n, device="cuda"), None, u, path,
                          accepted, following)
    path, accepted, following = path.cpu().numpy(), accepted.cpu().numpy(), following.cpu().numpy()
    first = np.where(accepted > 1, ids[np.arange(n), np.maximum(path[:, 1], 0)], following)
    frequencies_near(np.bincount(first, minlength=V), p, n)
    second = accepted > 1                            # and the one after it
    after = np.where(accepted > 2, ids[np.arange(n), np.maximum(path[:, 2], 0)], following)[second]
    frequencies_near(np.bincount(after, minlength=V), p, int(second.sum()))


@pytest.mark.gpu
def test_verify_captured_beside_eager_calls():
    c, d = make(4, 9, 6000, "bf16", False, seed=1), make(4, 9, 6000, "bf16", False, seed=2)
    a = [gpu(c[k]) for k in ("logits", "ids", "mask", "temperature", "u")]
    b = [gpu(d[k]) for k in ("logits", "ids", "mask", "temperature", "u")]

    def outs():
        return (torch.empty(4, 9, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda"),
                torch.empty(4, dtype=torch.int32, device="cuda"))

    def call(t, o):
        q8.q8ta_verify_drafts(t[0], None, t[1], None, t[2], t[3], None, t[4], *o)
    want, other = outs(), outs()
    call(a, want)
    call(b, other)
    got, eager = outs(), outs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a, got)
    side = torch.cuda.Stream()
    for _ in range(4):
        for o in got:
            o.fill_(7)
        graph.replay()
        with torch.cuda.stream(side):
            call(b, eager)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(torch.equal(x, y) for x, y in zip(eager, other))


# ---------------------------------------------------------------- refusals
FAKE = 4096


def test_verify_refuses():
    base = dict(x=FAKE, bs=640, ts=64, d=None, dbs=0, dts=0, dt=0, B=2, T=5, V=64, ids=FAKE, counts=None, mask=None, t=FAKE, td=None,
                u=FAKE, p=FAKE, a=FAKE, n=FAKE, st=None)

    def call(**kw):
        rc = q8.lib().q8ta_verify_drafts(*{**base, **kw}.values())
        return rc, q8.q8ta_last_error()
    for kw, status, words in [
            (dict(dt=-1), q8.Q8TA_ERR_UNSUPPORTED, "dtype"), (dict(B=-1), q8.Q8TA_ERR_SHAPE, "batch"), (dict(B=65536), q8.Q8TA_ERR_SHAPE, "batch"),
            (dict(T=0), q8.Q8TA_ERR_SHAPE, "tokens"), (dict(T=65), q8.Q8TA_ERR_SHAPE, "tokens"), (dict(V=0), q8.Q8TA_ERR_SHAPE, "vocab"),
            (dict(V=(1 << 24) + 1), q8.Q8TA_ERR_SHAPE, "vocab"), (dict(bs=-1), q8.Q8TA_ERR_SHAPE, "strides"),
            (dict(ts=1 << 41), q8.Q8TA_ERR_SHAPE, "strides"), (dict(d=FAKE, dts=-5), q8.Q8TA_ERR_SHAPE, "strides"),
            (dict(d=FAKE, mask=FAKE), q8.Q8TA_ERR_UNSUPPORTED, "chains")]:
        rc, said = call(**kw)
        assert rc == status and words in said, (kw, rc, said)
    for name in ("x", "ids", "t", "u", "p", "a", "n"):
        assert call(**{name: None})[0] == q8.Q8TA_ERR_NULL, name
    assert call(B=0)[0] == q8.Q8TA_OK
    assert call(B=0, d=None, dbs=-7)[0] == q8.Q8TA_OK      # no drafter, no strides


@pytest.mark.gpu
def test_binding_refuses_shapes():
    c = make(2, 4, 50, "fp32", True)
    ok = dict(logits=gpu(c["logits"]), draft=gpu(c["draft"]), ids=gpu(c["ids"]), counts=None, mask=None,
              t=gpu(c["temperature"]), td=None, u=gpu(c["u"]), path=torch.empty(2, 4, dtype=torch.int32, device="cuda"),
              a=torch.empty(2, dtype=torch.int32, device="cuda"), n=torch.empty(2, dtype=torch.int32, device="cuda"))
    q8.q8ta_verify_drafts(*ok.values())
    for bad in (dict(draft=ok["draft"][:, :2]), dict(draft=ok["draft"].half()), dict(ids=ok["ids"][:, :3]), dict(u=ok["u"][:1]),
                dict(path=ok["path"][:, :3]), dict(t=ok["t"][:1]), dict(a=ok["a"][:1]), dict(counts=ok["a"][:1]),
                dict(td=ok["t"][:1]), dict(logits=ok["logits"][0])):
        with pytest.raises(ValueError):
            q8.q8ta_verify_drafts(*{**ok, **bad}.values())
    with pytest.raises((ValueError, TypeError)):
        q8.q8ta_verify_drafts(*{**ok, "ids": ok["ids"].long()}.values())
