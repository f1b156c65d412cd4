"""q8ta_sample against its definition in 64 bits (numpy, a stable sort): filters alone and together,
ties, masked logits, greedy rows, types, sizes from one token up, and the calls it refuses.

Tokens are whole numbers and equal.  A log-probability is one rounding to fp32 of a 64-bit value
whose weights are held to 2^-shift (shift >= 38), so half a step of fp32 and 2^-30 cover it.
"""
import math

import numpy as np
import pytest

import int8_quantized_amd as q8

torch = pytest.importorskip("torch")

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def definition(row, t, k, p, mp, u):
    row = np.where(np.isnan(row), -np.inf, row.astype(np.float64))
    if np.isneginf(row).all():
        return -1, -math.inf
    order = np.argsort(-row, kind="stable")
    if not t > 0:
        return int(order[0]), 0.0
    top = row[order[0]]

    def weight(x):
        d = np.where(x == top, 0.0, (x - np.where(np.isinf(top) & (x == top), 0.0, top)) / t)
        return np.exp(d)
    w = weight(row[order])
    if k > 0:
        w[k:] = 0.0
    keep = np.arange(len(w)) < (k if k > 0 else len(w))
    if p < 1:
        keep &= np.cumsum(w) - w < p * w.sum()
    keep &= w >= mp
    keep[0] = True
    kept = np.sort(order[keep])
    wk = weight(row[kept])
    cum = np.cumsum(wk)
    i = min(int(np.searchsorted(cum, u * cum[-1], side="right")), len(kept) - 1)
    while wk[i] == 0.0:
        i -= 1
    return int(kept[i]), math.log(wk[i] / cum[-1])


def run(logits, t, k, p, mp, u, dtype="fp32", stride=0, logprobs=True):
    x = torch.from_numpy(logits.astype(np.float32)).to(TYPES[dtype]).cuda()
    B, V = x.shape
    if stride:
        wide = torch.full((B, V + stride), 99.0, dtype=x.dtype, device="cuda")
        wide[:, :V] = x
        x = wide[:, :V]

    def dev(v, ty):
        return None if v is None else torch.from_numpy(np.asarray(v, ty)).cuda()
    tokens = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((B,), 3.0, device="cuda") if logprobs else None
    q8.q8ta_sample(x, dev(t, np.float32), dev(k, np.int32), dev(p, np.float32), dev(mp, np.float32),
                   dev(u, np.float32), tokens, lp)
    torch.cuda.synchronize()
    return x.float().cpu().numpy(), tokens.cpu().numpy(), None if lp is None else lp.double().cpu().numpy()


def check(logits, t, k, p, mp, u, **kw):
    B = len(logits)
    x, tokens, lp = run(logits, t, k, p, mp, u, **kw)

    def at(v, i, off, ty):
        return off if v is None else ty(v[i])
    for i in range(B):
        tok, want = definition(x[i], np.float32(t[i]).astype(np.float64), at(k, i, 0, int),
                               np.float64(at(p, i, 1.0, np.float32)),
                               np.float64(at(mp, i, 0.0, np.float32)), np.float64(np.float32(u[i])))
        assert tokens[i] == tok, (i, tokens[i], tok)
        if lp is not None:
            assert lp[i] == want or abs(lp[i] - want) <= abs(want) * 2.0 ** -24 * 1.001 + 2.0 ** -30, i


def rows(B, V, seed, likely=40):
    g = np.random.default_rng(seed)
    x = g.standard_normal((B, V)) * 2.0
    x += (g.random((B, V)) < likely / V) * (g.standard_normal((B, V)) * 3.0 + 8.0)
    return x, g


SETTINGS = [(0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0), (0.7, 50, 0.9, 0.0), (1.0, 0, 0.95, 0.0),
            (0.8, 100, 0.9, 0.02), (1.5, 1, 0.5, 0.1), (0.3, 0, 1.0, 0.1), (1.2, 20, 1.0, 0.0),
            (0.9, 1000, 0.5, 0.0), (1.0, 0, 0.9, 0.02), (0.8, 7, 1.0, 0.3), (1.0, 1000, 0.999, 0.0),
            (1.3, 0, 0.5, 0.0), (1.0, 3000, 0.97, 0.0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 63, 64, 65, 1000, 1025, 4097, 32000, 100003])
def test_sample_settings(V, dtype):
    B = len(SETTINGS)
    x, g = rows(B, V, V)
    t, k, p, mp = zip(*SETTINGS)
    check(x, t, k, p, mp, g.random(B), dtype=dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_sample_one_row_many_numbers(dtype):
    """Every kept token is met by its own stretch of u, the borders included."""
    x, g = rows(1, 300, 5)
    B = 200
    u = (np.arange(B) / B).astype(np.float32)
    check(np.repeat(x, B, 0), [1.0] * B, [40] * B, [0.9] * B, [0.01] * B, u, dtype=dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [37, 5000, 70001])
def test_sample_ties(V):
    """Few distinct logits: borders fall among equal ones, the lowest indices stay."""
    B = len(SETTINGS) * 2
    g = np.random.default_rng(V)
    x = g.integers(0, 4, (B, V)).astype(np.float32)
    x[::3] = 1.0                                   # all equal
    t, k, p, mp = (list(v) * 2 for v in zip(*SETTINGS))
    check(x, t, k, p, mp, g.random(B), dtype="bf16")


@pytest.mark.gpu
def test_sample_top_p_border_on_equal_weights():
    x = np.zeros((4, 8))
    check(x, [1.0] * 4, [0, 0, 4, 4], [0.5, 0.25, 0.5, 0.75], [0.0] * 4, [0.99, 0.99, 0.99, 0.0])


@pytest.mark.gpu
@pytest.mark.parametrize("V", [64, 20000, (1 << 19) + 5])
def test_sample_settings_that_are_no_numbers(V):
    """A NaN keeps the first token alone: no sum is below it, no weight reaches it."""
    x, g = rows(4, V, V)
    nan = np.nan
    _, tokens, lp = run(x, [1.0, 1.0, nan, 1.0], [0, 5000, 0, 20], [nan, nan, 0.9, 0.9], [0.0, 0.0, 0.0, nan],
                        g.random(4))
    assert (tokens == x.astype(np.float32).argmax(1)).all() and (lp == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("V", [64, 20000])
def test_sample_masked_logits(V):
    B = len(SETTINGS)
    t, k, p, mp = zip(*SETTINGS)
    for seed, fill in enumerate((-np.inf, np.finfo(np.float32).min, np.nan)):
        x, g = rows(B, V, V + seed)
        allowed = g.integers(0, V, (B, 5))
        m = np.ones((B, V), bool)
        np.put_along_axis(m, allowed, False, 1)
        x = np.where(m, fill, x)
        x[3] = -np.inf                              # nothing allowed
        x[4] = -np.inf
        x[4, V // 2] = -3.0                         # one token
        if np.isnan(fill):
            x[5] = np.nan
        check(x, t, k, p, mp, g.random(B))


@pytest.mark.gpu
def test_sample_infinite_and_extreme():
    x, g = rows(6, 500, 1)
    x[0, [3, 77, 400]] = np.inf
    x[1] *= 1e30
    x[2] = x[2] * 1e-30
    x[3, 9] = 3e38
    x[4, ::2] = -3e38
    check(x, [1.0, 0.5, 1.0, 2.0, 1e-4, 50.0], [0, 0, 0, 5, 0, 0], [0.9] * 6, [0.0] * 6,
          [0.5, 0.3, 0.999, 0.1, 0.7, 0.2])


@pytest.mark.gpu
def test_sample_off_settings_strides_and_no_logprobs():
    x, g = rows(5, 777, 3)
    u = g.random(5)
    check(x, [1.0] * 5, None, None, None, u, stride=5, dtype="fp16")
    check(x, [1.0] * 5, None, [0.8] * 5, None, u, stride=1)
    check(x, [0.6] * 5, [9] * 5, None, None, u, logprobs=False)
    check(x, [0.6, -1.0, 1.0, 1.0, 1.0], [9, 9, -4, 10 ** 9, 777], [2.0, 0.5, 0.0, -1.0, 1.0],
          [0.0, 0.0, 0.0, 0.0, 2.0], u)


@pytest.mark.gpu
def test_sample_many_rows_repeat_and_graph():
    x, g = rows(300, 9001, 8)
    n = len(SETTINGS)
    t, k, p, mp = zip(*[SETTINGS[i % n] for i in range(300)])
    u = g.random(300)
    check(x, t, k, p, mp, u)
    _, a, la = run(x, t, k, p, mp, u)
    _, b, lb = run(x, t, k, p, mp, u)
    assert (a == b).all() and (la == lb).all()
    f = [torch.from_numpy(np.asarray(v, ty)).cuda() for v, ty in
         ((x, np.float32), (t, np.float32), (k, np.int32), (p, np.float32), (mp, np.float32),
          (u, np.float32))]
    tok = torch.zeros(300, dtype=torch.int32, device="cuda")
    lp = torch.zeros(300, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q8.q8ta_sample(*f, tok, lp, stream=side)
    torch.cuda.synchronize()
    assert (tok.cpu().numpy() == a).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q8.q8ta_sample(*f, tok, lp)
    for _ in range(3):
        tok.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert (tok.cpu().numpy() == a).all()
        q8.q8ta_sample(*f, tok, lp)


# ---------------------------------------------------------------- refusals (no GPU)
FAKE = 4096   # never dereferenced: every call below fails validation first
GOOD = dict(logits=FAKE, stride=100, dtype=0, rows=3, vocab=100, t=FAKE, k=None, p=None, mp=None,
            u=FAKE, tokens=FAKE, logprobs=None, s=None)


def refuse(status, **kw):
    a = dict(GOOD)
    a.update(kw)
    assert q8.lib().q8ta_sample(*a.values()) == status, kw
    assert "q8ta_sample" in q8.q8ta_last_error()


def test_sample_refusals():
    for name in ("logits", "t", "u", "tokens"):
        refuse(q8.Q8TA_ERR_NULL, **{name: None})
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(vocab=0), dict(vocab=(1 << 24) + 1),
                dict(stride=99), dict(stride=1 << 40)):
        refuse(q8.Q8TA_ERR_SHAPE, **bad)
    refuse(q8.Q8TA_ERR_UNSUPPORTED, dtype=3)


def test_sample_no_rows_launches_nothing():
    a = dict(GOOD, rows=0, logits=None)
    assert q8.lib().q8ta_sample(*a.values()) == q8.Q8TA_OK
