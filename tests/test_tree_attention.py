"""q8ta_tree_attention against its definition in 64 bits (numpy): grouped heads, odd lengths, pages
in any order, trees, rows that see nothing, rows of the cache that hold anything, splits over the
keys, and the calls it refuses.

Tolerances, with c_j = |softmax_j value_j|: a probability's rounding to fp16 is off by at most 2^-12
of it (2^-11 leaves room for its 32-bit steps and for those that fp16 holds below its normal range,
under 2^-24 of the largest), the output's own rounding by half a step of the type.  A score is a
sum of dim exact products in 32 bits, off by at most dim * 2^-24 of sum |q k|, which moves its
probability by as much and lse by at most the largest of them.
"""
import math

import numpy as np
import pytest

import int8_quantized_amd as q8

torch = pytest.importorskip("torch")

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def make(B, T, hq, hk, d, page, lens, seed=0, dtype="bf16", tree=True, counts=None, spare=1,
         q_scale=1.5, scale_spread=0.3, fill=None):
    g = np.random.default_rng(seed)
    need = max(-(-(n + T) // page) for n in lens) + spare
    pages = B * need + 3
    cache = np.clip(np.rint(g.standard_normal((pages, 2, hk, page, d)) * 36), -128, 127).astype(np.int8)
    scales = (np.exp(g.standard_normal((pages, 2, hk, page)) * scale_spread) * 0.03).astype(np.float32)
    table = g.permutation(pages)[:B * need].reshape(B, need).astype(np.int32)
    q = torch.from_numpy((g.standard_normal((B, T, hq, d)) * q_scale).astype(np.float32))
    mask = np.zeros((B, T), np.uint64)
    mask[:, 0] = 1
    for t in range(1, T):
        p = g.integers(max(0, t - 4), t, B)
        mask[:, t] = mask[np.arange(B), p] | (np.uint64(1) << np.uint64(t))
    c = dict(q=q.to(TYPES[dtype]), cache=cache, scales=scales, table=table,
             lens=np.array(lens, np.int32), counts=None if counts is None else np.array(counts, np.int32),
             mask=mask.view(np.int64) if tree else None, scale=1.0 / math.sqrt(d))
    if fill is not None:      # rows that no query sees hold `fill` as their scale
        keep = np.zeros(scales.shape[:1] + (page,), bool)
        for b in range(B):
            for s in range(lens[b] + (T if counts is None else counts[b])):
                keep[table[b, s // page], s % page] = True
        scales[~np.broadcast_to(keep[:, None, None], scales.shape)] = fill
    return c


def definition(c):
    q = c["q"].double().numpy()
    B, T, hq, d = q.shape
    pages, _, hk, page, _ = c["cache"].shape
    out, lse = np.zeros(q.shape), np.full((B, T, hq), -np.inf)
    tol, tol_lse = np.zeros(q.shape), np.zeros((B, T, hq))
    for b in range(B):
        n = max(0, int(c["lens"][b]))
        used = T if c["counts"] is None else int(np.clip(c["counts"][b], 0, T))
        total = min(n + used, c["table"].shape[1] * page)
        n = min(n, total)
        pg = c["table"][b][np.arange(total) // page].astype(np.int64)
        good = (pg >= 0) & (pg < pages)
        at = np.where(good, pg, 0)
        off = np.arange(total) % page
        for h in range(hq):
            kh = h // (hq // hk)
            ks, vs = (c["scales"][at, p, kh, off].astype(np.float64)[:, None] for p in (0, 1))
            k = c["cache"][at, 0, kh, off].astype(np.float64) * ks
            v = c["cache"][at, 1, kh, off].astype(np.float64) * vs
            for t in range(used):
                m = int(np.uint64(c["mask"][b, t])) if c["mask"] is not None else (2 << t) - 1
                seen = good & np.array([j < n or (m >> (j - n)) & 1 == 1 for j in range(total)], bool)
                if not seen.any():
                    continue
                s = k[seen] @ q[b, t, h] * c["scale"]
                off_s = (np.abs(k[seen]) @ np.abs(q[b, t, h])) * c["scale"] * (d + 8) * 2.0 ** -24
                top = s.max()
                w = np.exp(s - top)
                p = w / w.sum()
                out[b, t, h] = p @ v[seen]
                lse[b, t, h] = top + math.log(w.sum())
                rel = 2.0 ** -11 + 2 * off_s.max() + 2.0 ** -20
                tol[b, t, h] = (p * rel) @ np.abs(v[seen]) + 2.0 ** -23 * np.abs(v[seen]).max() * \
                    min(1.0, len(s) * 2.0 ** -8)
                tol_lse[b, t, h] = off_s.max() + 2.0 ** -21 * max(1.0, abs(lse[b, t, h]))
    return out, lse, tol, tol_lse


def run(c, strided=False, with_lse=True):
    q = c["q"].cuda()
    if strided:
        B, T, hq, d = q.shape
        wide = torch.zeros((B, T, hq + 3, d), dtype=q.dtype, device="cuda")
        wide[:, :, 1:hq + 1] = q
        q = wide[:, :, 1:hq + 1]
    dev = {k: None if v is None else torch.from_numpy(v).cuda() for k, v in c.items()
           if k not in ("q", "scale")}
    out = torch.full(c["q"].shape, 5.0, dtype=q.dtype, device="cuda")
    lse = torch.full(c["q"].shape[:3], 5.0, device="cuda") if with_lse else None
    q8.q8ta_tree_attention(q, dev["cache"], dev["scales"], dev["table"], dev["lens"], dev["counts"],
                           dev["mask"], c["scale"], out, lse)
    torch.cuda.synchronize()
    return out, lse


def check(c, **kw):
    out, lse = run(c, **kw)
    want, want_lse, tol, tol_lse = definition(c)
    eps = torch.finfo(out.dtype).eps / 2
    got = out.double().cpu().numpy()
    err = np.abs(got - want)
    bad = ~(err <= tol * 1.01 + np.abs(want) * eps * 1.01 + 1e-7)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])
    if lse is not None:
        g = lse.double().cpu().numpy()
        none = np.isneginf(want_lse)
        assert (np.isneginf(g) == none).all()
        assert (np.abs(g - want_lse)[~none] <= tol_lse[~none]).all()
    return out, lse


SIZES = [  # B, T, hq, hk, d, page, lens
    (1, 1, 1, 1, 64, 16, [0]), (1, 1, 8, 2, 128, 16, [1]), (2, 1, 8, 1, 64, 16, [63, 64]),
    (3, 1, 4, 4, 80, 32, [15, 16, 17]), (2, 1, 32, 8, 128, 16, [700, 255]), (1, 1, 14, 2, 256, 64, [1000]),
    (2, 5, 8, 2, 128, 16, [130, 0]), (1, 17, 4, 4, 64, 32, [300]), (2, 24, 8, 2, 128, 32, [257, 511]),
    (1, 64, 8, 1, 64, 128, [513]), (2, 33, 7, 1, 80, 16, [100, 1]), (1, 64, 4, 2, 256, 48, [200]),
    (1, 3, 6, 2, 16, 16, [77]), (1, 2, 4, 1, 144, 16, [90]), (2, 9, 16, 2, 96, 256, [40, 300])]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("size", SIZES)
def test_tree_attention(size, dtype):
    check(make(*size, dtype=dtype, seed=sum(size[:6])))


@pytest.mark.gpu
@pytest.mark.parametrize("size", [(2, 6, 8, 2, 128, 16, [50, 3]), (1, 64, 4, 4, 64, 16, [0])])
def test_tree_attention_chain_strides_and_no_lse(size):
    c = make(*size, tree=False, seed=1)
    out, _ = check(c, strided=True)
    again, _ = run(c, with_lse=False)
    assert torch.equal(out, again)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 40])
def test_tree_attention_counts_and_empty_rows(T):
    c = make(5, T, 4, 2, 64, 16, [20, 0, 0, 77, 0], seed=2, counts=[T, 0, 2, 3, T + 9])
    c["mask"][2, 1] = 0            # in use, no context, an empty mask: sees nothing
    c["mask"][4, :2] = 0
    out, lse = check(c)
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    assert (out[2, 1:] == 0).all() and (out[4, :2] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fill", [math.nan, math.inf, -3e38])
@pytest.mark.parametrize("T", [1, 3, 30])
def test_tree_attention_unseen_rows_hold_anything(T, fill):
    c = make(2, T, 8, 2, 64, 16, [70, 5], seed=3, fill=fill)
    check(c)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("fill", [math.nan, math.inf, -6e4])
@pytest.mark.parametrize("T", [2, 7, 40])
def test_tree_attention_queries_not_in_use_hold_anything(T, fill, dtype):
    c = make(3, T, 8, 2, 64, 16, [300, 5, 0], seed=12, counts=[T - 1, 1, 0], dtype=dtype)
    for b, n in enumerate((T - 1, 1, 0)):
        c["q"][b, n:] = fill * (1e30 if dtype == "bf16" else 1.0)
    clean = dict(c, q=torch.where(c["q"].float().abs() < 100, c["q"], torch.zeros_like(c["q"])))
    want, want_lse, tol, tol_lse = definition(clean)
    out, lse = run(c)
    got, g = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (np.abs(got - want) <= tol * 1.01 + np.abs(want) * torch.finfo(out.dtype).eps * 0.505 + 1e-7).all()
    none = np.isneginf(want_lse)
    assert (np.isneginf(g) == none).all()
    assert (np.abs(g - np.where(none, 0, want_lse))[~none] <= tol_lse[~none]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fill", [math.nan, math.inf, 3e38])
@pytest.mark.parametrize("T,n", [(3, 70), (24, 500), (40, 9)])
def test_tree_attention_drafted_rows_that_others_see_hold_anything(T, n, fill):
    """A drafted token's cache row whose scales are no numbers spoils the tokens that see it and no
    other; one that no token sees may hold any number too."""
    c = make(1, T, 8, 2, 64, 16, [n], seed=13)
    bad = 1
    if math.isfinite(fill):
        c["mask"][0, 2:] &= ~(1 << bad)
        c["mask"][0, bad] = 1
    saw = ((c["mask"][0].view(np.uint64) >> np.uint64(bad)) & np.uint64(1)) == 1
    assert saw.any() != math.isfinite(fill) and not saw.all()
    want, want_lse, tol, tol_lse = definition(c)
    s = n + bad
    c["scales"][c["table"][0, s // 16], :, :, s % 16] = fill
    out, lse = run(c)
    err = np.abs(out.double().cpu().numpy() - want)
    ok = err <= tol * 1.01 + np.abs(want) * torch.finfo(out.dtype).eps * 0.505 + 1e-7
    assert ok[0, ~saw].all()
    assert (np.abs(lse.double().cpu().numpy() - want_lse) <= tol_lse)[0, ~saw].all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20])
def test_tree_attention_heads_of_different_size(T):
    """Queries of one head 2^60 times another's: each keeps its own precision."""
    c = make(1, T, 8, 1, 64, 16, [100], seed=14)
    c["q"][:, :, 1::2] *= 2.0 ** -60
    c["q"][:, :, 0] *= 2.0 ** 20
    check(c)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20])
def test_tree_attention_wide_scores_and_scales(T):
    """Scores of hundreds (one key takes all), value scales over many orders."""
    check(make(2, T, 4, 2, 128, 32, [400, 33], seed=4, q_scale=60.0, dtype="bf16"))
    check(make(2, T, 4, 2, 128, 32, [400, 33], seed=5, scale_spread=3.0, q_scale=0.05, dtype="fp16"))
    c = make(1, T, 4, 2, 64, 16, [200], seed=6)
    c["scales"][:, 1] *= np.float32(1e-30)
    out, lse = run(c)
    assert torch.isfinite(lse).all() and (out.float().abs() < 1e-25).all()
    c["q"][:] = 0                                   # uniform weights
    c["scales"][:, 1] = 0.0                         # values of zero
    out, lse = check(c)
    assert (out == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20])
def test_tree_attention_long_context_is_split(T):
    check(make(1, T, 2, 1, 64, 64, [9001], seed=7))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 20])
def test_tree_attention_bad_pages_and_lengths(T):
    c = make(4, T, 4, 2, 64, 16, [100, 90, 30, 30], seed=8)
    pages = c["cache"].shape[0]
    c["table"][0, 2], c["table"][1, 0], c["table"][1, 5] = -1, pages, 1 << 30
    c["lens"][2] = -7
    c["lens"][3] = 1 << 30          # keys past the table's pages are not there
    check(c)


@pytest.mark.gpu
def test_tree_attention_repeats_bit_for_bit():
    c = make(2, 24, 8, 2, 128, 16, [3000, 1234], seed=10)
    a, b = run(c), run(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_tree_attention_on_another_stream_and_in_a_graph():
    c = make(2, 3, 8, 2, 64, 16, [2000, 777], seed=11)
    want, _ = run(c)
    dev = {k: torch.from_numpy(v).cuda() for k, v in c.items() if k not in ("q", "scale", "counts")}
    q, out = c["q"].cuda(), torch.zeros_like(want)

    def call(stream=None):
        q8.q8ta_tree_attention(q, dev["cache"], dev["scales"], dev["table"], dev["lens"], None,
                               dev["mask"], c["scale"], out, None, stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        call()


# ---------------------------------------------------------------- refusals (no GPU)
FAKE = 4096   # never dereferenced: every call below fails validation first
GOOD = dict(q=FAKE, qb=1024, qt=512, qh=64, dtype=2, batch=2, tokens=2, heads=8, kv_heads=2, dim=64,
            cache=FAKE, scales=FAKE, pages=9, page=16, table=FAKE, table_pages=4, lens=FAKE,
            counts=None, mask=None, scale=0.125, out=FAKE, lse=None, s=None)


def refuse(status, **kw):
    a = dict(GOOD)
    a.update(kw)
    assert q8.lib().q8ta_tree_attention(*a.values()) == status, kw
    assert "q8ta_tree_attention" in q8.q8ta_last_error()


def test_tree_attention_refusals():
    for name in ("q", "cache", "scales", "table", "lens", "out"):
        refuse(q8.Q8TA_ERR_NULL, **{name: None})
    for bad in (dict(batch=-1), dict(batch=65536), dict(tokens=0), dict(tokens=65), dict(heads=0),
                dict(kv_heads=0), dict(heads=7), dict(heads=65536, kv_heads=1), dict(dim=0),
                dict(heads=65535, kv_heads=65535, tokens=64), dict(pages=0), dict(page=0),
                dict(batch=65535, heads=65535, kv_heads=65535, tokens=1),
                dict(table_pages=0), dict(table_pages=1 << 27), dict(page=1 << 31),
                dict(pages=1 << 40), dict(qb=-1), dict(qt=1 << 41)):
        refuse(q8.Q8TA_ERR_SHAPE, **bad)
    for bad in (dict(dtype=0), dict(dtype=3), dict(dim=72), dict(dim=272), dict(page=24),
                dict(cache=FAKE + 8), dict(scales=FAKE + 4)):
        refuse(q8.Q8TA_ERR_UNSUPPORTED, **bad)
    for bad in (0.0, -1.0, math.nan, math.inf, 1e-60):
        refuse(q8.Q8TA_ERR_QPARAM, scale=bad)


def test_tree_attention_no_requests_launches_nothing():
    a = dict(GOOD, batch=0, q=None, out=None)
    assert q8.lib().q8ta_tree_attention(*a.values()) == q8.Q8TA_OK
