"""q8ta_linear_lora against its definition in 64 bits (torch): one row to hundreds, adapters in runs
and scattered, ranks of their own, rows without one, types, odd sizes and alignments, and the calls
it refuses.

Tolerances: the base term is three roundings of an exact integer (its sum to fp32, two products and
an addition: 4 * 2^-24 of the terms' magnitudes); the adapter's two sums are K and rank products in
32 bits, off by at most (K + rank + 8) * 2^-24 of the sums of magnitudes, and where the second
product runs on the matrix cores t is held to 2^-16 (16-bit outputs) or 2^-21 (fp32) of its row;
then one rounding to the type.
"""
import numpy as np
import pytest

import int8_quantized_amd as q8

torch = pytest.importorskip("torch")

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def make(M, K, N, r, na, ids, ad="bf16", out="fp32", seed=0, zp=5, scales=True, ranks=None, bias=True,
         offset=0):
    g = np.random.default_rng(seed)

    def codes(*shape):
        n = int(np.prod(shape))
        buf = torch.zeros(n + offset, dtype=torch.int8, device="cuda")
        v = np.clip(np.rint(g.standard_normal(n) * 40), -128, 127).astype(np.int8)
        buf[offset:] = torch.from_numpy(v).cuda()
        return buf[offset:].view(*shape)

    def normal(*shape):
        return torch.from_numpy(g.standard_normal(shape).astype(np.float32)).cuda()
    c = dict(x=codes(M, K), s_in=0.021, zp=zp, w=codes(N, K), ws=normal(N).abs_().mul_(0.001) + 1e-4,
             bias=normal(N) if bias else None,
             a=(normal(na, r, K) / np.sqrt(K)).to(TYPES[ad]), b=(normal(na, N, r) / np.sqrt(r)).to(TYPES[ad]),
             ad_scales=normal(na).abs_() + 0.5 if scales else None,
             ranks=None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device="cuda"),
             ids=torch.from_numpy(np.asarray(ids, np.int32)).cuda(), out=TYPES[out])
    return c


def run(c, act="none", stream=None, out=None):
    if out is None:
        out = torch.full((c["x"].shape[0], c["w"].shape[0]), 3.0, dtype=c["out"], device="cuda")
    q8.q8ta_linear_lora(c["x"], c["s_in"], c["zp"], c["w"], c["ws"], c["bias"], c["a"], c["b"],
                        c["ad_scales"], c["ranks"], c["ids"], act, out, stream=stream)
    return out


def definition(c, act):
    x = c["x"].double() - c["zp"]
    s_in = float(np.float32(c["s_in"]))
    M, K = x.shape
    acc = x @ c["w"].double().t()
    y = acc * s_in * c["ws"].double()
    mag = y.abs()
    if c["bias"] is not None:
        y = y + c["bias"].double()
        mag = mag + c["bias"].double().abs()
    tol = mag * 4 * 2.0 ** -24
    na, r = c["a"].shape[:2]
    for ad in range(na):
        rows = (c["ids"] == ad).nonzero().squeeze(1)
        rk = r if c["ranks"] is None else int(c["ranks"][ad].clamp(0, r))
        if len(rows) == 0 or rk == 0:
            continue
        f = s_in * (1.0 if c["ad_scales"] is None else float(c["ad_scales"][ad]))
        A, B = c["a"][ad, :rk].double(), c["b"][ad, :, :rk].double()
        t = f * (x[rows] @ A.t())
        tm = f * (x[rows].abs() @ A.abs().t())
        y[rows] += t @ B.t()
        part = 2.0 ** -21 if c["out"] == torch.float32 else 2.0 ** -16
        low = t.abs().amax(1, keepdim=True) * part
        tol[rows] += (tm @ B.abs().t()) * ((K + rk + 8) * 2.0 ** -24) + low * B.abs().sum(1)
        tol[rows] += (t @ B.t()).abs() * 2.0 ** -23
    if act == "relu":
        y = y.clamp(min=0)
    return y, tol


def check(c, act="none"):
    got = run(c, act).double()
    want, tol = definition(c, act)
    eps = torch.finfo(c["out"]).eps / 2
    tiny = torch.finfo(c["out"]).smallest_normal * torch.finfo(c["out"]).eps
    bad = ~((got - want).abs() <= tol * 1.01 + want.abs() * eps * 1.01 + tiny)
    assert not bad.any(), (bad.nonzero()[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


def scattered(M, na, seed=0):
    return np.random.default_rng(seed).integers(-1, na, M)


def in_runs(M, na, runs, seed=0):
    g = np.random.default_rng(seed)
    return g.integers(-1, na, runs)[np.arange(M) * runs // M]


@pytest.mark.gpu
@pytest.mark.parametrize("ad", ["fp16", "bf16"])
@pytest.mark.parametrize("out", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("M,K,N,r,na", [
    (1, 64, 16, 4, 1), (1, 4096, 300, 16, 4), (2, 256, 33, 8, 3), (4, 1040, 100, 64, 2), (5, 512, 257, 32, 5),
    (16, 256, 64, 16, 40), (17, 272, 31, 8, 3), (50, 1024, 130, 32, 24), (64, 64, 1, 4, 2),
    (65, 192, 48, 16, 7), (130, 320, 100, 64, 5)])
def test_linear_lora(M, K, N, r, na, out, ad):
    check(make(M, K, N, r, na, scattered(M, na, M), ad, out, seed=M + K, zp=(M * 7) % 41 - 20))


@pytest.mark.gpu
@pytest.mark.parametrize("ad", ["fp16", "bf16"])
@pytest.mark.parametrize("out", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("M,K,N,r,na,runs", [
    (200, 512, 300, 16, 3, 4), (300, 1024, 520, 64, 5, 7), (513, 2048, 769, 32, 4, 20),
    (1030, 1088, 1100, 8, 6, 1030), (700, 1040, 513, 64, 4, 3), (2050, 1024, 4200, 64, 6, 9)])
def test_linear_lora_prompts(M, K, N, r, na, runs, out, ad):
    check(make(M, K, N, r, na, in_runs(M, na, runs, M), ad, out, seed=M + K))


@pytest.mark.gpu
@pytest.mark.parametrize("ad", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N,r,na,offset", [
    (3, 1, 5, 1, 1, 0), (7, 15, 9, 3, 2, 0), (40, 100, 65, 5, 3, 0), (70, 1001, 40, 20, 4, 0),
    (9, 64, 33, 8, 2, 1), (300, 1037, 520, 12, 3, 0), (520, 1024, 520, 100, 2, 8), (2, 40, 7, 512, 2, 0)])
def test_linear_lora_odd_sizes_and_alignment(M, K, N, r, na, offset, ad):
    check(make(M, K, N, r, na, scattered(M, na, M), ad, "fp32", seed=M, offset=offset))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 90, 600])
def test_linear_lora_ranks_ids_and_optional_tensors(M):
    na, r = 5, 32
    ids = scattered(M, na, 1)
    ids[0], ids[1] = na, -(1 << 31)                 # outside: no adapter
    c = make(M, 1024, 520, r, na, ids, seed=2, ranks=[0, 3, 16, 40, 32], scales=False, bias=False)
    c["a"][1, 3:] = float("nan")                    # past an adapter's rank: not numbers
    c["b"][1, :, 3:] = float("nan")
    c["b"][2, :, 16:] = float("inf")
    check(c)
    check(c, "relu")
    c["ids"][:] = -1
    check(c)


@pytest.mark.gpu
@pytest.mark.parametrize("ad", ["fp16", "bf16"])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N", [(40, 100), (200, 300), (2050, 4200)])
def test_linear_lora_adapter_that_is_no_number_spoils_its_own_rows_only(M, N, out, ad):
    c = make(M, 1024, N, 24, 4, scattered(M, 4, 9), ad, out, seed=8)
    want = run(c)
    own = c["ids"] == 2
    c["b"][2, ::3, 5] = float("inf")
    c["b"][2, 1, 20] = float("nan")
    got = run(c)
    assert torch.equal(got[~own], want[~own])
    assert not torch.isfinite(got[own][:, ::3]).any() and torch.isfinite(got[own][:, 2::3]).all()
    c["a"][2, 0, 7] = float("nan")
    assert torch.equal(run(c)[~own], want[~own])


@pytest.mark.gpu
@pytest.mark.parametrize("ad", ["fp16", "bf16"])
@pytest.mark.parametrize("out", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("M,K,N,offset", [(1100, 1037, 1100, 0), (1030, 1024, 1111, 3), (2100, 1024, 4200, 0),
                                          (2050, 1100, 4199, 0)])
def test_linear_lora_large_products_in_detail(M, K, N, offset, out, ad):
    """What the small sizes above cover, where the product is a GEMM of large tiles."""
    na, r = 5, 32
    c = make(M, K, N, r, na, in_runs(M, na, 40, 1), ad, out, seed=9, ranks=[0, 3, 16, 40, 32], scales=False,
             bias=False, offset=offset)
    c["a"][1, 3:] = float("nan")
    c["b"][1, :, 3:] = float("nan")
    c["b"][2, :, 16:] = float("inf")
    check(c)
    check(c, "relu")
    want = run(c)
    own = c["ids"] == 4
    c["b"][4, ::3, 5] = float("inf")
    got = run(c)
    assert torch.equal(got[~own], want[~own])
    assert not torch.isfinite(got[own][:, ::3]).any() and torch.isfinite(got[own][:, 2::3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 40, 520])
@pytest.mark.parametrize("zp", [-128, 127])
def test_linear_lora_zero_points_and_far_adapters(M, zp):
    c = make(M, 1024, 512, 16, 2, scattered(M, 2, 4) | 0, "fp16", "fp32", seed=5, zp=zp)
    c["a"] *= 300.0                                 # t of thousands
    c["ad_scales"] *= 200.0
    c["b"] *= 0.001
    check(c)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 50, 600])
def test_linear_lora_without_adapter_is_the_dequantized_sum(M):
    c = make(M, 512, 300, 8, 2, [-1] * M, seed=6)
    acc = torch.empty((M, 300), dtype=torch.int32, device="cuda")
    q8.q8ta_linear_acc(c["x"], c["zp"], c["w"], acc)
    want = (acc.float() * np.float32(c["s_in"])) * c["ws"] + c["bias"]
    assert torch.equal(run(c), want)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [2, 40, 600])
def test_linear_lora_repeats_streams_and_graph(M):
    c = make(M, 1024, 520, 16, 4, scattered(M, 4, 3), out="bf16", seed=7)
    want = run(c)
    assert torch.equal(run(c), want)
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(c, stream=side, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(c, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        run(c, out=out)


# ---------------------------------------------------------------- refusals (no GPU)
FAKE = 4096   # never dereferenced: every call below fails validation first
GOOD = dict(x=FAKE, M=4, K=64, s_in=0.02, zp=3, w=FAKE, N=32, ws=FAKE, bias=None, a=FAKE, b=FAKE, ad=2,
            na=2, r=8, scales=None, ranks=None, ids=FAKE, act=b"none", out=FAKE, ot=0, s=None)


def refuse(status, **kw):
    a = dict(GOOD)
    a.update(kw)
    assert q8.lib().q8ta_linear_lora(*a.values()) == status, kw
    assert "q8ta_linear_lora" in q8.q8ta_last_error()


def test_linear_lora_refusals():
    for name in ("x", "w", "ws", "a", "b", "ids", "out"):
        refuse(q8.Q8TA_ERR_NULL, **{name: None})
    for bad in (dict(M=0), dict(K=0), dict(N=-1), dict(M=(1 << 21) + 1), dict(N=1 << 31), dict(r=0),
                dict(r=513), dict(na=0), dict(na=1 << 25), dict(N=1 << 30, K=1 << 30)):
        refuse(q8.Q8TA_ERR_SHAPE, **bad)
    for bad in (dict(s_in=0.0), dict(s_in=float("nan")), dict(zp=128), dict(zp=-129)):
        refuse(q8.Q8TA_ERR_QPARAM, **bad)
    for bad in (dict(ad=0), dict(ad=3), dict(ot=3), dict(act=b"gelu"), dict(act=None)):
        refuse(q8.Q8TA_ERR_UNSUPPORTED, **bad)
