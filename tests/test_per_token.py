"""q8ta_norm_quantize, q8ta_quantize_per_token, q8ta_linear_per_token and q8ta_gated_linear against their
definitions in 64 bits: types, strides, odd sizes and alignment, each kernel's sizes, values that are not
finite, ties of the codes, and the calls they refuse.

Tolerances.  A stored sum is off by half a step of its type, after one rounding to fp32.  Codes are those
of the sum as it is stored, formed in 64 bits: equal, but where the quotient is within 1e-9 of a tie,
which the order of 64-bit operations decides.  A scale is off by half a step of fp32.

A product (acc xs) ws has three roundings to fp32 (the sum of integers, two products), the bias adds one, the
output's own rounding half a step of its type.  The gated block: an activation's slope is at most 1.13; its own
steps (an exponential and a reciprocal of one unit each, a sum, two products) make 2^-21 of it, and the roundings
inside the argument of the error function and of the logistic of the tanh form 2^-23 of the gate's product.
"""
import math

import numpy as np
import pytest

import int8_quantized_amd as q8

torch = pytest.importorskip("torch")

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
U32 = 2.0 ** -24
EPS = 1e-6


def half_step(t):
    return torch.finfo(t).eps / 2


def smallest(t):
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps


# ---------------------------------------------------------------- norms and codes
def norm_case(T, N, dtype, post=True, gate="row", residual=True, weight=True, out=True, seed=0, pad=0, offset=0,
              scale=0.875, spread=1.0):
    g = torch.Generator().manual_seed(seed)

    def rows(n, std):
        whole = (torch.randn(n, N + pad + offset, generator=g) * std).to(TYPES[dtype])
        return whole[:, offset:offset + N]
    return dict(x=rows(T, spread), residual=rows(T, 3.0) if residual else None,
                post=torch.randn(N, generator=g) * 0.2 + 1 if post else None,
                gate=None if gate is None else rows(1 if gate == "one" else T, 0.5),
                weight=torch.randn(N, generator=g) * 0.2 + 1 if weight else None, scale=scale, out=out)


def to_gpu(t):
    """On the GPU with the strides it has here."""
    if t is None:
        return None
    base = torch.as_strided(t, (t.untyped_storage().nbytes() // t.element_size(),), (1,), 0)
    return torch.as_strided(base.cuda(), t.shape, t.stride(), t.storage_offset())


def run_norm(c, in_place=False):
    T, N = c["x"].shape
    x, residual = to_gpu(c["x"]), to_gpu(c["residual"])
    out = torch.full((T, N), 77.0, dtype=c["x"].dtype, device="cuda") if c["out"] else None
    if in_place:
        out = residual
    codes = torch.full((T, N), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((T,), 5.0, device="cuda")
    q8.q8ta_norm_quantize(x, residual, to_gpu(c["post"]), to_gpu(c["gate"]), c["scale"], to_gpu(c["weight"]), EPS, out,
                          codes, scales)
    torch.cuda.synchronize()
    return None if out is None else out.cpu(), codes.cpu(), scales.cpu()


def unit(v):
    return v / (v.square().mean(1, keepdim=True) + EPS).sqrt()


def codes_of(h, weight):
    """64-bit codes, scales, and where a code is next to a tie, of stored sums h."""
    p = h.double() if weight is None else h.double() * weight.double()
    z = p if weight is None else unit(h.double()) * weight.double()
    top = p.abs().amax(1, keepdim=True)
    q = p * 127.0 / torch.where(top > 0, top, 1.0)
    near = ((q - q.floor()) - 0.5).abs() < 1e-9
    return q.round(), z.abs().amax(1) / 127.0, near


def check_norm(c, **kw):
    out, codes, scales = run_norm(c, **kw)
    b = c["x"].double()
    if c["post"] is not None:
        b = unit(b) * c["post"].double()
    if c["gate"] is not None:
        b = b * c["gate"].double()
    if c["residual"] is not None:
        b = b + c["residual"].double() * c["scale"]
    t = c["x"].dtype
    if out is not None:
        off = (out.double() - b).abs()
        assert (off <= b.abs() * (half_step(t) + U32) * 1.001 + smallest(t)).all(), off.max()
    h = b.float().to(t) if out is None else out
    want, want_scale, near = codes_of(h, c["weight"])
    differ = codes.double() != want
    if out is None:   # a stored sum next to its own rounding may be the other one here
        assert differ.double().mean() < 1e-3
    else:
        assert not (differ & ~near).any(), (codes[differ & ~near][:5], want[differ & ~near][:5])
        assert ((codes.double() - want).abs() <= 1).all()
    assert ((scales.double() - want_scale).abs() <= want_scale * U32 * 1.001 + 1e-45).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,N", [(1, 1), (1, 8), (3, 7), (2, 64), (5, 513), (1, 4096), (7, 4100), (600, 520), (2, 8192),
                                 (3, 8200), (2, 16384), (2, 16385), (1, 40000), (513, 1000), (520, 4096), (512, 9001)])
def test_norm_quantize(T, N, dtype):
    check_norm(norm_case(T, N, dtype, seed=T + N))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("post,gate,residual,weight,out", [
    (False, None, False, False, False), (False, None, False, True, True), (True, None, False, False, True),
    (False, "one", False, True, True), (False, "row", True, False, True), (True, "one", True, True, True),
    (False, None, True, True, False)])
def test_norm_quantize_parts(post, gate, residual, weight, out, dtype):
    for T, N in ((4, 1000), (600, 264), (2, 17000)):
        check_norm(norm_case(T, N, dtype, post, gate, residual, weight, out, seed=N))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (8, 0), (24, 8), (3, 5)])
def test_norm_quantize_strides_and_alignment(pad, offset, dtype):
    check_norm(norm_case(6, 512, dtype, pad=pad, offset=offset, seed=pad + offset))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", [512, 4097, 20000])
def test_norm_quantize_in_the_residuals_place(N, dtype):
    check_norm(norm_case(4, N, dtype, seed=1), in_place=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("N", [256, 18000])
def test_quantize_per_token_keeps_ties(N, dtype):
    """x * 127 / max is a tie for many 16-bit values: halves of whole numbers below a largest of 127."""
    g = np.random.default_rng(3)
    x = torch.from_numpy(g.integers(-254, 255, (5, N)) / 2.0)
    x[:, 7] = 127.0
    x = x.to(TYPES[dtype])
    codes = torch.empty(5, N, dtype=torch.int8, device="cuda")
    scales = torch.empty(5, device="cuda")
    q8.q8ta_quantize_per_token(x.cuda(), codes, scales)
    assert (codes.cpu().double() == x.double().round()).all() and (scales == 1.0).all()   # (halves to even)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [256, 1000, 20000])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_quantize_per_token_zeros_and_values_that_are_not_finite(N, dtype):
    x = torch.randn(6, N, generator=torch.Generator().manual_seed(1)).to(TYPES[dtype])
    x[1] = 0.0
    x[2, N - 1] = float("nan")
    x[3, 0] = float("-inf")
    x[4] *= smallest(TYPES[dtype]) * 100
    codes = torch.empty(6, N, dtype=torch.int8, device="cuda")
    scales = torch.empty(6, device="cuda")
    q8.q8ta_quantize_per_token(x.cuda(), codes, scales)
    codes, scales = codes.cpu(), scales.cpu()
    assert (codes[1] == 0).all() and scales[1] == 0
    for r in (2, 3):
        assert (codes[r] == 0).all() and torch.isnan(scales[r])
    for r in (0, 4, 5):
        want, scale, near = codes_of(x[r:r + 1], None)
        assert ((codes[r].double() == want[0]) | near[0]).all()
        assert abs(scales[r].double() - scale[0]) <= scale[0] * U32 * 1.001 + 1e-45


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,N", [(512, 4104), (513, 5120), (600, 5001), (515, 6144), (512, 6145), (514, 7168), (516, 8184),
                                 (513, 8192)])
def test_norm_quantize_of_many_long_rows(T, N, dtype):
    check_norm(norm_case(T, N, dtype, seed=N))
    check_norm(norm_case(T, N, dtype, post=False, gate=None, weight=False, out=False, seed=N + 1))


@pytest.mark.gpu
def test_norm_quantize_of_more_tokens_than_one_launch():
    check_norm(norm_case((1 << 21) + 77, 8, "fp16", seed=4))


@pytest.mark.gpu
def test_norm_quantize_no_tokens():
    x = torch.empty(0, 64, device="cuda")
    q8.q8ta_quantize_per_token(x, torch.empty(0, 64, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"))


# ---------------------------------------------------------------- products
def product_case(M, K, N, seed=0, bias=True, mats=1, offset=0):
    g = torch.Generator().manual_seed(seed)

    def codes(*shape):
        n = math.prod(shape)
        flat = torch.randint(-127, 128, (n + offset,), generator=g).to(torch.int8)
        return flat[offset:].view(shape)
    return dict(x=codes(M, K), xs=torch.exp(torch.randn(M, generator=g) * 0.3) * 0.02,
                w=[codes(N, K) for _ in range(mats)],
                ws=[torch.exp(torch.randn(N, generator=g) * 0.2) * 0.02 / math.sqrt(K) for _ in range(mats)],
                bias=[torch.randn(N, generator=g) * 0.5 if bias else None for _ in range(mats)])


def product(c, q):
    """In 64 bits, and what three roundings and the bias's leave it off by at most."""
    acc = c["x"].double() @ c["w"][q].double().t()
    p = acc * c["xs"].double()[:, None] * c["ws"][q].double()
    y = p if c["bias"][q] is None else p + c["bias"][q].double()
    return y, 3.01 * U32 * p.abs() + U32 * y.abs()


def close(got, want, tol, t):
    off = (got.double() - want).abs()
    bad = off > 1.01 * tol + 1.01 * half_step(t) * want.abs() + smallest(t) + 2.0 ** -110
    assert not bad.any(), (bad.nonzero()[:4], got[bad][:4], want[bad][:4])


def gpu(ts):
    return [to_gpu(t) for t in ts]


def check_linear(c, dtype, act="none"):
    t = TYPES[dtype]
    out = torch.full((c["x"].shape[0], c["w"][0].shape[0]), 9.0, dtype=t, device="cuda")
    q8.q8ta_linear_per_token(to_gpu(c["x"]), c["xs"].cuda(), to_gpu(c["w"][0]), c["ws"][0].cuda(),
                             to_gpu(c["bias"][0]), act, out)
    y, tol = product(c, 0)
    close(out.cpu(), y.clamp(min=0) if act == "relu" else y, tol, t)


ACTS = {
    "silu": lambda g: g * torch.sigmoid(g),
    "gelu": lambda g: 0.5 * g * torch.special.erfc(-g / math.sqrt(2.0)),
    "gelu_tanh": lambda g: g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)),
    "relu": lambda g: g.clamp(min=0),
}


def check_gated(c, dtype, act):
    t = TYPES[dtype]
    out = torch.full((c["x"].shape[0], c["w"][0].shape[0]), 9.0, dtype=t, device="cuda")
    w, ws, bias = gpu(c["w"]), gpu(c["ws"]), gpu(c["bias"])
    q8.q8ta_gated_linear(to_gpu(c["x"]), c["xs"].cuda(), w[0], ws[0], bias[0], w[1], ws[1], bias[1], act, out)
    (g, tg), (u, tu) = product(c, 0), product(c, 1)
    a = ACTS[act](g)
    ta = 1.13 * tg + (0.0 if act == "relu" else 2.0 ** -21 * a.abs() + 2.0 ** -23 * g.abs())
    y = a * u
    close(out.cpu(), y, u.abs() * ta + a.abs() * tu + U32 * y.abs(), t)


# rows and channels of the row kernel, of each tile, and around their edges
SIZES = [(1, 64, 16), (1, 4096, 300), (2, 16, 1), (3, 272, 33), (16, 1040, 100), (17, 512, 257), (33, 192, 48), (50, 1024, 130),
         (64, 80, 4097), (24, 256, 4200), (65, 64, 17), (70, 208, 130), (128, 1104, 520), (200, 512, 1030), (300, 2064, 2000),
         (257, 1024, 4100), (1025, 144, 300), (700, 4096, 3500), (513, 48, 5000), (2050, 320, 4160), (1500, 1088, 6001)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_linear_per_token(M, K, N, dtype):
    check_linear(product_case(M, K, N, seed=M + K, bias=M % 2 == 1), dtype, "relu" if N % 3 == 0 else "none")


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_gated_linear(M, K, N, act):
    dtype = ["fp32", "fp16", "bf16"][(M + N) % 3]
    check_gated(product_case(M, K, N, seed=M + K, bias=M % 2 == 0, mats=2), dtype, act)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N,offset", [(1, 1, 5, 0), (7, 15, 9, 0), (40, 100, 65, 0), (3, 64, 33, 1), (90, 1001, 40, 0),
                                          (300, 130, 520, 8), (70, 17, 300, 3), (520, 1030, 600, 0)])
def test_products_odd_sizes_and_alignment(M, K, N, offset):
    check_linear(product_case(M, K, N, seed=M, offset=offset), "fp32")
    check_gated(product_case(M, K, N, seed=M, offset=offset, mats=2), "bf16", "silu")


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("M,K,N", [(1, 15, 17), (1, 16, 40), (2, 17, 33), (5, 31, 20), (16, 63, 50), (1, 65, 800), (3, 1023, 17),
                                   (16, 1025, 40), (30, 1040, 33), (31, 2047, 18), (60, 2049, 20), (64, 95, 300), (4, 4095, 30),
                                   (2, 4097, 65), (9, 7001, 12400), (17, 5003, 16)])
def test_products_of_rows_as_they_lie(M, K, N, offset):
    check_linear(product_case(M, K, N, seed=K, offset=offset), "fp32")
    check_gated(product_case(M, K, N, seed=K + 1, offset=offset, mats=2), "fp16", "silu")


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(3, 40), (100, 200), (600, 4500)])
def test_products_outputs_at_odd_addresses(M, N):
    c = product_case(M, 128, N, seed=5)
    whole = torch.full((M * N + 9,), 3.0, dtype=torch.bfloat16, device="cuda")
    out = whole[1:1 + M * N].view(M, N)
    q8.q8ta_linear_per_token(c["x"].cuda(), c["xs"].cuda(), c["w"][0].cuda(), c["ws"][0].cuda(), c["bias"][0].cuda(),
                             "none", out)
    y, tol = product(c, 0)
    close(out.cpu(), y, tol, torch.bfloat16)
    assert whole[0] == 3 and (whole[1 + M * N:] == 3).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [2, 90])
def test_products_of_rows_past_a_tiles_offsets(M):
    K, N = (1 << 23) + 16, 3
    g = torch.Generator(device="cuda").manual_seed(M)
    x, w = (torch.randint(-1, 2, (n, K), generator=g, dtype=torch.int8, device="cuda") for n in (M, N))
    one = torch.ones(max(M, N), device="cuda")
    out = torch.empty(M, N, device="cuda")
    q8.q8ta_linear_per_token(x, one[:M], w, one[:N], None, "none", out)
    want = torch.stack([(x[:, a:a + 4096].int().float() @ w[:, a:a + 4096].float().t()) for a in range(0, K, 4096)]).sum(0)
    assert want.abs().max() < 2 ** 24 and torch.equal(out, want)   # (whole numbers: exact in fp32)


@pytest.mark.gpu
def test_products_largest_sums():
    """Codes of -128 and 127 throughout: the largest sums that K allows."""
    M, K, N = 70, 4096, 96
    c = product_case(M, K, N, seed=1)
    c["x"] = torch.full((M, K), -128, dtype=torch.int8)
    c["w"][0] = torch.full((N, K), -128, dtype=torch.int8)
    c["x"][1::2] = 127
    check_linear(c, "fp32")
    check_linear(dict(c, x=c["x"][:5], xs=c["xs"][:5]), "fp32")


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("M", [2, 80])
def test_gates_far_from_zero(act, M):
    """Gates up to +-200, where a logistic is 0 or 1 and a complementary error function is 0 or 2."""
    c = product_case(M, 64, 96, seed=4, bias=False, mats=2)
    y, _ = product(c, 0)
    c["ws"][0] = c["ws"][0] * (200.0 / y.abs().max())
    check_gated(c, "fp32", act)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [4, 100])
def test_a_tokens_scale_that_is_not_finite_spoils_its_own_row(M):
    c = product_case(M, 256, 80, seed=2)
    c["xs"][1] = float("nan")
    out = torch.empty(M, 80, device="cuda")
    q8.q8ta_linear_per_token(c["x"].cuda(), c["xs"].cuda(), c["w"][0].cuda(), c["ws"][0].cuda(), c["bias"][0].cuda(),
                             "none", out)
    out = out.cpu()
    assert torch.isnan(out[1]).all() and not torch.isnan(out[[0] + list(range(2, M))]).any()


@pytest.mark.gpu
def test_a_block_together_on_a_side_stream():
    """norm -> gated block -> codes -> product, on a stream of its own beside the default one, three times."""
    g = torch.Generator().manual_seed(0)
    T, H, F = 90, 512, 1100
    x, res = ((torch.randn(T, H, generator=g)).bfloat16().cuda() for _ in range(2))
    weight = torch.ones(H, device="cuda")
    c, d = product_case(T, H, F, seed=8, mats=2, bias=False), product_case(T, F, H, seed=9, bias=False)
    w, ws, wd, wsd = gpu(c["w"]), gpu(c["ws"]), d["w"][0].cuda(), d["ws"][0].cuda()

    def block():
        codes, s = torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        h, mid = torch.empty_like(x), torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
        q8.q8ta_norm_quantize(x, res, None, None, 1.0, weight, EPS, h, codes, s)
        q8.q8ta_gated_linear(codes, s, w[0], ws[0], None, w[1], ws[1], None, "silu", mid)
        codes2, s2 = torch.empty(T, F, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        q8.q8ta_quantize_per_token(mid, codes2, s2)
        return q8.q8ta_linear_per_token(codes2, s2, wd, wsd, None, "none",
                                        torch.empty(T, H, dtype=torch.bfloat16, device="cuda"))
    want = block()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [block() for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)
    assert want.float().std() > 0


@pytest.mark.gpu
def test_captured_block_with_copies():
    """A captured product of odd K (its copies take memory in the graph), replayed beside eager calls."""
    c = product_case(70, 333, 200, seed=3)
    x, xs, w, ws, b = c["x"].cuda(), c["xs"].cuda(), c["w"][0].cuda(), c["ws"][0].cuda(), c["bias"][0].cuda()
    out = torch.empty(70, 200, device="cuda")
    q8.q8ta_linear_per_token(x, xs, w, ws, b, "none", out)
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q8.q8ta_linear_per_token(x, xs, w, ws, b, "none", out)
    for _ in range(4):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
        other = torch.empty(70, 200, device="cuda")
        q8.q8ta_linear_per_token(x, xs, w, ws, b, "none", other)
        torch.cuda.synchronize()
        assert torch.equal(other, want)


# ---------------------------------------------------------------- refusals
FAKE = 4096


def refused(rc, status, words):
    assert rc == status and words in q8.q8ta_last_error(), (rc, q8.q8ta_last_error())


def test_norm_quantize_refuses():
    base = dict(x=FAKE, xs=64, r=FAKE, rs=64, dt=2, T=4, N=64, pw=FAKE, g=FAKE, gs=0, scale=1.0, w=FAKE, eps=EPS, o=FAKE,
                c=FAKE, s=FAKE, st=None)

    def call(**kw):
        return q8.lib().q8ta_norm_quantize(*{**base, **kw}.values())
    for kw, status, words in [
            (dict(dt=3), q8.Q8TA_ERR_UNSUPPORTED, "dtype"), (dict(T=-1), q8.Q8TA_ERR_SHAPE, "tokens"),
            (dict(T=1 << 31), q8.Q8TA_ERR_SHAPE, "tokens"), (dict(N=0), q8.Q8TA_ERR_SHAPE, "N must"),
            (dict(N=(1 << 30) + 1), q8.Q8TA_ERR_SHAPE, "N must"), (dict(T=1 << 20, N=(1 << 20) + 1), q8.Q8TA_ERR_SHAPE, "2^40"),
            (dict(xs=-1), q8.Q8TA_ERR_SHAPE, "stride"), (dict(rs=1 << 41), q8.Q8TA_ERR_SHAPE, "stride"),
            (dict(gs=-8), q8.Q8TA_ERR_SHAPE, "stride"), (dict(scale=math.inf), q8.Q8TA_ERR_QPARAM, "residual_scale"),
            (dict(eps=0.0), q8.Q8TA_ERR_QPARAM, "eps"), (dict(eps=math.nan), q8.Q8TA_ERR_QPARAM, "eps"),
            (dict(x=None), q8.Q8TA_ERR_NULL, "NULL"), (dict(c=None), q8.Q8TA_ERR_NULL, "NULL"),
            (dict(s=None), q8.Q8TA_ERR_NULL, "NULL")]:
        refused(call(**kw), status, words)
    assert call(T=0) == q8.Q8TA_OK
    assert call(T=0, eps=-1.0, pw=None, w=None) == q8.Q8TA_OK     # no norm, no eps
    refused(q8.lib().q8ta_quantize_per_token(FAKE, 64, 1, 4, 64, None, FAKE, None), q8.Q8TA_ERR_NULL, "q8ta_quantize_per_token")


def test_products_refuse():
    base = dict(x=FAKE, M=4, K=64, xs=FAKE, w=FAKE, N=32, ws=FAKE, b=None, act=b"none", o=FAKE, dt=0, st=None)

    def linear(**kw):
        return q8.lib().q8ta_linear_per_token(*{**base, **kw}.values())
    gbase = dict(x=FAKE, M=4, K=64, xs=FAKE, gw=FAKE, gs=FAKE, gb=None, uw=FAKE, us=FAKE, ub=None, N=32, act=b"silu", o=FAKE,
                 dt=0, st=None)

    def gated(**kw):
        return q8.lib().q8ta_gated_linear(*{**gbase, **kw}.values())
    for kw, status, words in [
            (dict(M=0), q8.Q8TA_ERR_SHAPE, ">= 1"), (dict(K=0), q8.Q8TA_ERR_SHAPE, ">= 1"), (dict(N=0), q8.Q8TA_ERR_SHAPE, ">= 1"),
            (dict(M=(1 << 21) + 1), q8.Q8TA_ERR_SHAPE, "too large"), (dict(N=(1 << 30) + 1), q8.Q8TA_ERR_SHAPE, "too large"),
            (dict(K=1 << 30, N=1 << 11), q8.Q8TA_ERR_SHAPE, "too large"), (dict(dt=7), q8.Q8TA_ERR_UNSUPPORTED, "dtype"),
            (dict(act=b"tanh"), q8.Q8TA_ERR_UNSUPPORTED, "activation"), (dict(act=None), q8.Q8TA_ERR_UNSUPPORTED, "activation"),
            (dict(x=None), q8.Q8TA_ERR_NULL, "NULL"), (dict(xs=None), q8.Q8TA_ERR_NULL, "NULL"), (dict(o=None), q8.Q8TA_ERR_NULL, "NULL")]:
        refused(linear(**kw), status, words)
        refused(gated(**kw), status, words)
    refused(linear(act=b"silu"), q8.Q8TA_ERR_UNSUPPORTED, "activation")
    refused(gated(act=b"none"), q8.Q8TA_ERR_UNSUPPORTED, "activation")
    for name in ("w", "ws"):
        refused(linear(**{name: None}), q8.Q8TA_ERR_NULL, "NULL")
    for name in ("gw", "gs", "uw", "us"):
        refused(gated(**{name: None}), q8.Q8TA_ERR_NULL, "NULL")


def test_bindings_refuse():
    x, codes, s = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="device tensor"):
        q8.q8ta_quantize_per_token(x, codes, s)
    with pytest.raises(ValueError):
        q8.q8ta_linear_per_token(codes, s, torch.zeros(32, 63, dtype=torch.int8), torch.zeros(32), None, "none", torch.zeros(4, 32))
    with pytest.raises(ValueError, match="x_scales"):
        q8.q8ta_linear_per_token(codes, s[:3], torch.zeros(32, 64, dtype=torch.int8), torch.zeros(32), None, "none",
                                 torch.zeros(4, 32))
    with pytest.raises(ValueError):
        q8.q8ta_gated_linear(codes, s, torch.zeros(32, 64, dtype=torch.int8), torch.zeros(32), None,
                             torch.zeros(31, 64, dtype=torch.int8), torch.zeros(32), None, "silu", torch.zeros(4, 32))


@pytest.mark.gpu
def test_bindings_refuse_shapes_on_the_gpu():
    x, codes, s = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    w = torch.ones(64, device="cuda")
    for bad in (dict(residual=x[:3]), dict(residual=x.half()), dict(gate=x[:2]), dict(gate=x[:, :63]), dict(weight=w[:63]),
                dict(post=w[:1]), dict(codes=codes[:3]), dict(scales=s[:3])):
        a = dict(residual=None, post=None, gate=None, weight=w, codes=codes, scales=s)
        a.update(bad)
        with pytest.raises(ValueError):
            q8.q8ta_norm_quantize(x, a["residual"], a["post"], a["gate"], 1.0, a["weight"], EPS, None, a["codes"], a["scales"])
    with pytest.raises(TypeError):
        q8.q8ta_quantize_per_token(x.double(), codes, s)
    with pytest.raises(TypeError):
        q8.q8ta_linear_per_token(codes, s, torch.zeros(32, 64, dtype=torch.int8, device="cuda"), torch.zeros(32, device="cuda"), None,
                                 "none", torch.zeros(4, 32, dtype=torch.int32, device="cuda"))
