"""q8ta_rope_append against its definition in 64 bits (numpy): turned queries, codes and scales of
the appended rows, the rows it must leave alone, and the calls it refuses.

Tolerances: the kernel turns in 64 bits, so a query differs from the definition by its one
rounding to the type (half a step, doubled where fp32 lies between) and a scale by its rounding to
fp32; codes are whole numbers and equal, but for a quotient within 1e-9 of a tie.
"""
import numpy as np
import pytest

import int8_quantized_amd as q8

torch = pytest.importorskip("torch")

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def definition(q, k, v, positions, inv_freq, factor, interleaved):
    rot = 2 * len(inv_freq)
    ang = positions.astype(np.float64)[:, None] * inv_freq
    cos, sin = (np.cos(ang) * factor)[:, None], (np.sin(ang) * factor)[:, None]

    def turn(x):
        y = x.astype(np.float64).copy()
        i = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
        j = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
        a, b = y[..., i].copy(), y[..., j].copy()
        y[..., i], y[..., j] = a * cos - b * sin, b * cos + a * sin
        return y

    def quant(x):
        top = np.abs(x).max(-1, keepdims=True)
        return x * 127.0 / np.where(top > 0, top, 1.0), top[..., 0] / 127.0

    return turn(q), quant(turn(k)), quant(v.astype(np.float64))


def check_codes(got, want, where):
    tie = np.abs(want - np.floor(want) - 0.5) < 1e-9
    bad = (np.abs(got - np.rint(want)) > tie)
    assert not bad.any(), (where, got[bad][:4], want[bad][:4])


def case(T, hq, hk, d, rot, dtype, interleaved, page, fused=True, offset=0, factor=1.0, seed=0,
         start=0, pad=0):
    """Inputs on the device, as slices of one fused projection or as dense tensors."""
    g = np.random.default_rng(seed)
    width = (hq + 2 * hk) * d + offset
    x = torch.from_numpy(g.standard_normal((T, width)).astype(np.float32)).to(TYPES[dtype]).cuda()
    x = x[:, offset:]
    q = x[:, :hq * d].unflatten(1, (hq, d))
    k = x[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    v = x[:, (hq + hk) * d:].unflatten(1, (hk, d))
    if not fused:
        q, k, v = (t.contiguous() for t in (q, k, v))
    pages = (T + page - 1) // page + 2
    slots = g.permutation(pages * page)[:T].astype(np.int64)
    if pad:
        slots[g.permutation(T)[:pad]] = -1
    positions = (start + g.integers(0, 5000, T)).astype(np.int32)
    inv_freq = 10000.0 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))
    return q, k, v, positions, slots, inv_freq, factor, interleaved, pages


def run(q, k, v, positions, slots, inv_freq, factor, interleaved, pages, page):
    T, hq, d = q.shape
    hk = k.shape[1]
    q_out = torch.full((T, hq, d), 7.0, dtype=q.dtype, device="cuda")
    cache = torch.full((pages, 2, hk, page, d), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((pages, 2, hk, page), -3.0, dtype=torch.float32, device="cuda")
    q8.q8ta_rope_append(q, k, v, torch.from_numpy(positions).cuda(), torch.from_numpy(slots).cuda(),
                        torch.from_numpy(inv_freq).cuda(), factor, interleaved, q_out, cache, scales)
    torch.cuda.synchronize()
    return q_out, cache, scales


def check(c, page):
    q, k, v, positions, slots, inv_freq, factor, interleaved, pages = c
    q_out, cache, scales = run(*c, page)
    wq, (kc, ks), (vc, vs) = definition(*(t.double().cpu().numpy() for t in (q, k, v)), positions,
                                        inv_freq, factor, interleaved)
    got = q_out.double().cpu().numpy()
    eps = torch.finfo(q.dtype).eps / 2
    tiny = torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps
    # one rounding to the type, one to fp32 before it
    assert (np.abs(got - wq) <= np.abs(wq) * (eps + 2.0 ** -24) * 1.001 + tiny).all()
    codes, sc = cache.cpu().numpy(), scales.double().cpu().numpy()
    touched = np.zeros(sc.shape, bool)
    for t, s in enumerate(slots):
        if s < 0 or s >= pages * page:
            continue
        p, r = divmod(int(s), page)
        touched[p, :, :, r] = True
        check_codes(codes[p, 0, :, r].astype(float), kc[t], ("k", t))
        check_codes(codes[p, 1, :, r].astype(float), vc[t], ("v", t))
        for part, want in ((0, ks[t]), (1, vs[t])):
            assert (np.abs(sc[p, part, :, r] - want) <= want * 2.0 ** -24 * 1.001 + 1e-45).all()
    assert (codes[~touched] == 99).all() and (sc[~touched] == -3.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hk,d,rot,page", [
    (1, 32, 8, 128, 128, 16), (3, 7, 1, 64, 32, 16), (5, 4, 2, 80, 80, 32), (2, 8, 8, 80, 40, 64),
    (4, 8, 2, 96, 48, 128), (33, 16, 2, 256, 256, 16), (520, 4, 4, 64, 64, 64), (2, 2, 1, 512, 512, 1),
    (2, 3, 1, 128, 0, 16)])
def test_rope_append(T, hq, hk, d, rot, page, interleaved, dtype):
    check(case(T, hq, hk, d, rot, dtype, interleaved, page, seed=T + d + rot), page)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,offset,fused", [
    (1, 0, 0, True), (2, 2, 0, True), (7, 6, 0, False), (100, 100, 0, True), (65, 64, 0, True),
    (128, 64, 1, True), (64, 64, 3, True), (1000, 10, 0, False), (128, 126, 0, True)])
def test_rope_append_odd_sizes_and_alignment(d, rot, offset, fused, interleaved, dtype):
    check(case(5, 3, 2, d, rot, dtype, interleaved, 3, fused=fused, offset=offset, seed=d + rot), 3)


@pytest.mark.gpu
def test_rope_append_far_positions_and_factor():
    check(case(40, 4, 2, 128, 64, "fp32", True, 64, factor=1.2079441541679836, start=2000000000,
               seed=3), 64)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_rope_append_padding_tokens_and_bad_slots(dtype):
    c = list(case(20, 4, 2, 64, 64, dtype, False, 16, seed=9, pad=6))
    c[4][3], c[4][4] = c[8] * 16, 1 << 40      # past the cache: not stored
    check(tuple(c), 16)


@pytest.mark.gpu
def test_rope_append_zero_rows_ties_and_in_place():
    c = list(case(4, 2, 2, 64, 0, "fp32", False, 16, fused=False, seed=4))
    c[1][1], c[2][2] = 0.0, 0.0
    tie = torch.zeros(64, device="cuda")
    tie[0], tie[1:5] = 254.0, torch.tensor([1.0, 3.0, -1.0, -5.0], device="cuda")   # 0.5, 1.5, ..
    c[1][0, 0], c[2][3, 1] = tie, tie
    check(tuple(c), 16)
    q, k, v, positions, slots, _, _, _, pages = c
    f = 10000.0 ** (-2.0 * np.arange(32) / 64)
    want, _, _ = run(q, k, v, positions, slots, f, 1.0, False, pages, 16)
    cache = torch.zeros((pages, 2, 2, 16, 64), dtype=torch.int8, device="cuda")
    scales = torch.zeros((pages, 2, 2, 16), device="cuda")
    q8.q8ta_rope_append(q, k, v, torch.from_numpy(positions).cuda(), torch.from_numpy(slots).cuda(),
                        torch.from_numpy(f).cuda(), 1.0, False, q, cache, scales)
    assert torch.equal(q, want)


@pytest.mark.gpu
def test_rope_append_no_tokens():
    c = case(1, 2, 1, 64, 64, "bf16", False, 16)
    q, k, v, positions, slots, f, factor, il, pages = c
    q_out, cache, scales = run(q[:0], k[:0], v[:0], positions[:0], slots[:0], f, factor, il, pages, 16)
    assert (cache == 99).all() and (scales == -3.0).all()


# ---------------------------------------------------------------- refusals (no GPU)
FAKE = 4096   # never dereferenced: every call below fails validation first
GOOD = dict(q=FAKE, qt=1024, qh=64, k=FAKE, kt=1024, kh=64, v=FAKE, vt=1024, vh=64, dtype=2,
            tokens=3, heads=8, kv_heads=2, dim=64, positions=FAKE, slots=FAKE, inv_freq=FAKE, rot=64,
            factor=1.0, interleaved=0, q_out=FAKE, cache=FAKE, scales=FAKE, pages=4, page=16, s=None)


def refuse(status, **kw):
    a = dict(GOOD)
    a.update(kw)
    assert q8.lib().q8ta_rope_append(*a.values()) == status
    assert "q8ta_rope_append" in q8.q8ta_last_error()


def test_rope_append_refusals():
    for name in ("q", "k", "v", "positions", "slots", "inv_freq", "q_out", "cache", "scales"):
        refuse(q8.Q8TA_ERR_NULL, **{name: None})
    for bad in (dict(tokens=-1), dict(tokens=1 << 31), dict(heads=0), dict(kv_heads=0),
                dict(heads=65535), dict(dim=0), dict(dim=65537), dict(rot=3), dict(rot=66),
                dict(rot=-2), dict(pages=0), dict(page=0), dict(pages=1 << 40), dict(qt=-1),
                dict(vh=-1), dict(kt=1 << 41)):
        refuse(q8.Q8TA_ERR_SHAPE, **bad)
    refuse(q8.Q8TA_ERR_UNSUPPORTED, dtype=3)
    refuse(q8.Q8TA_ERR_UNSUPPORTED, interleaved=2)
    refuse(q8.Q8TA_ERR_QPARAM, factor=float("nan"))
    refuse(q8.Q8TA_ERR_QPARAM, factor=float("inf"))


def test_rope_append_no_tokens_launches_nothing():
    a = dict(GOOD, tokens=0, q=None, k=None, v=None)
    assert q8.lib().q8ta_rope_append(*a.values()) == q8.Q8TA_OK


def test_rope_append_binding_rejects_host_tensors():
    z = torch.zeros
    with pytest.raises(ValueError):
        q8.q8ta_rope_append(z(1, 2, 64), z(1, 1, 64), z(1, 1, 64), z(1, dtype=torch.int32),
                            z(1, dtype=torch.int64), z(32, dtype=torch.float64), 1.0, False,
                            z(1, 2, 64), z((1, 2, 1, 16, 64), dtype=torch.int8), z(1, 2, 1, 16))
