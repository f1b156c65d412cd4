"""q8ta_tree_attention: the precision of its probabilities, many requests, queries at odd addresses.

With fp16 outputs a probability is held in two fp16 parts (2^-22 of it) and everything else in 32
bits, so that an output is off by its own rounding and little else: the tests below leave half a step
of the type, and of sums over n keys (n / 8 + 64) * 2^-24 of sum |p v|.
"""
import numpy as np
import pytest

import int8_quantized_amd as q8
from test_tree_attention import check, definition, make, run

torch = pytest.importorskip("torch")


def uniform(c):
    """The outputs of queries of zero: means over the seen values, and of their magnitudes."""
    B, T, hq, d = c["q"].shape
    _, _, hk, page, _ = c["cache"].shape
    want, mag = np.zeros((B, T, hq, d)), np.zeros((B, T, hq, d))
    for b in range(B):
        n = int(c["lens"][b])
        at, off = c["table"][b][np.arange(n + T) // page], np.arange(n + T) % page
        for h in range(hq):
            kh = h // (hq // hk)
            v = c["cache"][at, 1, kh, off].astype(np.float64) * c["scales"][at, 1, kh, off].astype(np.float64)[:, None]
            for t in range(T):
                m = int(np.uint64(c["mask"][b, t]))
                seen = [j < n or (m >> (j - n)) & 1 == 1 for j in range(n + T)]
                want[b, t, h], mag[b, t, h] = v[seen].mean(0), np.abs(v[seen]).mean(0)
    return want, mag


@pytest.mark.gpu
@pytest.mark.parametrize("size", [(3, 1, 8, 2, 128, 16, [0, 3, 40]), (2, 24, 8, 2, 128, 32, [0, 300]),
                                  (2, 5, 4, 1, 64, 16, [1, 2500]), (1, 33, 4, 2, 80, 16, [700]),
                                  (2, 3, 4, 2, 256, 16, [0, 90])])
def test_tree_attention_fp16_output_is_off_by_its_rounding_alone(size):
    c = make(*size, dtype="fp16", seed=21)
    c["q"][:] = 0
    want, mag = uniform(c)
    got = run(c)[0].double().cpu().numpy()
    n = max(size[6]) + size[1]
    tol = np.abs(want) * 2.0 ** -11 + mag * (n / 8 + 64) * 2.0 ** -24 + 2.0 ** -25
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / tol)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [(2, 1, 8, 2, 128, 16, [900, 77]), (1, 24, 8, 2, 128, 32, [500]),
                                  (1, 33, 4, 2, 64, 16, [300]), (1, 3, 4, 2, 256, 16, [200])])
def test_tree_attention_fp16_error_is_that_of_rounding_the_exact_outputs(size):
    """In the mean over all outputs: probabilities of 11 bits made it 1.4 times as large."""
    c = make(*size, dtype="fp16", seed=22)
    want = definition(c)[0]
    got = run(c)[0].double().cpu().numpy()
    rounded = want.astype(np.float16).astype(np.float64)
    assert np.linalg.norm(got - want) <= 1.05 * np.linalg.norm(rounded - want)


def ragged(B, most, seed):
    """Context lengths of B requests, one in five of them none."""
    g = np.random.default_rng(seed)
    n = g.integers(1, most, B)
    n[g.permutation(B)[:B // 5]] = 0
    return n.tolist()


@pytest.mark.gpu
@pytest.mark.parametrize("B", [63, 64, 65, 128, 130, 200])
@pytest.mark.parametrize("T,hk,most,spare", [(1, 2, 300, 1), (3, 1, 150, 90), (20, 1, 120, 1), (1, 1, 90, 1)])
def test_tree_attention_more_requests_than_a_round(B, T, hk, most, spare):
    """The requests' lengths are summed 64 at a time: units that are cut across those borders, and the
    forms without cuts (the first and the last)."""
    c = make(B, T, 2 * hk, hk, 64, 16, ragged(B, most, B + T), seed=B, spare=spare,
             counts=[(T * 7 + b) % (T + 1) for b in range(B)] if T > 1 else None)
    check(c)


@pytest.mark.gpu
def test_tree_attention_requests_of_very_different_length():
    """One long request among 150 short and empty ones: most of the runs are its own."""
    n = ragged(150, 20, 3)
    n[97] = 9000
    check(make(150, 1, 4, 1, 64, 64, n, seed=6))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,d,hq,odd", [(1, 64, 4, 1), (5, 128, 8, 3), (20, 80, 4, 7), (2, 256, 4, 5), (1, 64, 4, 8)])
def test_tree_attention_queries_at_odd_addresses_and_strides(T, d, hq, odd, dtype):
    """Rows that do not start on 16 bytes, heads and tokens an odd number of elements apart."""
    c = make(2, T, hq, 2, d, 16, [70, 9], seed=T + d, dtype=dtype)
    out, lse = check(c)
    q = c["q"].cuda()
    B, (heads, tokens) = 2, (d + odd, (hq + 1) * (d + odd) + odd)
    flat = torch.full((odd + B * T * tokens + 1000,), 3.0, dtype=q.dtype, device="cuda")
    view = flat[odd:].as_strided((B, T, hq, d), (T * tokens, tokens, heads, 1))
    view.copy_(q)
    assert torch.equal(view, q)
    dev = {k: None if v is None else torch.from_numpy(v).cuda() for k, v in c.items() if k not in ("q", "scale")}
    again, lse2 = torch.empty_like(out), torch.empty_like(lse)
    q8.q8ta_tree_attention(view, dev["cache"], dev["scales"], dev["table"], dev["lens"], dev["counts"],
                           dev["mask"], c["scale"], again, lse2)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20])
def test_tree_attention_powers_of_two_move_from_keys_to_queries(T):
    """Queries of any bf16 size: what a power of two takes from the keys' scales and gives to the queries
    leaves every score, and so every bit, as it is."""
    c = make(2, T, 4, 2, 64, 16, [300, 9], seed=31)
    want = run(c)
    for e in (-20, 60, 110, 116, 118):
        moved = dict(c, q=(c["q"].float() * 2.0 ** e).to(c["q"].dtype), scales=c["scales"].copy())
        moved["scales"][:, 0] *= np.float32(2.0 ** -e)
        assert torch.isfinite(moved["q"].float()).all() and (moved["scales"][:, 0] > 2.0 ** -126).all()
        got = run(moved)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), e


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("e", [-80, -30, 60, 84])
def test_tree_attention_value_scales_over_the_stated_range(T, e):
    """Powers of two on all value scales come out on the outputs, exactly."""
    c = make(2, T, 4, 2, 64, 16, [900, 9], seed=32)
    want, lse = run(c)
    c["scales"][:, 1] *= np.float32(2.0 ** e)
    got, lse2 = run(c)
    assert torch.equal(got.double(), want.double() * 2.0 ** e) and torch.equal(lse, lse2)
