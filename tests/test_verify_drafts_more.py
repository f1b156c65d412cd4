"""q8ta_verify_drafts at temperatures and logits at the ends of fp32, how far off the sums are that shares are divided
by, and the longest vocabulary with a drafter's logits.

Tolerance of the sums.  A weight 2^-y of its chunk's largest that is formed in 32 bits has y off by 2^-23 of itself
(a difference and a multiply-add) and its exponential by 2^-23: 2^-23 (1 + 0.7 y) in all; four are added at a time, with
three roundings of 2^-24.  A chunk's sum takes these by the shares of its 4096 weights, of which the mean of y
is at most log2 4096 = 12: 2^-23 (1 + 8.4 + 1.5) < 2^-19 of the sum.
"""
import numpy as np
import pytest

import int8_quantized_amd as q8
from test_verify_drafts import check, definition, make, run

torch = pytest.importorskip("torch")


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("size,temperature", [(1e30, 4e30), (2e37, 3e37), (1e38, 3e38), (1e30, 1e31), (1e-33, 1e-33), (1e-36, 3e-36),
                                              (1e-30, 2e-31), (1.0, 3e38), (1e36, np.inf), (1.0, np.inf)])
def test_temperatures_and_logits_at_the_ends_of_fp32(size, temperature, draft):
    for seed in range(3):
        c = make(4, 6, 700, "fp32", draft, seed=seed, spread=1.0)
        for x in (c["logits"], c["draft"]):
            if x is not None:
                x.copy_((x.double() * size).clamp(-3.4e38, 3.4e38).float())
        c["temperature"][:] = temperature
        check(c)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("temperature", [np.inf, 3e38, 2.0])
def test_masks_of_the_types_lowest_value(temperature, dtype):
    """At an infinite temperature such a token's weight is any other's."""
    for seed in range(8):
        for draft in (True, False):
            c = make(12, 6, 8, dtype, draft, seed=seed)
            for x in (c["logits"], c["draft"]):
                if x is not None:
                    x[:, :, 1::2] = torch.finfo(x.dtype).min
            if draft:                                # (a drawn token's share is above 0)
                c["ids"] &= ~1
            c["temperature"][:] = temperature
            check(c)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V,low,temperature", [(4096, -9.5, 1.0), (40960, -4.5, 0.8), (40960, -5.75, 1.0), (131072, -2.25, 0.8),
                                               (131072, -7.0, 0.9), (8192, -1.5, 1.0)])
def test_sums_of_few_distinct_logits(V, low, temperature, dtype):
    """Equal logits' errors do not cancel: one child, whose random number goes through its share in steps of 2^-22."""
    j = np.arange(-40, 41)
    B = len(j)
    c = make(B, 2, V, dtype, False, seed=1)
    c["logits"][:] = low
    c["logits"][:, :, ::4096] = 0.0
    c["ids"][:, 1] = 0
    c["temperature"][:] = temperature
    tops = -(-V // 4096)
    low = float(c["logits"][0, 0, 1])
    share = 1.0 / (tops + (V - tops) * np.exp(low / float(np.float32(temperature))))
    c["u"][:, 1] = share * (1 + j * 2.0 ** -22)
    off = c["u"][:, 1].astype(np.float64) / share - 1
    _, accepted, _ = run(c)
    assert (accepted[off < -2.0 ** -19] == 2).all() and (accepted[off > 2.0 ** -19] == 1).all(), (off, accepted)
    assert (np.diff(accepted[np.argsort(off)]) <= 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("seed", [3, 5])
def test_longest_vocabulary_with_a_drafter(seed):
    """A residual over 4096 chunks, and a kept token with the one after it."""
    c = make(1, 2, 1 << 24, "bf16", True, seed=seed, temperature=0.3)
    want = definition(c)
    assert want[3][0] > 1e-2 and want[1][0] == 1     # far from every border, nothing kept
    assert all((a == b).all() for a, b in zip(run(c), want))
    c["u"][0, 1] = 0.0
    want = definition(c)
    assert want[3][0] > 1e-9 and want[1][0] == 2
    assert all((a == b).all() for a, b in zip(run(c), want))


@pytest.mark.gpu
def test_more_requests_than_a_launchs_workspace_holds():
    """One row of logits, read by every request with numbers of its own."""
    B, V = 65535, 65536
    g = torch.Generator(device="cuda").manual_seed(2)
    x = (torch.randn(1, 1, V, generator=g, device="cuda") * 2).bfloat16().expand(B, 1, V)
    ids, heat = torch.zeros(B, 1, dtype=torch.int32, device="cuda"), torch.rand(B, generator=g, device="cuda") + 0.5
    u = torch.rand(B, 1, generator=g, device="cuda")

    def run_rows(a, b):
        outs = [torch.full(s, -7, dtype=torch.int32, device="cuda") for s in ((b - a, 1), (b - a,), (b - a,))]
        q8.q8ta_verify_drafts(x[a:b], None, ids[a:b], None, None, heat[a:b], None, u[a:b], *outs)
        return outs
    whole, parts = run_rows(0, B), [run_rows(a, min(a + 9999, B)) for a in range(0, B, 9999)]
    for i, o in enumerate(whole):
        assert torch.equal(o, torch.cat([p[i] for p in parts]))
    assert (whole[1] == 1).all() and ((whole[2] >= 0) & (whole[2] < V)).all() and whole[2].unique().numel() > 1000
