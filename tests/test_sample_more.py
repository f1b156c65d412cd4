"""q8ta_sample: numbers outside [0, 1), vocabularies beyond the groups, more rows than a launch takes."""
import numpy as np
import pytest

from test_sample import SETTINGS, check, rows, run

torch = pytest.importorskip("torch")


@pytest.mark.gpu
@pytest.mark.parametrize("V", [3, 64, 5000, 32000])
@pytest.mark.parametrize("wrong,stands_for", [(-0.25, 0.0), (-np.inf, 0.0), (1.0, 2.0), (np.inf, 2.0), (np.nan, 2.0)])
def test_sample_numbers_outside_their_range(V, wrong, stands_for):
    """Below 0 the first kept token, from 1 on (and for a NaN) the last, with its log-probability."""
    B = len(SETTINGS)
    t, k, p, mp = zip(*SETTINGS)
    x, _ = rows(B, V, V + 1)
    _, tokens, lp = run(x, t, k, p, mp, np.full(B, wrong))
    _, want, want_lp = run(x, t, k, p, mp, np.full(B, stands_for))
    assert (tokens == want).all() and (tokens >= 0).all() and (lp == want_lp).all()


@pytest.mark.gpu
@pytest.mark.parametrize("V,dtype", [(1 << 20, "fp32"), ((1 << 20) + 5, "fp32"), ((1 << 21) + 5, "bf16"),
                                     ((1 << 21) - 3, "fp16")])
def test_sample_long_vocabularies(V, dtype):
    """On both sides of the longest vocabulary that is read in groups (2^20 fp32, 2^21 16-bit tokens)."""
    B = len(SETTINGS)
    t, k, p, mp = zip(*SETTINGS)
    x, g = rows(B, V, 31)
    x[2, ::3] = -np.inf
    x[9, 5:] = np.nan
    check(x, t, k, p, mp, g.random(B), dtype=dtype)


@pytest.mark.gpu
def test_sample_long_vocabulary_settings_that_are_no_numbers():
    V, nan = (1 << 20) + 5, np.nan
    x, g = rows(5, V, 32)
    x[4] = -np.inf
    _, tokens, lp = run(x, [1.0, 1.0, nan, 1.0, 1.0], [0, 5000, 0, 20, 0], [nan, nan, 0.9, 0.9, 0.9],
                        [0.0, 0.0, 0.0, nan, 0.0], g.random(5))
    assert (tokens[:4] == x[:4].astype(np.float32).argmax(1)).all() and (lp[:4] == 0).all()
    assert tokens[4] == -1 and np.isneginf(lp[4])


@pytest.mark.gpu
@pytest.mark.parametrize("B,V,dtype,optional", [(1030, 700, "fp32", True), (2100, 333, "bf16", True),
                                                (1025, 2000, "fp16", False)])
def test_sample_more_rows_than_a_launch(B, V, dtype, optional):
    """A second and a third group of launches, the last one smaller, on the same workspace."""
    x, g = rows(B, V, B)
    n = len(SETTINGS)
    t, k, p, mp = zip(*[SETTINGS[(i * 5 + i // n) % n] for i in range(B)])
    u = g.random(B)
    if optional:
        check(x, t, k, p, mp, u, dtype=dtype, stride=3)
    else:
        check(x, t, None, p, None, u, dtype=dtype)
        check(x, t, k, None, mp, u, dtype=dtype, logprobs=False)


@pytest.mark.gpu
def test_sample_rows_bounded_by_the_workspace():
    """1000 rows of 500000 tokens go in two groups of launches; each row's token is the one it gets alone."""
    B, V, n = 1000, 500000, len(SETTINGS)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    import int8_quantized_amd as q8
    x = torch.randn((B, V), generator=g, device="cuda") * 3
    t, k, p, mp = (torch.tensor(v, device="cuda") for v in zip(*[SETTINGS[i % n] for i in range(B)]))
    k, u = k.int(), torch.rand(B, generator=g, device="cuda")
    got, lp = torch.full((B,), -7, dtype=torch.int32, device="cuda"), torch.zeros(B, device="cuda")
    q8.q8ta_sample(x, t, k, p, mp, u, got, lp)
    want, want_lp = torch.full_like(got, -8), torch.ones_like(lp)
    for a in range(0, B, 100):
        q8.q8ta_sample(*(v[a:a + 100] for v in (x, t, k, p, mp, u, want, want_lp)))
    assert torch.equal(got, want) and torch.equal(lp, want_lp) and (got >= 0).all()
