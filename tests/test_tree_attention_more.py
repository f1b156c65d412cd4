"""q8ta_tree_attention: the precision of its probabilities.

With fp16 outputs a probability is held in two fp16 parts (2^-22 of it) and everything else in 32
bits, so that an output is off by its own rounding and little else: the tests below leave half a step
of the type, and of sums over n keys (n / 8 + 64) * 2^-24 of sum |p v|.
"""
import numpy as np
import pytest

from test_tree_attention import make, definition, run

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
