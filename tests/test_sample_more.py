"""q8ta_sample: numbers outside [0, 1)."""
import numpy as np
import pytest

from test_sample import SETTINGS, rows, run

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
