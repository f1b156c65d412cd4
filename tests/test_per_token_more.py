"""q8ta_norm_quantize of rows whose mean square is infinite, or next to it.

Tolerance.  What is left of a row with an infinite mean square is residual_scale * residual: half a step of the type
after one rounding to fp32.
"""
import math

import pytest

from test_per_token import EPS, TYPES, U32, half_step, norm_case, run_norm, smallest

torch = pytest.importorskip("torch")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,N", [(4, 1), (5, 300), (4, 512), (520, 4104), (514, 5120), (513, 7168), (515, 9000), (3, 16400), (3, 20000)])
@pytest.mark.parametrize("residual,gate", [(True, None), (True, "row"), (False, "one")])
def test_an_infinite_value_before_a_norm_leaves_the_others_of_its_row(residual, gate, T, N, dtype):
    """rms(x) is 0 there: b is 0, or NaN where x is infinite; a NaN spoils its row, and no row another."""
    c = norm_case(T, N, dtype, post=True, gate=gate, residual=residual, seed=N)
    plain = run_norm(c)
    x = c["x"]
    x[0, N // 2] = math.inf
    x[1, 0] = -math.inf
    x[1, N - 1] = math.inf
    x[2, N // 3] = math.nan
    out, codes, scales = run_norm(c)
    for r in (0, 1):
        odd = torch.isinf(x[r])
        assert torch.isnan(out[r][odd]).all()
        want = c["residual"][r].double() * c["scale"] if residual else torch.zeros(N, dtype=torch.float64)
        off = (out[r].double() - want).abs()[~odd]
        assert (off <= want.abs()[~odd] * (half_step(TYPES[dtype]) + U32) * 1.001 + smallest(TYPES[dtype])).all()
    assert torch.isnan(out[2]).all()
    assert torch.isnan(scales[:3]).all() and (codes[:3] == 0).all()
    for got, want in zip((out, codes, scales), plain):
        assert torch.equal(got[3:], want[3:])


@pytest.mark.gpu
@pytest.mark.parametrize("N", [256, 20000])
def test_large_values_are_not_infinite(N):
    """The squares of fp32's and bf16's largest values fit the mean."""
    for dtype in ("fp32", "bf16"):
        c = norm_case(3, N, dtype, seed=2)
        c["x"][0] = torch.finfo(TYPES[dtype]).max
        c["x"][1, 3] = -torch.finfo(TYPES[dtype]).max
        b = c["x"].double()
        b = b / (b.square().mean(1, keepdim=True) + EPS).sqrt() * c["post"].double() * c["gate"].double()
        b = b + c["residual"].double() * c["scale"]
        out, codes, scales = run_norm(c)
        assert ((out.double() - b).abs() <= b.abs() * (half_step(TYPES[dtype]) + U32) * 1.001 + smallest(TYPES[dtype])).all()
        assert torch.isfinite(scales).all() and (codes.abs().amax(1) == 127).all()
