"""q8ta_norm_quantize of rows whose mean square is infinite, or next to it, and the gated block's activations down to
the smallest that are promised.

Tolerances.  What is left of a row with an infinite mean square is residual_scale * residual: half a step of the type
after one rounding to fp32.  A gate's activation is off by 2^-21 of itself (as in test_per_token.py), or is 0 where
it is below 2^-118; the argument z of the tanh form's logistic has up to six roundings, each of 2^-24 of z,
and e^z changes by that much of itself.
"""
import math

import numpy as np
import pytest

import int8_quantized_amd as q8
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


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M", [2, 100, 900])
@pytest.mark.parametrize("up", [1.0, 2.0 ** 100])
def test_gates_whose_activation_is_small(act, M, up):
    """A gate's bias alone: activations down to 2^-118, and that or less from there on."""
    N, K = 4096, 64
    g = torch.linspace(-140.0, -60.0, N) if act == "silu" else torch.linspace(-12.5, -8.0, N)
    x, w = torch.zeros(M, K, dtype=torch.int8, device="cuda"), torch.zeros(N, K, dtype=torch.int8, device="cuda")
    one, out = torch.ones(max(M, N), device="cuda"), torch.full((M, N), 9.0, device="cuda")
    q8.q8ta_gated_linear(x, one[:M], w, one[:N], g.cuda(), w, one[:N], torch.full((N,), up, device="cuda"), act, out)
    v = g.double().numpy()
    z = v if act == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    a = v * np.exp(z) / (1 + np.exp(z))
    tol = np.abs(a) * (2.0 ** -21 + (6 * np.abs(z) * 2.0 ** -24 if act == "gelu_tanh" else 0.0))
    tol = np.where(np.abs(a) < 2.0 ** -118, np.abs(a), tol)
    want, tol = a * up, 1.01 * tol * up + U32 * np.abs(a * up) + 2.0 ** -150
    got = out.cpu().double().numpy()
    assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()
    assert (a < 0).all() and ((got <= 0).all())
