"""q8ta_rope_append: queries are rounded to fp32 and from there to their type."""
import pytest

from test_rope_append import TYPES, case, run

torch = pytest.importorskip("torch")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d", [128, 100])    # the vector kernel, and the one for any size
def test_rope_append_roundings_of_queries(d, interleaved, dtype):
    """Angles of 0 leave factor * x, one product in 64 bits: what becomes of it next to the type's ties."""
    half = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    for factor in (1 + half + 2.0 ** -30, 1 + 3 * half - 2.0 ** -30, 1 + half + 2.0 ** -51, 1.2079441541679836):
        c = list(case(64, 16, 2, d, d, dtype, interleaved, 16, fused=False, seed=d))
        c[0].copy_(torch.where(torch.rand(c[0].shape, device="cuda") < 0.5, torch.ones_like(c[0]), c[0]))
        c[3][:], c[6] = 0, factor
        got = run(*c, 16)[0]
        want = (c[0].double() * factor).float().to(TYPES[dtype])
        assert torch.equal(got, want), factor
