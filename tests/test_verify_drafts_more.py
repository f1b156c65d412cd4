"""q8ta_verify_drafts at temperatures and logits at the ends of fp32."""
import numpy as np
import pytest

from test_verify_drafts import check, make

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
