"""q8ta_linear_lora at the ends of its stated range."""
import numpy as np
import pytest

import int8_quantized_amd as q8

torch = pytest.importorskip("torch")


@pytest.mark.gpu
@pytest.mark.parametrize("K,N", [(16, 402653184 + 100), (3, 1 << 30)])
def test_linear_lora_channels_beyond_one_launch(K, N):
    """More channels than a launch has threads for, and (K = 3) more rows to copy: every channel is
    written.  Whole numbers below 2^8 and a scale of 1 make each output exact."""
    free, _ = torch.cuda.mem_get_info()
    if free < 120 << 30:
        pytest.skip("needs 120 GiB of device memory")
    i = torch.arange(N, device="cuda", dtype=torch.int32)
    w = torch.empty((N, K), dtype=torch.int8, device="cuda")
    w[:] = (i % 7 - 3).to(torch.int8).unsqueeze(1)
    b = (i % 5 - 2).to(torch.bfloat16).view(1, N, 1)
    del i
    x = torch.ones((1, K), dtype=torch.int8, device="cuda")
    a = torch.ones((1, 1, K), dtype=torch.bfloat16, device="cuda")
    ws = torch.ones(N, device="cuda")
    out = torch.full((1, N), -100.0, dtype=torch.bfloat16, device="cuda")
    q8.q8ta_linear_lora(x, 1.0, 0, w, ws, None, a, b, None, None,
                        torch.zeros(1, dtype=torch.int32, device="cuda"), "none", out)
    want = w[:, 0].to(torch.bfloat16)
    want += b.view(N)
    want *= K                                   # at most 5 * 16: exact
    assert torch.equal(out[0], want)
    del w, b, ws, out, want
    torch.cuda.empty_cache()
