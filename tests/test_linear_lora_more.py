"""q8ta_linear_lora at the ends of its stated range, and its adapter sums where their terms cancel."""
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


@pytest.mark.gpu
@pytest.mark.parametrize("ad", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("out", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,N", [(3, 40), (64, 700), (1100, 1100), (2050, 4200)])
def test_linear_lora_adapter_sums_are_held_in_32_bits(M, N, out, ad):
    """Row kernel and GEMMs alike.  t0 = sum x and t1 = t0 - x[m, 5] are whole numbers below 2^24, and the
    output b t0 - b t1 = b x[m, 5]: off by the roundings of two products and their sum, 4 * 2^-24 of
    |b| (t0 + t1), and by its own to the type.  (t in 17 bits: off by up to |b|.)"""
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N)
    K, r = 4096, 16
    x = torch.randint(1, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    a = torch.zeros((1, r, K), device="cuda", dtype=ad)
    a[0, :2] = 1
    a[0, 1, 5] = 0
    b = torch.zeros((1, N, r), device="cuda", dtype=ad)
    b[0, :, 0] = torch.randn(N, generator=g, device="cuda").to(ad)
    b[0, :, 1] = -b[0, :, 0]
    y = torch.full((M, N), 9.0, dtype=out, device="cuda")
    q8.q8ta_linear_lora(x, 1.0, 0, torch.zeros((N, K), dtype=torch.int8, device="cuda"),
                        torch.ones(N, device="cuda"), None, a, b, None, None,
                        torch.zeros(M, dtype=torch.int32, device="cuda"), "none", y)
    b0, t0 = b[0, :, 0].double(), x.double().sum(1, keepdim=True)
    want = b0 * x[:, 5:6].double()
    tol = 4 * 2.0 ** -24 * b0.abs() * (2 * t0 - x[:, 5:6].double())
    tol = tol + (want.abs() + tol) * torch.finfo(out).eps / 2 + torch.finfo(out).smallest_normal
    off = (y.double() - want).abs()
    assert (off <= tol).all(), float((off / tol).max())
