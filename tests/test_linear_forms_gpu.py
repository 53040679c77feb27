"""lora_linear: equal calls."""
import pytest
import torch

import lora_adapter_application_b200 as lora

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d,n,gated", [(1, 4096, 4096, False), (64, 4096, 1024, False), (257, 4096, 520, False), (200, 4096, 1024, True),
                                         (1500, 512, 2560, True), (3, 4095, 300, False), (500, 1001, 600, True)])
def test_equal_calls_give_equal_bits(cuda_lib, T, d, n, gated, dtype):
    """One tile a cluster and many, k split and whole, both ways that rows come; other work between the calls."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x, w = (torch.randn(m, d, generator=g, device="cuda").to(dtype) for m in (T, 2 * n if gated else n))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ys = [torch.full((T, n), float(i), dtype=dtype, device="cuda") for i in range(4)]
    for y in ys:
        lora.lora_linear(y, x, w, status, act=lora.ACT_SILU, gated=gated)
        lora.lora_linear(torch.empty_like(y), x.neg(), w, status, gated=gated)
    assert all(torch.equal(y, ys[0]) for y in ys) and int(status.item()) == 0
