"""lora_linear and lora_expert_linear over rows off 16-byte steps, at every offset of a row in its 16 bytes and with row ends in every
part of them (all around the rows lies NaN, none of which may reach a sum); calls repeated."""
import math

import pytest
import torch

import lora_adapter_application_b200 as lora
from dense_helpers import whole

pytestmark = pytest.mark.gpu


def _rows(t, off, pad):
    """t's rows in bf16 from element `off` of a buffer of NaN, `pad` elements apart."""
    rows, d = t.shape
    buf = torch.full((off + rows * (d + pad) + 8,), math.nan, dtype=torch.bfloat16, device="cuda")
    v = buf[off:off + rows * (d + pad)].view(rows, d + pad)[:, :d]
    v.copy_(t)
    return v


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("T", [1, 3, 150])
@pytest.mark.parametrize("d", [1, 2, 7, 9, 15, 17, 57, 63, 65, 71, 73, 127, 129, 135, 137, 193, 201, 263])
def test_rows_at_every_offset(cuda_lib, T, d, grouped):
    n, N = 10, 2
    g = torch.Generator(device="cuda").manual_seed(d)
    x, w = whole(g, (T, d), 2), whole(g, (N, n, d), 2)
    ids = (torch.arange(T) % N).int()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    meta = lora.Meta(T, N, min_run=0)
    lora.lora_build_segments(ids.cuda(), meta, status)
    want = torch.einsum("td,tnd->tn", x, w[ids.cuda().long()] if grouped else w[:1].expand(T, n, d)).bfloat16()   # exact in any order
    for off in range(8):
        for pad in (0, 1, 2, 6):
            y = torch.full((T, n), 7.0, dtype=torch.bfloat16, device="cuda")
            xs, ws = _rows(x, off, pad), _rows(w.view(N * n, d), (3 * off + 1) % 8, 0 if grouped else pad)
            if grouped:
                lora.lora_expert_linear(y, xs, ws.view(N, n, d), meta, status)
            else:
                lora.lora_linear(y, xs, ws[:n], status)
            assert torch.equal(y, want), (off, pad)
    assert int(status.item()) == 0


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
