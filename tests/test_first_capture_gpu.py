"""The first call of a process made while a stream is captured, for each kernel of the dense products and experts: nothing that
a call asks of the device or sets up once may need a call before the capture.  Each in a process of its own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import sys
import torch
import lora_adapter_application_b200 as lora

kind = sys.argv[1]
dtype = torch.float32 if kind.startswith("fp32") else torch.bfloat16
T, d, n, N, k = (300 if "tile" in kind else 40), (255 if "odd" in kind else 256), 264, 4, 2
g = torch.Generator(device="cuda").manual_seed(1)
ints = lambda most, *s: torch.randint(-most, most + 1, s, generator=g, device="cuda").double()
status = torch.zeros(1, dtype=torch.int32, device="cuda")
x, w = ints(2, T, d), ints(2, N, n, d) / 16      # z in steps of 1 / 16 up to 64: exact in any order
xs, ws = x.to(dtype), w.to(dtype)
ids, weights = torch.full((T, k), -7, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
logits = ints(9, T, N).to(dtype)
chosen = torch.sort(logits.double(), dim=1, descending=True, stable=True).indices[:, :k].int()
meta = lora.Meta(T * k, N, min_run=0)
y, z = torch.zeros(T, n, dtype=dtype, device="cuda"), torch.zeros(T * k, n, dtype=dtype, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    if "experts" in kind:
        lora.lora_expert_route(ids, weights, logits)
        lora.lora_build_segments(ids.view(-1), meta, status)
        lora.lora_expert_linear(z, xs, ws, meta, status, x_div=k)
        lora.lora_expert_sum(y, z, ids, weights, N)
    else:
        lora.lora_linear(y, xs, ws[0], status)
for _ in range(2):
    y.zero_(), z.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    if "experts" in kind:
        assert torch.equal(ids, chosen)
        for e in range(N):
            mine = (ids.view(-1) == e).nonzero()[:, 0]
            assert torch.equal(z[mine], (x[mine // k] @ w[e].T).to(dtype))
        total = (weights.double()[:, :, None] * z.double().view(T, k, n))
        assert ((y.double() - total.sum(1)).abs() <= total.abs().sum(1) * 3 * 2.0 ** -24 + total.sum(1).abs() * torch.finfo(dtype).eps / 2 * 1.01).all()
    else:
        assert torch.equal(y, (x @ w[0].T).to(dtype))
print("as it should be")
"""


@pytest.mark.parametrize("kind", ["bf16", "bf16 odd", "bf16 experts", "bf16 odd experts", "fp32", "fp32 tile experts"])
def test_first_call_of_a_process_is_captured(cuda_lib, kind):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", PROGRAM, kind], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "as it should be" in p.stdout, p.stdout + p.stderr
