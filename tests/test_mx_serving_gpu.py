"""The microscaled operators as a server runs them: the norm feeds the base product and the
adapters, the base product's y goes to lora_add_linear; an adapter is merged into a base weight
held in 4 bits; steps are captured and replayed, and run on streams side by side."""
import numpy as np
import pytest
import torch

import lora_adapter_application_b200 as lora
import oracle
import workloads
from gpu_helpers import DeviceLayer, assert_within, build_meta
from mx_helpers import as64, from_device, to_device
from oracle import mx

pytestmark = pytest.mark.gpu


class Step:
    """One fused layer of a step: norm with the residual's sum, base product, adapters."""

    def __init__(self, seed=5, T=96, d=1024, d_out=(512, 128, 128), r_max=16, runs=((40, 2),), fmt=lora.LORA_MXFP8):
        self.w = workloads.random_case(seed, T, 6, d, list(d_out), r_max, runs=list(runs), dtype=torch.bfloat16)
        self.lay = self.w.layers[0]
        self.dev = DeviceLayer(self.lay)
        self.meta, self.status = build_meta(self.w.ids, self.w.N)
        g = torch.Generator().manual_seed(seed)
        n = sum(d_out)
        self.W = lora.MxTensor(n, d, lora.LORA_MXFP4)
        lora.lora_mx_quantize(self.W, (torch.randn(n, d, generator=g) / d ** 0.5).to(torch.bfloat16).cuda())
        self.x = self.lay.x.cuda()
        self.residual = torch.randn(T, d, generator=g).to(torch.bfloat16).cuda()
        self.weight = (1 + 0.1 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda()
        self.sum, self.h = torch.empty_like(self.x), torch.empty_like(self.x)
        self.xq = lora.MxTensor(T, d, fmt)
        self.y = torch.empty(T, n, dtype=torch.bfloat16, device="cuda")
        self.ranks = self.w.ranks.cuda()
        self.alphas = lora.alphas_full(self.w.alpha, self.w.N)

    def base(self):
        lora.lora_rms_norm(self.h, self.x, self.weight, 1e-5, residual=self.residual, residual_out=self.sum, q=self.xq)
        lora.lora_mx_linear(self.y, self.xq, self.W, self.status)

    def __call__(self):
        self.base()
        lora.lora_add_linear(self.y, self.h, self.dev.A, self.dev.B, self.dev.col_off, self.ranks, self.alphas,
                             self.meta, self.status)


@pytest.mark.parametrize("fmt", [lora.LORA_MXFP8, lora.LORA_MXFP4])
def test_norm_base_product_and_adapters(cuda_lib, fmt):
    """Each operator against 64 bits on what the one before it gave."""
    s = Step(fmt=fmt)
    d = s.x.shape[1]
    s.base()
    y0 = s.y.cpu().clone()
    lora.lora_add_linear(s.y, s.h, s.dev.A, s.dev.B, s.dev.col_off, s.ranks, s.alphas, s.meta, s.status)
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    r = (s.x.cpu().double() + s.residual.cpu().double()).to(torch.bfloat16)
    assert torch.equal(s.sum.cpu(), r)
    ref = mx.rms_norm(as64(r), as64(s.weight)[None], 1e-5)
    # fp32 arithmetic (derivation: test_mx_rows_gpu.py) and one rounding to bf16
    assert (np.abs(as64(s.h) - ref) <= np.abs(ref) * ((d / 2 + 6) * 2.0 ** -24 + 2.0 ** -8)).all()
    codes, scales = from_device(s.xq)
    rc, rs = mx.quantize(as64(s.h), fmt)
    np.testing.assert_array_equal(codes, rc)
    np.testing.assert_array_equal(scales, rs)
    wc, ws = from_device(s.W)
    xv, wv = mx.values(codes, scales, fmt, d), mx.values(wc, ws, mx.MXFP4, d)
    ref = xv @ wv.T
    bound = np.abs(ref) * 2.0 ** -8 + d * 2.0 ** -23 * (np.abs(xv) @ np.abs(wv).T)
    assert (np.abs(as64(y0) - ref) <= bound).all()
    yref = oracle.lora_apply(s.h.cpu(), s.lay.A, s.lay.B, s.lay.col_off, s.w.ranks, s.w.alpha, s.w.ids, y0)
    assert_within(as64(s.y), yref, torch.bfloat16, "delta on the microscaled base")
    none = s.w.ids < 0
    assert torch.equal(s.y.cpu()[none], y0[none])


def test_merge_an_adapter_into_a_4_bit_base(cuda_lib):
    """Read back, merge, quantise again: each against 64 bits, and the product follows."""
    s = Step(seed=9, d_out=(384,))
    d, n = s.x.shape[1], 384
    dense = torch.empty(n, d, dtype=torch.bfloat16, device="cuda")
    lora.lora_mx_dequantize(dense, s.W)
    wc, ws = from_device(s.W)
    np.testing.assert_array_equal(as64(dense), mx.values(wc, ws, mx.MXFP4, d))
    before = dense.cpu().clone()
    lora.lora_merge_adapter(dense, s.dev.A[0], s.dev.B[0], 2, s.ranks, s.alphas, s.status)
    rank = int(s.w.ranks[2])
    ref = oracle.lora_merge(before, s.lay.A[0][2], s.lay.B[0][2], rank, float(s.w.alpha), 1)
    assert_within(as64(dense), ref, torch.bfloat16, "merge")
    merged = lora.MxTensor(n, d, lora.LORA_MXFP4)
    lora.lora_mx_quantize(merged, dense)
    mc, ms = from_device(merged)
    rc, rs = mx.quantize(as64(dense), mx.MXFP4)
    np.testing.assert_array_equal(mc, rc)
    np.testing.assert_array_equal(ms, rs)
    s.base()
    y = torch.empty(s.x.shape[0], n, device="cuda")
    lora.lora_mx_linear(y, s.xq, merged, s.status)
    codes, scales = from_device(s.xq)
    xv, wv = mx.values(codes, scales, mx.MXFP8, d), mx.values(mc, ms, mx.MXFP4, d)
    assert (np.abs(as64(y) - xv @ wv.T) <= d * 2.0 ** -23 * (np.abs(xv) @ np.abs(wv).T) + 1e-30).all()
    assert int(s.status.item()) == 0


@pytest.mark.parametrize("T,runs", [(1, ()), (96, ((40, 2),)), (700, ((300, 1), (200, 3)))])
def test_captured_step_replays(cuda_lib, T, runs):
    """A step captured once and replayed on new inputs = the same step run eagerly; two graphs that
    share every buffer but their outputs replay one after the other."""
    s = Step(seed=T, T=T, runs=runs)
    for _ in range(2):
        s()                                            # first calls before the capture
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        s.y = torch.empty_like(s.y)
        with torch.cuda.graph(g, stream=side):
            s()
        graphs.append((g, s.y))
    for k in range(3):
        gen = torch.Generator().manual_seed(100 + k)
        s.x.copy_(torch.randn(s.x.shape, generator=gen).to(torch.bfloat16))
        outs = []
        for g, y in graphs:
            g.replay()
            outs.append(y)
        torch.cuda.synchronize()
        outs = [y.clone() for y in outs]
        s.y = torch.empty_like(s.y)
        s()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], s.y) and torch.equal(outs[1], s.y)
    assert int(s.status.item()) == 0


@pytest.mark.parametrize("shapes", [[(1, 4096, 4096), (8, 4096, 4096)], [(64, 4096, 6144), (300, 2048, 4096)],
                                    [(2000, 1024, 2048), (48, 4096, 1024)], [(700, 1024, 2048), (900, 1024, 2048)]])
def test_products_on_two_streams(cuda_lib, shapes):
    """Products that run at the same time, sharing the status word alone, give what they give alone."""
    ops = []
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for k, (T, d, n) in enumerate(shapes):
        g = torch.Generator(device="cuda").manual_seed(k)
        x, w = lora.MxTensor(T, d, k % 2), lora.MxTensor(n, d, lora.LORA_MXFP4)
        lora.lora_mx_quantize(x, torch.randn(T, d, generator=g, device="cuda"))
        lora.lora_mx_quantize(w, torch.randn(n, d, generator=g, device="cuda"))
        alone = torch.empty(T, n, device="cuda")
        lora.lora_mx_linear(alone, x, w, status)
        ops.append((x, w, alone))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    outs = [[torch.empty_like(o[2]) for _ in range(12)] for o in ops]
    for i in range(12):
        for st, (x, w, _), ys in zip(streams, ops, outs):
            lora.lora_mx_linear(ys[i], x, w, status, stream=st)   # another stream than the current one
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for (_, _, alone), ys in zip(ops, outs):
        for y in ys:
            assert torch.equal(y, alone)


def test_product_beside_the_adapters_kernels(cuda_lib):
    """A base product on one stream while lora_add_linear's prompt and decode kernels (which hold tensor memory
    of their own) run on another."""
    s = Step(seed=3, T=1500, d=1024, runs=((600, 1), (500, 4)))
    s()
    torch.cuda.synchronize()
    want, base = s.y.clone(), None
    x, w = lora.MxTensor(8, 4096, lora.LORA_MXFP8), lora.MxTensor(4096, 4096, lora.LORA_MXFP4)
    lora.lora_mx_quantize(x, torch.randn(8, 4096, device="cuda"))
    lora.lora_mx_quantize(w, torch.randn(4096, 4096, device="cuda"))
    base = torch.empty(8, 4096, device="cuda")
    lora.lora_mx_linear(base, x, w, s.status)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    ys = [torch.empty_like(base) for _ in range(30)]
    for i in range(30):
        lora.lora_mx_linear(ys[i], x, w, s.status, stream=other)
        if i % 3 == 0:
            s()
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0 and torch.equal(s.y, want)
    assert all(torch.equal(y, base) for y in ys)


def test_first_calls_inside_a_capture(cuda_lib):
    """A fresh process whose first calls of every operator are captured (loading and planning happen there)."""
    code = """
import torch, lora_adapter_application_b200 as lora
T, d, n = 3, 1024, 512
x = torch.randn(T, d, device="cuda").bfloat16()
wf = (torch.randn(n, d, device="cuda") / 32).bfloat16()
wt = torch.ones(d, device="cuda").bfloat16()
xq, w, big = lora.MxTensor(T, d, 0), lora.MxTensor(n, d, 1), lora.MxTensor(2000, d, 1)
h, r, y = torch.empty_like(x), torch.zeros_like(x), torch.empty(T, n, device="cuda")
many, yb = torch.randn(2000, d, device="cuda"), torch.empty(2000, n, device="cuda")
st = torch.zeros(1, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
def step():
    lora.lora_mx_quantize(w, wf)
    lora.lora_rms_norm(h, x, wt, 1e-5, residual=r, residual_out=torch.empty_like(x), q=xq)
    lora.lora_mx_linear(y, xq, w, st)
    lora.lora_mx_quantize(big, many)
    lora.lora_mx_linear(yb, big, w, st)
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
a, b = y.clone(), yb.clone()
y.zero_(), yb.zero_()
step()
torch.cuda.synchronize()
assert torch.equal(a, y) and torch.equal(b, yb) and int(st) == 0 and float(y.abs().max()) > 0
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]


def test_an_events_wait_between_two_calls(cuda_lib):
    """A product whose rows another stream wrote, behind a product on its own stream: the event is waited for."""
    w, st = lora.MxTensor(2048, 2048, lora.LORA_MXFP4), torch.zeros(1, dtype=torch.int32, device="cuda")
    lora.lora_mx_quantize(w, torch.randn(2048, 2048, device="cuda"))
    x0, x1 = lora.MxTensor(16, 2048, 0), lora.MxTensor(16, 2048, 0)
    rows = [torch.randn(16, 2048, device="cuda") for _ in range(20)]
    lora.lora_mx_quantize(x0, rows[0])
    want = []
    for r in rows:
        lora.lora_mx_quantize(x1, r)
        want.append(torch.empty(16, 2048, device="cuda"))
        lora.lora_mx_linear(want[-1], x1, w, st)
    big = torch.randn(8192, 8192, device="cuda")
    torch.cuda.synchronize()
    other, scratch = torch.cuda.Stream(), torch.empty(16, 2048, device="cuda")
    for r, y in zip(rows, want):
        got = torch.empty_like(y)
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            big.mul_(1.0)                              # some time before the rows are there
            lora.lora_mx_quantize(x1, r)
            e = torch.cuda.Event()
            e.record()
        lora.lora_mx_linear(scratch, x0, w, st)
        torch.cuda.current_stream().wait_event(e)
        lora.lora_mx_linear(got, x1, w, st)
        torch.cuda.synchronize()
        assert torch.equal(got, y)
    assert int(st.item()) == 0
