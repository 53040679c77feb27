"""The microscaled base product on the GPU against 64-bit products of the stored values.

Two kinds of inputs.  Integers: values that are small whole numbers, so that every partial sum
is a whole number below 2^24 and fp32 holds it exactly in any order; y must then be the exact
sum, rounded once.  Random: fp32 accumulation of K exact products in any order is off by at most
K 2^-23 sum |x w| (2^-23: a hardware adder may truncate instead of rounding), then one
rounding of eps(dtype) / 2; and over a whole matrix the rounding errors are spread, so the
error's norm is held to the norm of y times eps(dtype) / 2."""
import numpy as np
import pytest
import torch

import lora_adapter_application_b200 as lora
from mx_helpers import as64, to_device
from oracle import mx

pytestmark = pytest.mark.gpu
FMT = [lora.LORA_MXFP8, lora.LORA_MXFP4]
DTYPES = [torch.bfloat16, torch.float32]


def _whole(seed, rows, cols, fmt):
    """Codes and scales of whole-number values: |element| <= 6, scales 1, 2, 4 (MXFP4: 2, 4, 8, its halves whole)."""
    g = np.random.default_rng(seed)
    t = mx.table(fmt)
    pick = np.array([c for c in range(len(t)) if t[c] <= 6 and (fmt == mx.MXFP4 or t[c] == int(t[c]))])
    codes = np.zeros((rows, mx.padded(cols)), np.uint8)
    codes[:, :cols] = pick[g.integers(0, len(pick), (rows, cols))]
    codes[:, :cols] += ((g.random((rows, cols)) < 0.5) * (128 if fmt == mx.MXFP8 else 8)).astype(np.uint8)
    scales = 127 + (fmt == mx.MXFP4) + g.integers(0, 3, (rows, mx.padded(cols) // 32))
    return codes, scales.astype(np.uint8)


def _product(x, w):
    """x w^T in fp64 on the GPU."""
    return (torch.from_numpy(x).cuda() @ torch.from_numpy(w).cuda().T).cpu()


def _run(T, xm, wm, dtype, ld=None):
    n = wm.rows
    y = torch.full((T, ld or n), 7.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lora.lora_mx_linear(y[:, :n], xm, wm, status)
    assert int(status.item()) == 0
    assert (y[:, n:] == 7).all()
    return y[:, :n].cpu()


SHAPES = [(1, 1, 1), (1, 32, 128), (1, 128, 128), (16, 256, 128), (17, 384, 100), (3, 1000, 260), (33, 512, 130),
          (64, 2048, 1024), (65, 640, 257), (128, 1003, 300), (129, 4096, 129), (200, 8192, 64), (300, 264, 520),
          (1000, 1152, 1000), (2, 14336, 640), (1, 4096, 4096), (256, 28672, 96), (513, 1, 1), (2049, 128, 33),
          (257, 1408, 384), (193, 128, 128), (400, 4224, 260), (500, 3000, 700), (16, 16384, 128), (31, 896, 9000),
          (7, 2176, 20000), (700, 640, 257), (1024, 8192, 2304), (5000, 300, 3000), (6000, 1920, 4500)]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("T,d,n", SHAPES)
def test_whole_numbers_are_exact(cuda_lib, T, d, n, fmt):
    xc, xs = _whole(T + d, T, d, fmt)
    wc, ws = _whole(n + d + 1, n, d, mx.MXFP4)
    ref = _product(mx.values(xc, xs, fmt, d), mx.values(wc, ws, mx.MXFP4, d))
    assert ref.abs().max() < 2 ** 24
    xm, wm = to_device(xc, xs, fmt, d), to_device(wc, ws, mx.MXFP4, d)
    for dtype in DTYPES:
        for ld in (None, n + 5):
            assert torch.equal(_run(T, xm, wm, dtype, ld), ref.to(dtype)), (dtype, ld)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,n", [(1, 4096, 4096), (48, 4096, 1024), (100, 14336, 512), (513, 2000, 777)])
def test_random_values(cuda_lib, T, d, n, fmt, dtype):
    g = np.random.default_rng(T * d)
    xc, xs = mx.quantize(g.standard_normal((T, d)) * np.exp(0.7 * g.standard_normal(d)), fmt)
    wc, ws = mx.quantize(g.standard_normal((n, d)) / d ** 0.5, mx.MXFP4)
    x, w = mx.values(xc, xs, fmt, d), mx.values(wc, ws, mx.MXFP4, d)
    ref, mag = _product(x, w).numpy(), _product(np.abs(x), np.abs(w)).numpy()
    y = as64(_run(T, to_device(xc, xs, fmt, d), to_device(wc, ws, mx.MXFP4, d), dtype))
    half = torch.finfo(dtype).eps / 2
    rel = np.linalg.norm(y - ref) / np.linalg.norm(ref)
    print(f"rel {rel:.3g}, max {np.abs(y - ref).max() / np.abs(ref).max():.3g}")
    assert (np.abs(y - ref) <= half * np.abs(ref) + d * 2.0 ** -23 * mag).all()
    if dtype == torch.bfloat16:
        assert rel <= half


@pytest.mark.parametrize("fmt", FMT)
def test_scale_extremes_and_nan_blocks(cuda_lib, fmt):
    """Scales far apart in x and w meet in range; a NaN block of x makes its row NaN, one of w its
    column, and nothing else; NaN scale bytes of rows that are not part of the call reach nothing."""
    T, d, n = 5, 512, 130
    xc, xs = _whole(1, 200, d, fmt)
    wc, ws = _whole(2, n, d, mx.MXFP4)
    up, down = xs.astype(int) + 90, ws.astype(int) - 90
    xs, ws = up.astype(np.uint8), down.astype(np.uint8)
    ref = _product(mx.values(xc, xs, fmt, d)[:T], mx.values(wc, ws, mx.MXFP4, d))
    xs[T:] = 255
    xm, wm = to_device(xc, xs, fmt, d), to_device(wc, ws, mx.MXFP4, d)
    wm.scales[torch.from_numpy(mx.scale_index(256, d // 32)[n:].ravel()).cuda()] = 255
    assert torch.equal(_run(T, xm, wm, torch.float32), ref.float())
    xs[2, 3], ws[7, 15] = 255, 255
    y = _run(T, to_device(xc, xs, fmt, d), to_device(wc, ws, mx.MXFP4, d), torch.float32)
    nan = torch.zeros(T, n, dtype=torch.bool)
    nan[2], nan[:, 7] = True, True
    assert torch.equal(torch.isnan(y), nan)
    assert torch.equal(y[~nan], ref.float()[~nan])


def test_no_rows(cuda_lib):
    xm, wm = lora.MxTensor(4, 128, 0), lora.MxTensor(64, 128, 1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lora.lora_mx_linear(torch.empty(0, 64, device="cuda"), xm, wm, status)
    assert int(status.item()) == 0


def _whole_on_gpu(rows, cols, fmt, most, g):
    v = torch.randint(-most, most + 1, (rows, cols), generator=g, device="cuda", dtype=torch.int8)
    m = lora.MxTensor(rows, cols, fmt)
    lora.lora_mx_quantize(m, v.to(torch.bfloat16))
    return m, v


def _check_whole(T, d, n, fmt, dtype, pad, seed):
    """Whole numbers up to 3 and 2 (exact in every format: a block's largest is at most 3): the exact product."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    (xm, xv), (wm, wv) = _whole_on_gpu(T, d, fmt, 3, g), _whole_on_gpu(n, d, mx.MXFP4, 2, g)
    y = torch.full((T + 1, n + pad), 99.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lora.lora_mx_linear(y[:T, :n], xm, wm, status)
    ref = torch.zeros(T, n, dtype=torch.float64, device="cuda")
    for lo in range(0, d, 65536):
        ref += xv[:, lo:lo + 65536].double() @ wv[:, lo:lo + 65536].double().T
    assert ref.abs().max() < 2 ** 24 and int(status.item()) == 0
    assert torch.equal(y[:T, :n], ref.to(dtype)), (T, d, n, fmt, dtype, pad)
    assert (y[T] == 99).all() and (y[:, n:] == 99).all()


@pytest.mark.parametrize("seed", range(8))
def test_random_shapes_are_exact(cuda_lib, seed):
    r = np.random.default_rng(seed)
    done = 0
    while done < 25:
        T, d, n = int(2 ** r.uniform(0, 11.5)), int(2 ** r.uniform(0, 13.5)), int(2 ** r.uniform(0, 14.5))
        if r.random() < 0.4:
            d = max(128, d // 128 * 128)
        if r.random() < 0.4:
            n = max(8, n // 8 * 8)
        if T * d * n > 1 << 36:
            continue
        done += 1
        _check_whole(T, d, n, int(r.integers(2)), DTYPES[int(r.integers(2))], int(r.choice([0, 0, 1, 8])), done)


@pytest.mark.parametrize("T,d,n", [(1, 512, 19000), (64, 1024, 28672), (100, 640, 20001), (128, 896, 37888), (128, 896, 38000),
                                   (17, 384, 18960), (250, 512, 11000)])
@pytest.mark.parametrize("fmt", FMT)
def test_wide_outputs_are_exact(cuda_lib, T, d, n, fmt):
    """Output widths of one to two tiles of features a multiprocessor, and beside them."""
    for dtype in DTYPES:
        _check_whole(T, d, n, fmt, dtype, 3, T + n)


@pytest.mark.parametrize("T,d,n,fmt", [(1, 1 << 20, 128, 0), (300, 1 << 20, 130, 1), (600, 1 << 19, 128, 0), (131072, 64, 72, 1),
                                       (1, 96, 1 << 20, 0)])
def test_largest_sizes_are_exact(cuda_lib, T, d, n, fmt):
    _check_whole(T, d, n, fmt, torch.float32, 0, 1)


# few rows: k split over a cluster with and without a place of its own for the partial sums, one tile and several a block,
# two accumulators of a tile, all of k within the ring; many rows: one tile a pair and several
@pytest.mark.parametrize("T,d,n,fmt", [(1, 4096, 4096, 0), (64, 4096, 4096, 1), (257, 14336, 4096, 0), (4, 256, 512, 0), (40, 384, 130, 1),
                                       (64, 4096, 28672, 0), (128, 4096, 28672, 1), (1024, 2048, 4096, 0), (1200, 256, 2300, 1),
                                       (3000, 1920, 4500, 0), (3000, 4096, 8192, 1)])
@pytest.mark.parametrize("role", [1, 2, 3, 4, 5])
def test_stalled_warp_times_out_and_the_context_survives(cuda_lib, monkeypatch, T, d, n, fmt, role):
    """LORA_DEBUG_STALL: a warp of one role waits for what never comes.  The bounded wait runs out (a few ms), the other
    warps stop, LORA_DEV_TIMEOUT is set, nothing behind y is written, and the call returns; the next call is exact."""
    g = torch.Generator(device="cuda").manual_seed(T + d)
    (xm, _), (wm, _) = _whole_on_gpu(T, d, fmt, 3, g), _whole_on_gpu(n, d, mx.MXFP4, 2, g)
    y = torch.full((T + 1, n + 8), 99.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    monkeypatch.setenv("LORA_DEBUG_STALL", str(role))
    lora.lora_mx_linear(y[:T, :n], xm, wm, status)
    monkeypatch.delenv("LORA_DEBUG_STALL")
    assert int(status.item()) == lora.DEV_TIMEOUT
    assert (y[T] == 99).all() and (y[:, n:] == 99).all()
    _check_whole(T, d, n, fmt, torch.bfloat16, 8, T)
