"""Microscaled rows on the GPU against the 64-bit oracle: quantise (bit for bit: a block's scale
is a power of two, so scaling is exact and only the rounding to the element remains),
read back (bit for bit: every value is exact in fp32, and in bf16 above its subnormals),
and the root-mean-square norm.

Norm tolerance: fp32 arithmetic.  The sum of d squares, each rounded, in any order is
within d 2^-24 of its value relatively (all terms positive); half of that passes
through the square root, and mean, root, reciprocal and the two products add at
most 6 roundings of 2^-24: h is within (d / 2 + 6) 2^-24 |h|, then one rounding of
eps(dtype) / 2."""
import numpy as np
import pytest
import torch

import lora_adapter_application_b200 as lora
from mx_helpers import as64, from_device, to_device
from oracle import mx

pytestmark = pytest.mark.gpu

FMT = [lora.LORA_MXFP8, lora.LORA_MXFP4]
DTYPES = [torch.bfloat16, torch.float32]
SHAPES = [(1, 1), (1, 32), (1, 4096), (2, 33), (31, 127), (33, 128), (127, 129), (129, 256), (130, 260), (300, 1003),
          (257, 384), (128, 8), (5, 20000)]


def _rows(seed, T, d, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, d, generator=g) * torch.exp(2 * torch.randn(T, d, generator=g))
    x[torch.rand(T, d, generator=g) < 0.1] = 0
    return x.to(dtype)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d", SHAPES)
def test_quantize_is_the_oracles(cuda_lib, T, d, dtype, fmt):
    x = _rows(T * 31 + d, T, d, dtype)
    q = lora.MxTensor(T, d, fmt)
    q.q.fill_(0xA5)
    lora.lora_mx_quantize(q, x.cuda())
    codes, scales = from_device(q)
    rc, rs = mx.quantize(as64(x), fmt)
    np.testing.assert_array_equal(scales, rs)
    np.testing.assert_array_equal(codes, rc)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d", [(2403, 2056), (2370, 2050), (18990, 100), (19000, 136)])
def test_quantize_of_four_rows_a_warp(cuda_lib, T, d, dtype, fmt):
    """Enough rows that a warp takes four of a band: bands of any height, a last group of half its
    columns, NaN blocks in one of the four rows, in several and beside others; rows behind
    the last stay as they were."""
    x = _rows(T + d, T, d, dtype)
    g = torch.Generator().manual_seed(T)
    for value in (float("nan"), float("inf"), -float("inf")):
        x[torch.randint(T, (200,), generator=g), torch.randint(d, (200,), generator=g)] = value
    x[5, 3] = x[37, 4] = x[101, 31] = float("nan")
    x[T - 1, d - 1] = float("inf")
    q = lora.MxTensor(T + 40, d, fmt)
    q.q.fill_(0xA5)
    q.scales.fill_(0x5A)
    lora.lora_mx_quantize(q, x.cuda())
    codes, scales = from_device(q)
    rc, rs = mx.quantize(as64(x), fmt)
    np.testing.assert_array_equal(scales[:T], rs)
    np.testing.assert_array_equal(codes[:T], rc)
    assert (q.q[T:] == 0xA5).all() and (scales[T:] == 0x5A).all()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_edge_values(cuda_lib, dtype, fmt):
    """Ties, saturation, the block's largest at and beside powers of two, zeros of both
    signs, the type's largest and smallest (subnormal) numbers; infinities and NaN
    make their block NaN and no other."""
    info = torch.finfo(dtype)
    rows = []
    for s in [1.0, -1.0, 2.0 ** -100, 2.0 ** 100]:
        t = torch.linspace(0, 8, 257, dtype=torch.float64)[:256] * s
        rows.append(torch.cat([t, t * 0.499999, t * 2 ** -9, torch.tensor([1.0, -1.0] * 128).double() * s]))
    r = torch.zeros(1024, dtype=torch.float64)
    r[0:32] = info.max
    r[32:64] = info.tiny
    r[64:96] = info.tiny * 2.0 ** -7          # subnormal in both types
    r[96] = -0.0
    r[128:160] = torch.tensor([info.max, info.tiny] * 16, dtype=torch.float64)
    r[200], r[300], r[400] = float("inf"), float("nan"), float("-inf")
    r[401:410] = 1.0
    rows.append(r)
    x = torch.stack(rows).to(dtype)
    q = lora.MxTensor(len(rows), 1024, fmt)
    lora.lora_mx_quantize(q, x.cuda())
    codes, scales = from_device(q)
    rc, rs = mx.quantize(as64(x), fmt)
    np.testing.assert_array_equal(scales, rs)
    np.testing.assert_array_equal(codes, rc)
    assert (scales[-1] == 255).sum() == 3
    out = torch.empty(len(rows), 1024, dtype=torch.float32, device="cuda")
    lora.lora_mx_dequantize(out, q)
    np.testing.assert_array_equal(as64(out), mx.values(rc, rs, fmt, 1024))


@pytest.mark.parametrize("fmt", FMT)
def test_dequantize_every_code_and_scale(cuda_lib, fmt):
    """All element codes (NaN among e4m3's) under all 256 scale bytes; fp32 holds each
    product or overflows to infinity where 2^(e-127) x element passes its largest."""
    n = 256 if fmt == mx.MXFP8 else 16
    codes = np.tile(np.arange(n, dtype=np.uint8), 256 * 1024 // n).reshape(256, 1024)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 32, 1)
    m = to_device(codes, scales, fmt, 1024)
    ref = mx.values(codes, scales, fmt, 1024)
    for dtype in DTYPES:
        out = torch.empty(256, 1024, dtype=dtype, device="cuda")
        lora.lora_mx_dequantize(out, m)
        want = torch.from_numpy(ref).to(torch.float32).to(dtype)
        got = out.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(1.0), want.nan_to_num(1.0))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("T,d", SHAPES)
def test_dequantize_shapes(cuda_lib, T, d, fmt):
    x = as64(_rows(T + d, T, d, torch.float32))
    codes, scales = mx.quantize(x, fmt)
    m = to_device(codes, scales, fmt, d)
    wide = torch.full((T, d + 3), 7.0, device="cuda")
    lora.lora_mx_dequantize(wide[:, :d], m)
    np.testing.assert_array_equal(as64(wide[:, :d]), mx.values(codes, scales, fmt, d))
    assert (wide[:, d:] == 7).all()


def test_row_strides_and_rows_left_alone(cuda_lib):
    """Strided and misaligned rows give the packed rows' bytes; rows past T, and the scale
    bytes past the last row, stay as they were."""
    base = _rows(5, 70, 400, torch.bfloat16).cuda()
    for lo in (0, 1, 8):
        x = base[:, lo:lo + 264]
        a, b = lora.MxTensor(70, 264, 1), lora.MxTensor(200, 264, 1)
        lora.lora_mx_quantize(a, x.contiguous())
        b.q.fill_(0x5A), b.scales.fill_(0x77)
        lora.lora_mx_quantize(b, x)
        assert torch.equal(a.q, b.q[:70]) and (b.q[70:] == 0x5A).all()
        at = mx.scale_index(200, 12)
        got = b.scales.cpu().numpy()
        np.testing.assert_array_equal(got[at[:70]], a.scales.cpu().numpy()[mx.scale_index(70, 12)])
        assert (got[at[70:]] == 0x77).all() and (np.delete(got, at[:70].ravel()) == 0x77).all()
    out = torch.full((70, 264), 3.0, device="cuda")
    lora.lora_mx_dequantize(out[:9], a)
    assert (out[9:] == 3).all()


def _norm_ref(x, res, w, eps, dtype):
    r = as64(x)
    if res is not None:
        r = as64((torch.from_numpy(r) + torch.from_numpy(as64(res))).to(dtype))
    return r, mx.rms_norm(r, as64(w)[None], eps)


def _norm_tol(ref, d, dtype):
    return np.abs(ref) * ((d / 2 + 6) * 2.0 ** -24 + torch.finfo(dtype).eps / 2) + 1e-37


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("T,d", [(1, 1), (1, 4096), (3, 64), (40, 1003), (700, 96), (130, 2056), (2, 33000), (1, 40008),
                                 (600, 8192), (650, 33000)])
def test_norm(cuda_lib, T, d, dtype, res):
    g = torch.Generator().manual_seed(T + d)
    x = _rows(T * 7 + d, T, d, dtype)
    r = (3 * torch.randn(T, d, generator=g)).to(dtype) if res else None
    w = torch.randn(d, generator=g).to(dtype)
    rsum, ref = _norm_ref(x, r, w, 1e-5, dtype)
    h = torch.empty(T, d, dtype=dtype, device="cuda")
    s = torch.empty_like(h) if res else None
    lora.lora_rms_norm(h, x.cuda(), w.cuda(), 1e-5, residual=r.cuda() if res else None, residual_out=s)
    assert (np.abs(as64(h) - ref) <= _norm_tol(ref, d, dtype)).all()
    if res:
        np.testing.assert_array_equal(as64(s), rsum)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("T,d", [(1, 4096), (1, 5), (133, 1003), (700, 640), (2, 33000), (600, 4104), (3, 132)])
def test_norm_microscaled_output_is_quantized_h(cuda_lib, T, d, fmt, dtype):
    """q from the norm = lora_mx_quantize of the stored h, whether h is stored or not."""
    x, w = _rows(T + d, T, d, dtype).cuda(), _rows(d, 1, d, dtype).cuda()[0]
    r = _rows(T + d + 1, T, d, dtype).cuda()
    h, s = torch.empty_like(x), torch.empty_like(x)
    a, b, c = (lora.MxTensor(T, d, fmt) for _ in range(3))
    a.q.fill_(0xFF), b.q.fill_(0xFF)
    lora.lora_rms_norm(h, x, w, 1e-6, residual=r, residual_out=s, q=a)
    lora.lora_rms_norm(None, x, w, 1e-6, residual=r, residual_out=s, q=b)
    lora.lora_mx_quantize(c, h)
    assert torch.equal(a.q, c.q) and torch.equal(a.scales, c.scales)
    assert torch.equal(b.q, c.q) and torch.equal(b.scales, c.scales)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("d", [8, 77, 136, 1003, 33008])
def test_norm_microscaled_rows_of_nan(cuda_lib, d, fmt, dtype):
    """Rows whose norm is not finite: every block of the row reads back as NaN where h does, and the
    padding's blocks stay zeros with e = 0."""
    x = torch.ones(3, d, dtype=dtype, device="cuda")
    x[0, d // 2] = float("nan")
    x[1, 0] = float("inf")
    w, h = torch.ones(d, dtype=dtype, device="cuda"), torch.empty_like(x)
    a, b = lora.MxTensor(3, d, fmt), lora.MxTensor(3, d, fmt)
    a.q.fill_(0xFF), a.scales.fill_(0xFF)
    lora.lora_rms_norm(h, x, w, 1e-5, q=a)
    lora.lora_mx_quantize(b, h)
    ca, sa = from_device(a)
    cb, sb = from_device(b)
    np.testing.assert_array_equal(ca, cb)
    np.testing.assert_array_equal(sa, sb)
    assert (sa[0, :-(-d // 32)] == 255).all() and (sa[:, -(-d // 32):] == 0).all() and (ca[:, d:] == 0).all()


@pytest.mark.parametrize("d", [96, 1003, 8192, 33000])
def test_norm_in_place_and_strided(cuda_lib, d):
    T = 20
    base = _rows(d, T, d + 8, torch.bfloat16).cuda()
    x, r = base[:, :d], _rows(d + 1, T, d, torch.bfloat16).cuda()
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    h, s = torch.empty_like(r), torch.empty_like(r)
    lora.lora_rms_norm(h, x.contiguous(), w, 0.0, residual=r, residual_out=s)
    r2 = r.clone()
    keep = base[:, d:].clone()
    lora.lora_rms_norm(x, x, w, 0.0, residual=r2)          # h = x, the sum in place of the residual
    assert torch.equal(x, h) and torch.equal(r2, s) and torch.equal(base[:, d:], keep)
    z = h.clone()
    h2 = torch.empty_like(h)
    lora.lora_rms_norm(h2, h, w, 0.0)
    lora.lora_rms_norm(z, z, w, 0.0)
    assert torch.equal(z, h2)


def test_norm_zero_rows_nan_rows_and_empty(cuda_lib):
    x = torch.ones(4, 64, device="cuda")
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    w, h = torch.ones(64, device="cuda"), torch.empty(4, 64, device="cuda")
    q = lora.MxTensor(4, 64, lora.LORA_MXFP8)
    lora.lora_rms_norm(h, x, w, 1e-5, q=q)
    assert (h[0] - 1).abs().max() < 1e-4 and (h[1] == 0).all() and torch.isnan(h[2]).all()
    assert torch.isnan(h[3, 7]) and (h[3, :7] == 0).all()     # inf / inf; finite / inf
    out = torch.empty(4, 64, device="cuda")
    lora.lora_mx_dequantize(out, q)
    assert torch.isnan(out[2]).all() and (out[1] == 0).all()
    empty = x[:0]
    lora.lora_rms_norm(h[:0], empty, w, 1e-5, q=q)
    lora.lora_mx_quantize(q, empty)
    lora.lora_mx_dequantize(out[:0], q)


@pytest.mark.parametrize("seed", range(6))
def test_random_shapes(cuda_lib, seed):
    """Random sizes, types, strides and formats through all three row operators."""
    r = np.random.default_rng(seed)
    for k in range(12):
        T, d = int(2 ** r.uniform(0, 11)), int(2 ** r.uniform(0, 12))
        if r.random() < 0.3:
            d = max(8, d // 8 * 8)
        dtype, fmt, pad = DTYPES[int(r.integers(2))], int(r.integers(2)), int(r.choice([0, 0, 1, 8]))
        x = _rows(seed * 100 + k, T, d + pad, dtype).cuda()[:, :d]
        q = lora.MxTensor(T, d, fmt)
        lora.lora_mx_quantize(q, x)
        codes, scales = from_device(q)
        rc, rs = mx.quantize(as64(x), fmt)
        np.testing.assert_array_equal(scales, rs)
        np.testing.assert_array_equal(codes, rc)
        out = torch.full((T + 1, d + pad), 5.0, device="cuda")
        lora.lora_mx_dequantize(out[:T, :d], q)
        np.testing.assert_array_equal(as64(out[:T, :d]), mx.values(rc, rs, fmt, d))
        assert (out[T] == 5).all() and (out[:, d:] == 5).all()
        w = torch.randn(d, generator=torch.Generator().manual_seed(k)).to(dtype).cuda()
        res = _rows(seed * 100 + k + 50, T, d, dtype).cuda()
        h, s = torch.full((T + 1, d + pad), 5.0, dtype=dtype, device="cuda"), torch.empty_like(res)
        lora.lora_rms_norm(h[:T, :d], x, w, 1e-6, residual=res, residual_out=s, q=q)
        rsum, ref = _norm_ref(x.cpu(), res.cpu(), w.cpu(), 1e-6, dtype)
        np.testing.assert_array_equal(as64(s), rsum)
        assert (np.abs(as64(h[:T, :d]) - ref) <= _norm_tol(ref, d, dtype)).all()
        assert (h[T] == 5).all() and (h[:, d:] == 5).all()
        codes, scales = from_device(q)
        rc, rs = mx.quantize(as64(h[:T, :d]), fmt)
        np.testing.assert_array_equal(scales, rs)
        np.testing.assert_array_equal(codes, rc)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("T,d", [(2403, 2056), (2370, 2050), (18990, 100), (19000, 136), (18944, 256)])
def test_dequantize_of_four_rows_a_warp(cuda_lib, T, d, pad, dtype, fmt):
    """Enough rows that a warp takes four of a band: bands of any height, a last group of half its columns, rows of out
    with and without 16-byte steps, NaN blocks in one of the four rows and in several; nothing beside out is written."""
    assert -(-mx.padded(d) // 256) * T // 4 >= 148 * 32
    x = as64(_rows(T + d + pad, T, d, torch.float32))
    g = np.random.default_rng(T)
    x[g.integers(0, T, 200), g.integers(0, d, 200)] = np.nan
    x[5, 3] = x[37, 4] = x[101, 31] = x[T - 1, d - 1] = np.inf
    codes, scales = mx.quantize(x, fmt)
    m = to_device(codes, scales, fmt, d)
    out = torch.full((T + 40, d + pad), 7.0, dtype=dtype, device="cuda")
    lora.lora_mx_dequantize(out[:T, :d], m)
    want = torch.from_numpy(mx.values(codes, scales, fmt, d)).to(torch.float32).to(dtype)
    got = out[:T, :d].cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and bool(torch.isnan(want).any())
    assert torch.equal(got.nan_to_num(1.0), want.nan_to_num(1.0))
    assert (out[T:] == 7).all() and (out[:, d:] == 7).all()


# The norm's forms by their rule: registers for 1, 2 or 4 groups of 8 columns a thread, or rows read twice; few rows
# (fewer than four for each of 148 multiprocessors) or many; 16-byte steps or not.  Widths at and beside each border.
NORM_FORMS = [(T, d) for T in (3, 700) for d in (256, 264, 408, 512, 520, 2048, 2049, 2184, 4096, 4104, 4108, 8192, 8200, 8215, 16384,
                                                 16392, 16429, 28672, 32768, 32776, 32783)] + [(591, 408), (592, 408), (591, 8200), (592, 8200)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("T,d", NORM_FORMS)
def test_every_form_of_the_norm(cuda_lib, T, d, dtype, res):
    """h and the sum against 64 bits; the microscaled copies are the quantised h; h is the same with and without them;
    nothing beside the outputs is written."""
    g = torch.Generator(device="cuda").manual_seed(T + d)
    x = (torch.randn(T, d, generator=g, device="cuda") * torch.exp(torch.randn(T, 1, generator=g, device="cuda"))).to(dtype)
    r = (3 * torch.randn(T, d, generator=g, device="cuda")).to(dtype) if res else None
    w = torch.randn(d, generator=g, device="cuda").to(dtype)
    total = (x.double() + r.double()).to(dtype) if res else x
    v = total.double()
    ref = v / (v.square().mean(1, keepdim=True) + 1e-5).sqrt() * w.double()
    h = torch.full((T + 1, d + 8), 9.0, dtype=dtype, device="cuda")
    s = torch.full((T + 1, d + 8), 9.0, dtype=dtype, device="cuda")
    out = {"residual": r, "residual_out": s[:T, :d]} if res else {}
    lora.lora_rms_norm(h[:T, :d], x, w, 1e-5, **out)
    tol = ref.abs() * ((d / 2 + 6) * 2.0 ** -24 + torch.finfo(dtype).eps / 2) + 1e-37
    assert ((h[:T, :d].double() - ref).abs() <= tol).all()
    for t in (h, s):
        assert (t[T] == 9).all() and (t[:, d:] == 9).all()
    assert torch.equal(s[:T, :d], total) if res else (s == 9).all()
    for fmt in FMT:
        a, b = lora.MxTensor(T + 1, d, fmt), lora.MxTensor(T + 1, d, fmt)
        for m in (a, b):
            m.q.fill_(0xA5), m.scales.fill_(0x5A)
        again = torch.empty(T, d, dtype=dtype, device="cuda")
        lora.lora_rms_norm(again, x, w, 1e-5, q=a, **out)
        lora.lora_mx_quantize(b, h[:T, :d])
        assert torch.equal(again, h[:T, :d])
        assert torch.equal(a.q, b.q) and torch.equal(a.scales, b.scales)
        if res:
            assert torch.equal(s[:T, :d], total)


@pytest.mark.parametrize("d", [64, 77, 8200])
def test_norm_of_rows_past_the_range_of_fp32_squares(cuda_lib, d):
    """A finite row whose squares pass fp32's largest number gives zeros (no NaN); one whose squares vanish is scaled by
    1 / sqrt(eps), which the formula gives too (mean r^2 of at most 1e-60 beside eps).  The sums are stored as ever."""
    x = torch.ones(3, d, device="cuda")
    x[0] *= 1e30
    x[1] *= 1e-30
    w, r = torch.full((d,), 2.0, device="cuda"), torch.zeros(3, d, device="cuda")
    h, q = torch.empty_like(x), lora.MxTensor(3, d, lora.LORA_MXFP8)
    lora.lora_rms_norm(h, x, w, 1e-5, residual=r, q=q)
    assert (h[0] == 0).all() and torch.equal(r, x)
    ref = as64(x[1:]) / np.sqrt((as64(x[1:]) ** 2).mean(1, keepdims=True) + 1e-5) * 2
    assert (np.abs(as64(h[1:]) - ref) <= _norm_tol(ref, d, torch.float32)).all()
    out = torch.empty_like(x)
    lora.lora_mx_dequantize(out, q)
    assert (out[0] == 0).all() and not torch.isnan(out).any()
