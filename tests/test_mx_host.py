"""Microscaled base, on the host: the oracle's formats pinned against the published tables,
sizes, and every refusal of the C entry points and of the binding (nothing here
reaches a GPU: pointers are numbers that no call follows)."""
import ctypes

import numpy as np
import pytest
import torch

import lora_adapter_application_b200 as lora
from lora_adapter_application_b200 import LoraError
from oracle import mx

NULL, DTYPE, SHAPE, ALIGN = -1, -2, -3, -5
P = 1 << 20   # a well-aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    from lora_adapter_application_b200 import build
    build.build()
    return lora.load()


# ------------------------------------------------------------------- the oracle
def test_element_tables():
    """OCP MX v1.0: e2m1's eight magnitudes; e4m3 runs from 2^-9 to 448 with 2^-6 its smallest normal
    number, and torch's float8_e4m3fn decodes every code alike."""
    assert mx.table(mx.MXFP4).tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    t = mx.table(mx.MXFP8)
    assert t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and t[-1] == 448 and len(t) == 127
    ref = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(t, ref)


def test_quantize_pins():
    """Worked blocks: largest 5 -> exponent 2, e = 127 + 2 - 2; 2.5 and 5 tie to the even codes; 7.9 saturates."""
    v = np.zeros((1, 64))
    v[0, :4] = [5.0, 2.5, -0.25, 0.75]
    v[0, 32:34] = [7.9, 1.0]
    c, s = mx.quantize(v, mx.MXFP4)
    assert s[0].tolist() == [127, 127, 0, 0]
    assert c[0, :4].tolist() == [6, 4, 8, 2]            # 4, 2, -0, 1
    assert c[0, 32:34].tolist() == [7, 2]
    c, s = mx.quantize(v, mx.MXFP8)
    assert s[0, 0] == 127 + 2 - 8
    got = mx.values(c, s, mx.MXFP8, 64)
    assert got[0, 0] == 5.0 and got[0, 1] == 2.5 and got[0, 32] == 448 / 64.0   # 7.9 * 64 > 448
    v[0, 40] = np.nan
    c, s = mx.quantize(v, mx.MXFP8)
    assert s[0, 1] == 255 and (c[0, 32:64] == 0).all() and s[0, 0] != 255


def test_quantize_agrees_with_torch_casts():
    """Elements against torch's own float8 cast of the scaled values."""
    x = np.random.default_rng(3).standard_normal((20, 256))
    c, s = mx.quantize(x, mx.MXFP8)
    scaled = (x.reshape(20, 8, 32) / 2.0 ** (s.astype(float) - 127)[:, :, None]).clip(-448, 448)
    ref = torch.from_numpy(scaled.reshape(20, 256)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(c, ref)


def test_scale_storage_round_trip():
    s = np.random.default_rng(4).integers(0, 256, (300, 12)).astype(np.uint8)
    flat = mx.pack_scales(s)
    assert flat.size == 3 * 3 * 512
    np.testing.assert_array_equal(mx.unpack_scales(flat, 300, 384), s)
    assert mx.scale_index(256, 12)[[0, 1, 32, 128], [0, 5, 2, 11]].tolist() == [0, 512 + 17, 6, 3 * 512 + 2 * 512 + 3]


# ------------------------------------------------------------------- sizes
def test_sizes(lib):
    for cols in (1, 31, 128, 129, 1003, 4096):
        pad = mx.padded(cols)
        assert lora.lora_mx_row_bytes(lora.LORA_MXFP8, cols) == pad
        assert lora.lora_mx_row_bytes(lora.LORA_MXFP4, cols) == pad // 2
        for rows in (0, 1, 128, 129):
            assert lora.lora_mx_scale_bytes(rows, cols) == -(-rows // 128) * (pad // 128) * 512
    assert lora.lora_mx_scale_bytes(1 << 20, 1 << 20) == (1 << 40) // 32
    for bad in [(2, 8), (-1, 8), (0, 0), (0, (1 << 20) + 1)]:
        assert lora.lora_mx_row_bytes(*bad) == 0
    for bad in [(-1, 8), (1, 0), ((1 << 20) + 1, 8), (1, (1 << 20) + 1)]:
        assert lora.lora_mx_scale_bytes(*bad) == 0


# ------------------------------------------------------------------- C refusals
def _m(**over):
    f = dict(q=P, scales=P, rows=64, cols=256, format=0)
    f.update(over)
    return lora.lora_mx(*[f[k] for k in ("q", "scales", "rows", "cols", "format")])


def _ref(m):
    return ctypes.addressof(m) if m is not None else None


BAD_MATRIX = [(dict(format=2), DTYPE), (dict(format=-1), DTYPE), (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE),
              (dict(rows=(1 << 20) + 1), SHAPE), (dict(cols=(1 << 20) + 1), SHAPE), (dict(rows=3), SHAPE),
              (dict(q=None), NULL), (dict(scales=None), NULL), (dict(q=P + 64), ALIGN), (dict(scales=P + 16), ALIGN)]


@pytest.mark.parametrize("over,want", BAD_MATRIX)
def test_every_call_refuses_a_bad_matrix(lib, over, want):
    m = _m(**over)
    assert lib.lora_mx_quantize(_ref(m), P, 256, 4, 0, None) == want
    assert lib.lora_mx_dequantize(P, 256, _ref(m), 4, 0, None) == want
    assert lib.lora_rms_norm(P, 256, P, 256, None, 0, None, 0, P, 1e-5, 4, 256, _ref(m), 0, None) == want
    assert lib.lora_mx_linear(P, 256, _ref(m), _ref(_m(format=1)), 4, 0, P, None) == want


def test_quantize_and_dequantize_refusals(lib):
    m = _m()
    for fn, a in ((lib.lora_mx_quantize, lambda p, ld, T, dt, q=m: (_ref(q), p, ld, T, dt, None)),
                  (lib.lora_mx_dequantize, lambda p, ld, T, dt, q=m: (p, ld, _ref(q), T, dt, None))):
        assert fn(*a(P, 256, 4, 2)) == DTYPE
        assert fn(*a(P, 256, -1, 0)) == SHAPE
        assert fn(*a(P, 255, 4, 0)) == SHAPE
        assert fn(*a(P, 256, 65, 0)) == SHAPE
        assert fn(*a(None, 256, 4, 0)) == NULL
        assert fn(*a(P, 256, 4, 0, None)) == NULL
        assert fn(*a(None, 256, 0, 0)) == 0             # no rows: nothing to do


def test_norm_refusals(lib):
    ok = dict(h=P, ld_h=256, x=P, ld_x=256, r=None, ld_r=0, ro=None, ld_ro=0, w=P, eps=1e-5, T=4, d=256, q=None, dt=0)

    def call(**over):
        f = dict(ok, **over)
        return lib.lora_rms_norm(f["h"], f["ld_h"], f["x"], f["ld_x"], f["r"], f["ld_r"], f["ro"], f["ld_ro"], f["w"],
                                 f["eps"], f["T"], f["d"], _ref(f["q"]), f["dt"], None)
    assert call(T=0) == 0
    for over, want in [(dict(dt=2), DTYPE), (dict(T=-1), SHAPE), (dict(T=131073), SHAPE), (dict(d=0), SHAPE),
                       (dict(d=(1 << 20) + 1), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
                       (dict(h=None), NULL), (dict(x=None), NULL), (dict(w=None), NULL), (dict(r=P, ld_r=256), NULL),
                       (dict(ro=P, ld_ro=256), NULL), (dict(ld_x=255), SHAPE), (dict(ld_h=255), SHAPE),
                       (dict(r=P, ro=P, ld_r=255, ld_ro=256), SHAPE), (dict(r=P, ro=P, ld_r=256, ld_ro=255), SHAPE),
                       (dict(q=_m(cols=128)), SHAPE), (dict(r=2 * P, ro=P, ld_r=256, ld_ro=256), SHAPE)]:
        assert call(**over) == want, over


def test_linear_refusals(lib):
    x, w = _m(), _m(rows=96, format=1)

    def call(y=P, ld=96, x=x, w=w, T=4, dt=0, status=P):
        return lib.lora_mx_linear(y, ld, _ref(x), _ref(w), T, dt, status, None)
    assert call(T=0) == 0
    assert call(dt=7) == DTYPE
    assert call(w=_m(rows=96)) == DTYPE                 # w in MXFP8
    assert call(T=-1) == call(T=65) == call(T=131073) == call(ld=95) == SHAPE
    assert call(w=_m(rows=96, cols=128, format=1)) == call(w=_m(rows=0, format=1)) == SHAPE
    assert call(status=None) == call(y=None) == call(x=None) == call(w=None) == NULL
    assert call(w=_m(rows=96, format=1, q=P + 1)) == ALIGN


# ------------------------------------------------------------------- binding refusals
def test_mxtensor_checks(lib):
    m = lora.MxTensor(5, 300, lora.LORA_MXFP4, device="cpu")
    assert m.q.shape == (5, 192) and m.scales.numel() == 3 * 512 and int(m.q.sum()) == 0
    for a, k in [((5, 300, 2), {}), ((-1, 300, 0), {}), ((5, 0, 0), {}), (((1 << 20) + 1, 8, 0), {}),
                 ((5, 300, 0), dict(q=torch.zeros(5, 300, dtype=torch.uint8))),
                 ((5, 300, 0), dict(q=torch.zeros(5, 384))),
                 ((5, 300, 0), dict(q=torch.zeros(384, 5, dtype=torch.uint8).t())),
                 ((5, 300, 0), dict(scales=torch.zeros(10, dtype=torch.uint8)))]:
        with pytest.raises(LoraError):
            lora.MxTensor(*a, **{"device": "cpu", **k})


def test_binding_refuses_cpu_and_mismatched_operands(lib):
    m = lora.MxTensor(5, 64, 0, device="cpu")
    x, st = torch.zeros(5, 64), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(LoraError, match="CUDA"):
        lora.lora_mx_quantize(m, x)
    with pytest.raises(LoraError, match="CUDA"):
        lora.lora_mx_dequantize(x, m)
    with pytest.raises(LoraError, match="CUDA"):
        lora.lora_mx_linear(x, m, m, st)
    with pytest.raises(LoraError, match="CUDA"):
        lora.lora_rms_norm(x, x, x[0], 1e-5)
    with pytest.raises(LoraError, match="MxTensor"):
        lora.lora_mx_quantize(x, x)
    with pytest.raises(LoraError, match="2-D"):
        lora.lora_rms_norm(x, x.t(), x[0], 1e-5)
    with pytest.raises(LoraError, match="overlap"):
        lora.lora_rms_norm(x, x[:1].expand(5, 64), x[0], 1e-5)


def test_mxtensor_is_its_memory(lib):
    """The C struct holds the addresses of construction: fields cannot be replaced, and a tensor that
    was given other memory in place (the old may belong to someone else by then) is refused by every call."""
    m = lora.MxTensor(5, 300, lora.LORA_MXFP4, device="cpu")
    for name, value in [("q", torch.zeros_like(m.q)), ("scales", torch.zeros_like(m.scales)), ("rows", 9), ("cols", 128),
                        ("fmt", lora.LORA_MXFP8), ("device", "cuda"), ("index", 0)]:
        with pytest.raises(LoraError, match="fixed"):
            setattr(m, name, value)
    x, h, st = torch.zeros(5, 300), torch.zeros(5, 300), torch.zeros(1, dtype=torch.int32)
    ok = lora.MxTensor(5, 300, lora.LORA_MXFP4, device="cpu")
    for change in (lambda q: q.q.resize_(4000, 192), lambda q: q.scales.set_(torch.zeros(4096, dtype=torch.uint8)),
                   lambda q: q.q.set_(), lambda q: setattr(q.scales, "data", q.scales.clone()),
                   lambda q: q.q.untyped_storage().resize_(0)):
        m = lora.MxTensor(5, 300, lora.LORA_MXFP4, device="cpu")
        change(m)
        for call in (lambda: lora.lora_mx_quantize(m, x), lambda: lora.lora_mx_dequantize(x, m),
                     lambda: lora.lora_mx_linear(torch.zeros(5, 5), m, ok, st),
                     lambda: lora.lora_mx_linear(torch.zeros(5, 5), ok, m, st)):
            with pytest.raises(LoraError, match="memory|CUDA"):
                call()
        with pytest.raises(LoraError, match="memory"):
            lora.lora_mx_quantize(m, x)
        with pytest.raises(LoraError, match="memory"):
            lora._mx(m, "q")


def test_sizes_past_32_bits_are_refused(lib):
    """ctypes would pass them modulo 2^32: a matrix of 2^32 + 64 columns as one of 64, the norm of such a row
    over its first 64."""
    big = 1 << 32
    for fmt, cols in [(0, big + 64), (1, big + 64), (0, 64 - big), (big, 64)]:
        assert lora.lora_mx_row_bytes(fmt, cols) == 0
    for rows, cols in [(big + 1, 64), (1 - big, 64), (1, big + 64)]:
        assert lora.lora_mx_scale_bytes(rows, cols) == 0
    for a in [(2, big + 64, 0), (big + 2, 64, 0), (2, 64, big)]:
        with pytest.raises(LoraError, match="at most"):
            lora.MxTensor(*a, q=torch.zeros(2, 128, dtype=torch.uint8), scales=torch.zeros(512, dtype=torch.uint8))
    for T, d in [(1, big + 64), (big + 1, 64), (131073, 8), (1, (1 << 20) + 1)]:
        x, w = torch.empty(T, d, dtype=torch.bfloat16, device="meta"), torch.empty(d, dtype=torch.bfloat16, device="meta")
        with pytest.raises(LoraError, match="at most"):
            lora.lora_rms_norm(torch.empty_like(x), x, w, 1e-5)


def test_tensor_memory_is_fenced_after_every_wait():
    """The order that no run can be relied on to show wrong: between a wait on another warp's barrier and the first
    tensor-memory access behind it (store of scales, load of sums, MMAs) stands tcgen05.fence::after_thread_sync."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(lora.__file__), "csrc", "mx_linear.cu")).read()
    src = src[src.index("mx_linear_few_kernel(const"):]
    waits = [m.start() for m in re.finditer(r"wait(<\w+>)?\((sf_full|full|acc_full|acc_empty)\b", src)]
    uses = [m.start() for m in re.finditer(r"\b(tmem_st4|tc_ld16|tc_ld32|mx_stage_mmas<)", src)]
    assert len(waits) >= 8 and len(uses) >= 8
    for u in uses:
        last = max((w for w in waits if w < u), default=None)
        assert last is None or "tc_fence_after();" in src[last:u], src[last:u]


def test_mxtensor_copies(lib):
    """copy.copy shares the tensors, deepcopy and pickle carry their contents; each has its own struct and addresses."""
    import copy
    import pickle
    m = lora.MxTensor(5, 300, lora.LORA_MXFP4, device="cpu")
    m.q.fill_(7)
    for c, shared in ((copy.copy(m), True), (copy.deepcopy(m), False), (pickle.loads(pickle.dumps(m)), False)):
        assert (c.rows, c.cols, c.fmt) == (5, 300, lora.LORA_MXFP4) and torch.equal(c.q, m.q)
        assert (c.q.data_ptr() == m.q.data_ptr()) == shared and c.ref != m.ref
        assert (c.c.q, c.c.scales) == (c.q.data_ptr(), c.scales.data_ptr())
