"""lora_linear against the formula in 64 bits: sizes at and beside the tiles' borders, each
operand of the epilogue, each activation, both types, strides and alignments (tolerances: dense_helpers)."""
import math

import pytest
import torch

import lora_adapter_application_b200 as lora
from dense_helpers import ACTS, assert_close, assert_frame, dense64, nan_frame, whole

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


def _operands(seed, T, d, n, dtype, gated, bias, addend, residual):
    """Whole operands, fp64 and in dtype; rows far past the tile's borders differ from their neighbours."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n_w = 2 * n if gated else n
    # z within about +-8, so that activations are in the range where they bend
    o = {"x": whole(g, (T, d), 2), "w": whole(g, (n_w, d), 2, 0.25 if d <= 64 else 2.0 ** -round(math.log2(d) / 2))}
    o["bias"] = whole(g, (n_w,), 8, 0.25) if bias else None
    o["addend"] = whole(g, (T, n_w), 8, 0.25) if addend else None
    o["residual"] = whole(g, (T, n), 64, 0.5) if residual else None
    return o, {k: None if v is None else v.to(dtype) for k, v in o.items()}


def _run(o, n, gated, act=lora.ACT_NONE, y=None, **kw):
    T, dtype = o["x"].shape[0], o["x"].dtype
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    buf = None
    if y is None:
        buf, y = nan_frame((T, n), dtype)
    lora.lora_linear(y, o["x"], o["w"], status, bias=o["bias"], addend=o["addend"], residual=o["residual"], act=act,
                     gated=gated, **kw)
    assert int(status.item()) == 0
    if buf is not None:
        assert_frame(buf, (T, n))
    return y


def _check(seed, T, d, n, dtype, gated=False, act=lora.ACT_NONE, bias=False, addend=False, residual=False):
    o64, o = _operands(seed, T, d, n, dtype, gated, bias, addend, residual)
    want, tol = dense64(**o64, act=act, gated=gated, dtype=dtype)
    assert_close(_run(o, n, gated, act), want, tol, f"T={T} d={d} n={n}")


SHAPES = [(1, 1, 1), (1, 8, 8), (1, 64, 128), (1, 4096, 4096), (2, 72, 136), (3, 1000, 264), (7, 1003, 333), (8, 128, 1024),
          (9, 256, 40), (15, 512, 120), (16, 64, 128), (17, 72, 129), (31, 448, 2056), (32, 2048, 256), (33, 512, 130),
          (63, 4096, 384), (64, 2048, 1024), (65, 640, 257), (100, 14336, 256), (127, 200, 136), (128, 1024, 512),
          (129, 4096, 128), (144, 320, 648), (160, 512, 3000), (176, 640, 8), (191, 128, 264), (192, 256, 256),
          (193, 128, 128), (224, 4096, 4096), (240, 72, 4104), (255, 264, 264), (256, 256, 256), (257, 1408, 384),
          (300, 264, 520), (384, 1024, 2048), (500, 3000, 704), (512, 64, 64), (513, 8, 8), (1000, 1152, 1000),
          (1024, 512, 2304), (2049, 128, 40), (4096, 256, 512), (5000, 304, 3000), (8192, 64, 264),
          (40, 4097, 1001), (300, 1003, 520), (520, 65, 257), (1030, 777, 1001), (2100, 129, 4099), (260, 8191, 129)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,n", SHAPES)
def test_shapes(cuda_lib, T, d, n, dtype, gated):
    _check(T + d + n, T, d, n, dtype, gated)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,n", [(1, 4096, 520), (33, 512, 136), (300, 264, 264), (70, 37, 43), (1500, 128, 2560)])
def test_epilogue(cuda_lib, T, d, n, dtype, gated, act):
    _check(T * 7 + act, T, d, n, dtype, gated, act, bias=True, addend=True, residual=True)


@pytest.mark.parametrize("which", ["bias", "addend", "residual"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,n", [(5, 2048, 384), (260, 512, 520)])
def test_one_operand(cuda_lib, T, d, n, dtype, gated, which):
    _check(11, T, d, n, dtype, gated, lora.ACT_SILU, **{which: True})


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,n", [(1, 4096, 4096), (64, 4096, 1024), (257, 2048, 1032), (1024, 1024, 1024), (90, 333, 70)])
def test_random_values(cuda_lib, T, d, n, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    x, w = torch.randn(T, d, generator=g, device="cuda").to(dtype), torch.randn(n, d, generator=g, device="cuda").to(dtype)
    dz = d * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T)
    want, tol = dense64(x.double(), w.double(), dtype=dtype, dz=dz)
    y = _run({"x": x, "w": w, "bias": None, "addend": None, "residual": None}, n, False)
    assert_close(y, want, tol)
    # over a whole matrix the errors are spread: their norm is within the rounding's own
    unit = torch.finfo(dtype).eps / 2 if dtype == torch.bfloat16 else 2.0 ** -24 * math.sqrt(d)
    assert (y.double() - want).norm() <= unit * want.norm()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,n", [(1, 512, 264), (40, 512, 264), (300, 512, 264), (2500, 512, 2056), (40, 333, 257), (700, 333, 600)])
def test_in_place(cuda_lib, T, d, n, dtype):
    """y over the residual, over the addend; a gated y over the residual."""
    o64, o = _operands(5, T, d, n, dtype, False, True, True, True)
    want, tol = dense64(**o64, act=lora.ACT_GELU, dtype=dtype)
    for name in ("residual", "addend"):
        y = o[name].clone()
        assert_close(_run({**o, name: y}, n, False, lora.ACT_GELU, y=y), want, tol, name)
    o64, o = _operands(6, T, d, n, dtype, True, False, True, True)
    want, tol = dense64(**o64, act=lora.ACT_SILU, gated=True, dtype=dtype)
    y = o["residual"].clone()
    assert_close(_run({**o, "residual": y}, n, True, lora.ACT_SILU, y=y), want, tol, "gated")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,d,n", [(3, 256, 136), (50, 512, 264), (400, 256, 264)])
def test_strides_and_alignment(cuda_lib, T, d, n, gated, dtype):
    """Rows with gaps (of NaN), in steps of 16 bytes and off them, at addresses off 16 bytes."""
    o64, o = _operands(9, T, d, n, dtype, gated, True, True, True)
    want, tol = dense64(**o64, act=lora.ACT_SILU, gated=gated, dtype=dtype)

    def spread(t, pad, off):
        buf = torch.full((t.shape[0], t.shape[1] + pad + off), math.nan, dtype=dtype, device="cuda")
        v = buf[:, off:off + t.shape[1]]
        v.copy_(t)
        return v
    for pad, off in [(64, 0), (56, 8), (3, 0), (8, 1), (0, 0)]:
        s = {k: v if k == "bias" else spread(v, pad, off) for k, v in o.items()}
        assert_close(_run(s, n, gated, lora.ACT_SILU), want, tol, f"pad {pad} off {off}")
    # one operand off at a time: each alone takes the call off the tensor cores or off wide accesses
    for name in ("x", "w", "addend", "residual"):
        assert_close(_run({**o, name: spread(o[name], 7, 1)}, n, gated, lora.ACT_SILU), want, tol, name)
    ybuf = torch.full((T, n + 3), 7.0, dtype=dtype, device="cuda")
    assert_close(_run(o, n, gated, lora.ACT_SILU, y=ybuf[:, 1:n + 1]), want, tol, "y")
    assert (ybuf[:, 0] == 7).all() and (ybuf[:, n + 1:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [2, 300])
def test_infinities_and_nan_stay_in_their_rows(cuda_lib, T, dtype):
    o64, o = _operands(3, T, 200, 264, dtype, False, False, False, False)
    clean = _run(o, 264, False).clone()
    o["x"][1, 3] = math.nan
    o["w"][17, 199] = math.inf
    y = _run(o, 264, False)
    rows = [i for i in range(T) if i != 1]
    cols = [c for c in range(264) if c != 17]
    assert torch.isnan(y[1]).all()
    assert torch.equal(y[rows][:, cols], clean[rows][:, cols])
    assert not torch.isfinite(y[:, 17]).any()


@pytest.mark.parametrize("act", [lora.ACT_SILU, lora.ACT_GELU, lora.ACT_GELU_TANH])
@pytest.mark.parametrize("dtype", DTYPES)
def test_activations_far_out(cuda_lib, dtype, act):
    """z from the bias alone: large of either sign, 0, -0, where e^-z passes fp32's range."""
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20, -20, -60, -87, 88, -104, 200, -200, 3e4, -3e4, 1e30, -1e30], dtype=dtype)
    x, w = torch.zeros(3, 16, dtype=dtype, device="cuda"), torch.zeros(16, 16, dtype=dtype, device="cuda")
    y = _run({"x": x, "w": w, "bias": z.cuda(), "addend": None, "residual": None}, 16, False, act)
    big = z.double().clamp(-1e3, 1e3)   # beyond, the value is z or 0
    want = torch.where(z.double() > 1e3, z.double(), torch.where(z.double() < -1e3, torch.zeros(16, dtype=torch.float64), act_of(big, act)))
    u = z.double().abs().clamp(max=104)
    tol = want.abs() * (torch.finfo(dtype).eps / 2 + (9 + 4 * u + u * u) * 2.0 ** -23) + 2.0 ** -120
    for row in y.cpu():
        assert_close(row, want, tol)
    ends = torch.tensor([math.inf, -math.inf, math.nan, 0] * 4, dtype=dtype)
    y = _run({"x": x, "w": w, "bias": ends.cuda(), "addend": None, "residual": None}, 16, False, act).cpu()
    assert (y[:, 0::4] == math.inf).all() and torch.isnan(y[:, 1::4]).all() and torch.isnan(y[:, 2::4]).all() and (y[:, 3::4] == 0).all()


@pytest.mark.parametrize("act", [lora.ACT_SILU, lora.ACT_GELU, lora.ACT_GELU_TANH])
def test_activations_of_every_bf16(cuda_lib, act):
    """All finite bf16 z in [-14, 60], from the bias."""
    z = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    z = z[torch.isfinite(z) & (z >= -14) & (z <= 60)]
    n = z.numel() // 8 * 8
    z = z[:n].cuda()
    x, w = torch.zeros(2, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda")
    y = _run({"x": x, "w": w, "bias": z, "addend": None, "residual": None}, n, False, act)
    want, tol = dense64(x.double(), w.double(), bias=z.double(), act=act)
    assert_close(y, want, tol)


def act_of(z, act):
    from dense_helpers import act64
    return act64(z, act)[0]


def test_zero_rows(cuda_lib):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, x = torch.empty(0, 8, device="cuda"), torch.empty(0, 16, device="cuda")
    lora.lora_linear(y, x, torch.empty(8, 16, device="cuda"), status)


def test_rows_of_a_batch_do_not_depend_on_it(cuda_lib):
    """A run repeated gives the same bits."""
    _, o = _operands(1, 200, 4096, 1024, torch.bfloat16, True, False, True, False)
    o["x"] = torch.randn_like(o["x"])
    first = _run(o, 1024, True, lora.ACT_SILU).clone()
    for _ in range(3):
        assert torch.equal(_run(o, 1024, True, lora.ACT_SILU), first)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 64, 300])
def test_captured_first_call_and_two_streams(cuda_lib, T, dtype):
    o64, o = _operands(2, T, 1024, 520, dtype, True, True, True, True)
    want, tol = dense64(**o64, act=lora.ACT_SILU, gated=True, dtype=dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.zeros(T, 520, dtype=dtype, device="cuda")
    kw = dict(bias=o["bias"], addend=o["addend"], residual=o["residual"], act=lora.ACT_SILU, gated=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lora.lora_linear(y, o["x"], o["w"], status, **kw)
        lora.lora_linear(y, o["x"], o["w"], status, **kw)
    for _ in range(2):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert_close(y, want, tol)
    ys = [torch.zeros_like(y) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, yy in zip(streams, ys):
            lora.lora_linear(yy, o["x"], o["w"], status, stream=s, **kw)
    torch.cuda.synchronize()
    for yy in ys:
        assert_close(yy, want, tol)
    assert int(status.item()) == 0


def test_largest_row_count(cuda_lib):
    """LORA_MAX_ROWS rows; offsets past 2^31 bytes in y."""
    T, d, n = lora.MAX_ROWS, 16, 16400
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = whole(g, (T, d), 2).to(torch.bfloat16), whole(g, (n, d), 2).to(torch.bfloat16)
    y = torch.empty(T, n, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lora.lora_linear(y, x, w, status)
    for lo in range(0, T, 16384):
        want = (x[lo:lo + 16384].float() @ w.float().T).to(torch.bfloat16)   # whole numbers up to 64: exact
        assert torch.equal(y[lo:lo + 16384], want)
    assert int(status.item()) == 0


def test_delta_ahead_of_the_activation(cuda_lib):
    """The run it is for: the adapters' delta of gate and up as the addend, the norm in front, the down projection with its
    delta into the residual stream."""
    import numpy as np
    import oracle
    T, d, f, N, r = 96, 256, 384, 5, 16
    g = torch.Generator().manual_seed(4)
    h = torch.randn(T, d, generator=g)
    res = torch.randn(T, d, generator=g).bfloat16()
    ids = torch.randint(-1, N, (T,), generator=g, dtype=torch.int32)
    Wgu, Wd = (torch.randn(2 * f, d, generator=g) / d ** 0.5).bfloat16(), (torch.randn(d, f, generator=g) / f ** 0.5).bfloat16()
    A = [(torch.randn(N, r, d, generator=g) / d ** 0.5).bfloat16() for _ in range(2)]
    B = [(torch.randn(N, f, r, generator=g) / r ** 0.5).bfloat16() for _ in range(2)]
    Ad, Bd = (torch.randn(N, r, f, generator=g) / f ** 0.5).bfloat16(), (torch.randn(N, d, r, generator=g) / r ** 0.5).bfloat16()
    ranks, alpha = torch.full((N,), r, dtype=torch.int32), 16.0
    c = lambda t: t.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    meta = lora.Meta(T, N, 16, 0)
    lora.lora_build_segments(c(ids), meta, status)
    x = c(h.bfloat16())
    alphas = lora.alphas_full(alpha, N)
    delta = torch.zeros(T, 2 * f, dtype=torch.bfloat16, device="cuda")
    lora.lora_add_linear(delta, x, [c(a) for a in A], [c(b) for b in B], [0, f], c(ranks), alphas, meta, status)
    u = torch.empty(T, f, dtype=torch.bfloat16, device="cuda")
    lora.lora_linear(u, x, c(Wgu), status, addend=delta, act=lora.ACT_SILU, gated=True)
    y = c(res.clone())
    lora.lora_linear(y, u, c(Wd), status, residual=y)
    lora.lora_add_linear(y, u, [c(Ad)], [c(Bd)], [0], c(ranks), alphas, meta, status)
    assert int(status.item()) == 0
    zero = torch.zeros(T, 2 * f, dtype=torch.bfloat16)
    d64 = oracle.lora_apply(h.bfloat16(), A, B, [0, f], ranks, alpha, ids, zero)
    z = h.bfloat16().double() @ Wgu.double().T + torch.from_numpy(np.asarray(d64))
    u64 = z[:, :f] * torch.sigmoid(z[:, :f]) * z[:, f:]
    # u: delta rounded to bf16 and the oracle's own tolerance (1e-2 of max(1, |delta|)), through slopes of at most 1.1 and |z|
    y64 = res.double() + u64 @ Wd.double().T
    y64 = torch.from_numpy(np.asarray(oracle.lora_apply(u64.bfloat16(), [Ad], [Bd], [0], ranks, alpha, ids,
                                                        torch.zeros(T, d, dtype=torch.bfloat16)))) + y64
    # norms: each rounding to bf16 (delta, u, y twice, the oracle's u) is off by 2^-9 on average at most of what it rounds
    scale = y64.norm() + res.double().norm()
    assert (y.cpu().double() - y64).norm() <= 6 * 2.0 ** -8 * scale


def test_widest(cuda_lib):
    """LORA_MX_MAX rows of W, both types and the gate's halves of them."""
    for dtype in DTYPES:
        for gated in (False, True):
            n = lora.MX_MAX // (2 if gated else 1)
            x = torch.tensor([[1.0] * 8, [2.0] * 8], dtype=dtype, device="cuda")
            w = (torch.arange(lora.MX_MAX, device="cuda") % 7).to(dtype)[:, None].expand(-1, 8).contiguous()
            y = _run({"x": x, "w": w, "bias": None, "addend": None, "residual": None}, n, gated)
            z = 8 * (torch.arange(lora.MX_MAX, device="cuda") % 7).double()
            want = z[:n] * z[n:] if gated else z
            assert torch.equal(y[0], want.to(dtype)) and torch.equal(y[1], ((4 if gated else 2) * want).to(dtype))


# a few rows (k split over pairs), row tiles, many tiles a pair; rows off 16-byte steps have other roles
STALLS = [(s, r) for s in [(1, 4096, 4096), (40, 4096, 1024), (257, 2048, 520), (3000, 512, 4104)] for r in (1, 3, 4, 5)] + \
    [(s, r) for s in [(70, 1001, 300), (2000, 333, 3000)] for r in (1, 2, 4)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("shape,role", STALLS)
def test_stalled_warp_times_out_and_the_context_survives(cuda_lib, monkeypatch, shape, gated, role):
    """LORA_DEBUG_STALL: a warp of one role waits for what never comes.  The bounded wait runs out (a few ms), the other
    warps stop, LORA_DEV_TIMEOUT is set, nothing beside y is written, and the call returns; the next call is exact."""
    T, d, n = shape
    _, o = _operands(T, T, d, n, torch.bfloat16, gated, False, True, False)
    y = torch.full((T + 1, n + 8), 99.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    monkeypatch.setenv("LORA_DEBUG_STALL", str(role))
    lora.lora_linear(y[:T, :n], o["x"], o["w"], status, addend=o["addend"], gated=gated)
    monkeypatch.delenv("LORA_DEBUG_STALL")
    assert int(status.item()) == lora.DEV_TIMEOUT
    assert (y[T] == 99).all() and (y[:, n:] == 99).all()
    _check(T, T, d, n, torch.bfloat16, gated, addend=True)
