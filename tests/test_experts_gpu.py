"""The block of experts against its formulas in 64 bits: the choice (ids equal, weights to fp32's roundings), the products of
ragged groups, the sum, and a run of them together (tolerances of the products: dense_helpers)."""
import math

import pytest
import torch

import lora_adapter_application_b200 as lora
from dense_helpers import ACTS, assert_close, assert_frame, dense64, nan_frame, whole

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------ route
def _route(logits, k, score, renorm, scale):
    T = logits.shape[0]
    ids = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), math.nan, device="cuda")
    lora.lora_expert_route(ids, w, logits, score=score, renormalize=renorm, scale=scale)
    return ids.cpu(), w.cpu()


def _route64(logits, k, score, renorm, scale):
    x = logits.double().cpu()
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    order = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = order.values[:, :k], order.indices[:, :k].int()
    gone = top == -math.inf
    m = x.max(1, keepdim=True).values
    e = lambda v: torch.where(v == m, torch.ones_like(v), torch.exp(v - m)).masked_fill(v == -math.inf, 0)
    if score == lora.SCORE_SOFTMAX:
        w = e(top) / e(x).sum(1, keepdim=True)
    elif renorm:   # over e^min(m, 0): the ratios are the same
        low = torch.clamp(top, max=0) - torch.clamp(m, max=0)
        w = torch.exp(low.masked_fill(gone, 0)) / (1 + torch.exp(-top.abs()))
    else:
        w = torch.sigmoid(top)
    w = w.masked_fill(gone, 0)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    return ids.masked_fill(gone, -1), (w * scale).masked_fill(gone, 0)


def _route_check(logits, k, score, renorm, scale=1.0):
    ids, w = _route(logits, k, score, renorm, scale)
    ids64, w64 = _route64(logits, k, score, renorm, scale)
    assert torch.equal(ids, ids64)
    # expf 2 units of 2^-23 and its argument's rounding, which it multiplies by the argument (at most 104 in a weight that
    # fp32 holds), a sum of up to 1024 terms in at most 37 steps, quotient and product: (50 + 104) 2^-23
    assert_close(w, w64, w64.abs() * 154 * 2.0 ** -23 + 2.0 ** -120)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", [lora.SCORE_SOFTMAX, lora.SCORE_SIGMOID])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n,k", [(1, 1, 1), (1, 64, 8), (3, 2, 2), (5, 31, 31), (7, 32, 32), (9, 33, 1), (100, 64, 6), (33, 65, 8),
                                   (64, 128, 8), (17, 129, 4), (1000, 256, 8), (13, 257, 3), (8, 512, 10), (5, 513, 32),
                                   (6, 1000, 5), (4, 1024, 32)])
def test_route(cuda_lib, T, n, k, dtype, score, renorm):
    g = torch.Generator(device="cuda").manual_seed(T * n + k)
    _route_check((3 * torch.randn(T, n, generator=g, device="cuda")).to(dtype), k, score, renorm, 2.5)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", [lora.SCORE_SOFTMAX, lora.SCORE_SIGMOID])
@pytest.mark.parametrize("dtype", DTYPES)
def test_route_ties_masks_and_ends(cuda_lib, dtype, score, renorm):
    n = 40
    low = torch.finfo(dtype).min
    rows = torch.zeros(12, n)
    rows[1] = torch.arange(n) % 3                    # ties in groups
    rows[2] = -math.inf                              # nothing is open
    rows[3] = math.nan
    rows[4] = -math.inf
    rows[4, [7, 39]] = torch.tensor([1.0, 1.0])      # two of eight
    rows[5] = low                                    # the type's lowest value is a logit like others
    rows[5, 20] = 0
    rows[6] = low
    rows[7, 9], rows[7, 3], rows[7, 5] = math.inf, math.inf, math.nan
    rows[8] = torch.where(torch.arange(n) % 2 == 0, 0.0, -0.0)   # the two zeros tie
    rows[9] = -200 - torch.arange(n).float()         # sigmoids that fp32 does not hold
    rows[10] = 1e30
    rows[10, 11] = 2e30
    rows[11] = torch.linspace(-90, 90, n)
    for k in (1, 8, 32):
        _route_check(rows.to(dtype).cuda(), k, score, renorm)


def test_route_strided_rows(cuda_lib):
    buf = torch.full((9, 50), math.inf, device="cuda")
    buf[:, 3:40] = torch.randn(9, 37, device="cuda")
    _route_check(buf[:, 3:40], 4, lora.SCORE_SOFTMAX, True)
    ids, w = _route(torch.empty(0, 8, device="cuda"), 2, 0, True, 1.0)
    assert ids.shape == (0, 2)


# ------------------------------------------------------------------------ products
def _meta(ids, N, **kw):
    meta = lora.Meta(ids.numel(), N, **kw)
    st = _status()
    lora.lora_build_segments(ids.cuda(), meta, st)
    return meta


def _group_ids(kind, slots, N, g):
    """Ids of a grouping's kinds: spread, one expert alone, a skewed few, some slots left out, none at all."""
    if kind == "spread":
        return torch.randint(0, N, (slots,), generator=g, dtype=torch.int32)
    if kind == "one":
        return torch.full((slots,), N - 1, dtype=torch.int32)
    if kind == "skewed":
        return (torch.rand(slots, generator=g) ** 4 * N).int().clamp(max=N - 1)
    if kind == "out":
        return torch.randint(-1, N, (slots,), generator=g, dtype=torch.int32) * (torch.rand(slots, generator=g) < 0.7).int() - \
            (torch.rand(slots, generator=g) < 0.1).int()
    return torch.full((slots,), -1, dtype=torch.int32)


def _experts_check(seed, slots, N, d, n, dtype, kind="spread", x_div=1, gated=False, act=lora.ACT_NONE, extras=False, pad=8):
    g = torch.Generator().manual_seed(seed)
    gc = torch.Generator(device="cuda").manual_seed(seed)
    ids = _group_ids(kind, slots, N, g).clamp(min=-1)
    n_w = 2 * n if gated else n
    rows = -(-slots // x_div)
    x, w = whole(gc, (rows, d), 2), whole(gc, (N, n_w, d), 2, 0.25 if d <= 64 else 2.0 ** -round(math.log2(d) / 2))
    bias, addend, res = (whole(gc, (N, n_w), 8, 0.25), whole(gc, (slots, n_w), 8, 0.25), whole(gc, (slots, n), 64, 0.5)) \
        if extras else (None, None, None)
    dev = lambda t: None if t is None else t.to(dtype)
    buf, y = nan_frame((slots, n), dtype, pad)
    y.copy_(torch.full((slots, n), 7.0))
    meta, st = _meta(ids, N), _status()
    lora.lora_expert_linear(y, dev(x), dev(w), meta, st, x_div=x_div, bias=dev(bias), addend=dev(addend), residual=dev(res),
                            act=act, gated=gated)
    assert int(st.item()) == 0
    assert_frame(buf, (slots, n))
    for e in range(-1, N):
        mine = (ids == e).nonzero()[:, 0].cuda()
        if mine.numel() == 0:
            continue
        if e < 0:
            assert (y[mine] == 7).all()
            continue
        want, tol = dense64(x[mine // x_div], w[e], None if bias is None else bias[e], None if addend is None else addend[mine],
                            None if res is None else res[mine], act, gated, dtype)
        assert_close(y[mine], want, tol, f"expert {e}")


SHAPES = [(1, 1, 8, 8), (1, 8, 64, 128), (2, 3, 72, 136), (16, 8, 4096, 512), (33, 4, 256, 264), (64, 64, 128, 128), (100, 7, 200, 40),
          (128, 2, 1024, 256), (200, 1, 512, 384), (257, 3, 264, 520), (300, 5, 1003, 77), (512, 128, 256, 136),
          (1000, 16, 128, 1000), (777, 1024, 64, 24), (2000, 8, 512, 512), (4096, 64, 264, 128), (3001, 2, 72, 2056), (2000, 9, 333, 257),
          (1200, 2, 1001, 600), (50, 6, 2047, 130)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("slots,N,d,n", SHAPES)
def test_experts_shapes(cuda_lib, slots, N, d, n, dtype, gated):
    _experts_check(slots + N, slots, N, d, n, dtype, "spread" if slots % 2 else "skewed", gated=gated)


@pytest.mark.parametrize("kind", ["spread", "one", "skewed", "out", "none"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("slots,N,x_div", [(30, 6, 1), (31, 6, 2), (512, 6, 4), (1500, 40, 5), (2400, 3, 8), (64, 1000, 32)])
def test_experts_groups(cuda_lib, slots, N, x_div, kind, dtype):
    _experts_check(slots * 3 + x_div, slots, N, 136, 264, dtype, kind, x_div, gated=slots % 4 == 0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("slots,N,d,n", [(40, 9, 256, 136), (700, 3, 256, 264), (70, 3, 37, 43)])
def test_experts_epilogue(cuda_lib, slots, N, d, n, dtype, gated, act):
    _experts_check(slots + act, slots, N, d, n, dtype, "out", 2, gated, act, extras=True)


@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("dtype", DTYPES)
def test_experts_strided_y(cuda_lib, dtype, pad):
    _experts_check(pad, 300, 4, 256, 136, dtype, "out", pad=pad)


def test_experts_one_row_for_all(cuda_lib):
    """x_div as large as it may be: every slot reads row 0."""
    _experts_check(1, 50, 4, 128, 64, torch.bfloat16, x_div=lora.MAX_ROWS)


def test_experts_nan_rows_stay_their_own(cuda_lib):
    """A slot whose row holds NaN changes no other slot, of its expert or another; rows of x that no slot reads may hold
    anything; so may another expert's weight."""
    g = torch.Generator(device="cuda").manual_seed(5)
    slots, N, d, n = 300, 4, 192, 264
    ids = (torch.arange(slots) % 3).int()
    ids[7] = -1
    x, w = torch.randn(slots, d, generator=g, device="cuda").bfloat16(), torch.randn(N, n, d, generator=g, device="cuda").bfloat16()
    meta, st = _meta(ids, N), _status()
    a = torch.zeros(slots, n, dtype=torch.bfloat16, device="cuda")
    lora.lora_expert_linear(a, x, w, meta, st)
    x[7], x[100], w[3] = math.nan, math.nan, math.nan
    b = torch.zeros_like(a)
    lora.lora_expert_linear(b, x, w, meta, st)
    keep = [i for i in range(slots) if i != 100]
    assert torch.equal(a[keep], b[keep]) and torch.isnan(b[100]).all() and (b[7] == 0).all()


def test_experts_bad_ids_are_left_out(cuda_lib):
    """Ids outside [-1, N) are flagged by the grouping and their slots left as they were."""
    ids = torch.tensor([0, 5, -7, 1, 2, 1], dtype=torch.int32)
    meta, st = lora.Meta(6, 2, min_run=0), _status()
    lora.lora_build_segments(ids.cuda(), meta, st)
    assert int(st.item()) == lora.DEV_BAD_ID
    y = torch.full((6, 8), 7.0, device="cuda")
    lora.lora_expert_linear(y, torch.ones(6, 4, device="cuda"), torch.ones(2, 8, 4, device="cuda"), meta, st)
    assert (y[[0, 3, 5]] == 4).all() and (y[[1, 2, 4]] == 7).all()


def test_experts_zero_slots(cuda_lib):
    meta, st = _meta(torch.empty(0, dtype=torch.int32), 3), _status()
    lora.lora_expert_linear(torch.empty(0, 8, device="cuda"), torch.empty(0, 4, device="cuda"), torch.empty(3, 8, 4, device="cuda"),
                            meta, st)


# ------------------------------------------------------------------------ sum
@pytest.mark.parametrize("residual", [None, "own", "in place"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,d", [(1, 1, 1), (1, 8, 4096), (3, 2, 7), (33, 8, 2048), (5, 3, 1003), (64, 4, 264), (7, 32, 520),
                                   (100, 5, 1032), (2, 1, 8192), (1000, 2, 256)])
def test_sum(cuda_lib, T, k, d, dtype, residual):
    g = torch.Generator(device="cuda").manual_seed(T + k + d)
    N = 6
    ids = torch.randint(-2, N + 2, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.randn(T, k, generator=g, device="cuda")
    x = torch.randn(T * k, d, generator=g, device="cuda").to(dtype)
    res = None if residual is None else (4 * torch.randn(T, d, generator=g, device="cuda")).to(dtype)
    there = (ids >= 0) & (ids < N)
    x[~there.view(-1)] = math.nan                     # rows of slots without an expert: not read
    terms = torch.where(there[:, :, None], w.double()[:, :, None] * x.double().view(T, k, d), torch.zeros((), dtype=torch.float64, device="cuda"))
    want, mag = terms.sum(1), terms.abs().sum(1)
    if res is not None:
        want, mag = want + res.double(), mag + res.double().abs()
    if residual == "in place":
        y = res.clone()
        lora.lora_expert_sum(y, x, ids, w, N, residual=y)
    else:
        buf, y = nan_frame((T, d), dtype)
        lora.lora_expert_sum(y, x, ids, w, N, residual=res)
        assert_frame(buf, (T, d))
    # k sums and products in fp32, one rounding
    assert_close(y, want, mag * (k + 1) * 2.0 ** -24 + want.abs() * torch.finfo(dtype).eps / 2 * 1.01)


# ------------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,N", [(1, 2, 8), (50, 3, 8), (700, 2, 16)])
def test_block(cuda_lib, T, k, N, dtype):
    """Router, grouping, gate and up, down, sum, with a shared expert through lora_linear; captured and replayed on new
    tokens, and equal to the same calls made eagerly."""
    d, f = 256, 392
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    Wr, Wgu, Wd = r(N, d).to(dtype), (r(N, 2 * f, d) / d ** 0.5).to(dtype), (r(N, d, f) / f ** 0.5).to(dtype)
    Sgu, Sd = (r(2 * f, d) / d ** 0.5).to(dtype), (r(d, f) / f ** 0.5).to(dtype)
    st = _status()
    x, res = torch.empty(T, d, dtype=dtype, device="cuda"), torch.empty(T, d, dtype=dtype, device="cuda")
    logits, ids = torch.empty(T, N, dtype=dtype, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    weights, meta = torch.empty(T, k, device="cuda"), lora.Meta(T * k, N, min_run=0)
    h, z = torch.zeros(T * k, f, dtype=dtype, device="cuda"), torch.zeros(T * k, d, dtype=dtype, device="cuda")
    sh, y = torch.empty(T, f, dtype=dtype, device="cuda"), torch.empty(T, d, dtype=dtype, device="cuda")

    def block():
        lora.lora_linear(logits, x, Wr, st)
        lora.lora_expert_route(ids, weights, logits)
        lora.lora_build_segments(ids.view(-1), meta, st)
        lora.lora_expert_linear(h, x, Wgu, meta, st, x_div=k, act=lora.ACT_SILU, gated=True)
        lora.lora_expert_linear(z, h, Wd, meta, st)
        lora.lora_linear(sh, x, Sgu, st, act=lora.ACT_SILU, gated=True)
        lora.lora_linear(y, sh, Sd, st, residual=res)
        lora.lora_expert_sum(y, z, ids, weights, N, residual=y)

    graph = torch.cuda.CUDAGraph()
    x.copy_(r(T, d)), res.copy_(r(T, d))
    with torch.cuda.graph(graph):
        block()
    for _ in range(3):
        x.copy_(r(T, d)), res.copy_(r(T, d))
        block()
        eager = y.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and int(st.item()) == 0
        X = x.double()
        ids64, w64 = _route64(logits, k, lora.SCORE_SOFTMAX, True, 1.0)   # of the logits as they were stored
        assert torch.equal(ids.cpu(), ids64)
        act = lambda u: u[:, :f] * torch.sigmoid(u[:, :f]) * u[:, f:]
        want = res.double() + act(X @ Sgu.double().T) @ Sd.double().T
        mag = want.norm()
        for t in range(T):
            for j in range(k):
                e = int(ids64[t, j])
                v = act(X[t:t + 1] @ Wgu[e].double().T) @ Wd[e].double().T
                want[t] += float(w64[t, j]) * v[0]
        # h, z, sh and y (twice) each rounded: norms off by at most eps / 2 of their parts
        assert (y.double() - want).norm() <= 5 * torch.finfo(dtype).eps / 2 * (want.norm() + mag) * (1 if dtype == torch.bfloat16 else 8)


def test_two_streams_share_a_grouping(cuda_lib):
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(0, 8, (600,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    meta, st = _meta(ids, 8), _status()
    x, w = torch.randn(600, 256, generator=g, device="cuda").bfloat16(), torch.randn(8, 512, 256, generator=g, device="cuda").bfloat16()
    want = torch.zeros(600, 512, dtype=torch.bfloat16, device="cuda")
    lora.lora_expert_linear(want, x, w, meta, st)
    torch.cuda.synchronize()
    ys, streams = [torch.zeros_like(want) for _ in range(3)], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, y in zip(streams, ys):
            lora.lora_expert_linear(y, x, w, meta, st, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in ys) and int(st.item()) == 0


STALLS = [(s, r) for s in [(4, 4, 2048, 264), (300, 5, 512, 520), (5000, 3, 256, 2056)] for r in (1, 2, 3, 4, 5)] + \
    [((200, 3, 333, 257), r) for r in (1, 2, 4)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("shape,role", STALLS)
def test_stalled_warp_times_out_and_the_context_survives(cuda_lib, monkeypatch, shape, gated, role):
    """As lora_linear's: the wait runs out, the call returns, the next one is exact."""
    slots, N, d, n = shape
    ids = (torch.arange(slots) * 7 % N).int()
    meta, st = _meta(ids, N), _status()
    y = torch.full((slots + 1, n + 8), 99.0, dtype=torch.bfloat16, device="cuda")
    x, w = torch.ones(slots, d, dtype=torch.bfloat16, device="cuda"), torch.ones(N, 2 * n if gated else n, d, dtype=torch.bfloat16, device="cuda")
    monkeypatch.setenv("LORA_DEBUG_STALL", str(role))
    lora.lora_expert_linear(y[:slots, :n], x, w, meta, st, gated=gated)
    monkeypatch.delenv("LORA_DEBUG_STALL")
    assert int(st.item()) == lora.DEV_TIMEOUT
    assert (y[slots] == 99).all() and (y[:, n:] == 99).all()
    _experts_check(slots, slots, N, d, n, torch.bfloat16, gated=gated)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 8704), (torch.bfloat16, 8701), (torch.float32, 8704)])
def test_experts_offsets_past_32_bits(cuda_lib, dtype, d):
    """Weights of more than 2^31 elements: the last expert's rows lie beyond."""
    N, n, slots = 9, 28672, 40
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.zeros(N, n, d, dtype=dtype, device="cuda")
    x, last = whole(g, (slots, d), 1).to(dtype), whole(g, (n, d), 1).to(dtype)
    w[N - 1] = last
    ids = torch.where(torch.arange(slots) % 3 == 0, N - 1, 0).int()
    meta, st = _meta(ids, N), _status()
    y = torch.full((slots, n), 7.0, dtype=dtype, device="cuda")
    lora.lora_expert_linear(y, x, w, meta, st)
    want = torch.where((ids == N - 1)[:, None].cuda(), x.float() @ last.float().T, torch.zeros((), device="cuda")).to(dtype)
    assert torch.equal(y, want) and int(st.item()) == 0   # whole numbers below 2^24


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 64), (torch.bfloat16, 33), (torch.float32, 64)])
def test_experts_most_slots_and_experts(cuda_lib, dtype, d):
    _experts_check(3, lora.MAX_ROWS, lora.MAX_EXPERTS, d, 72, dtype, "skewed", x_div=8)


def test_run_case(cuda_lib):
    from lora_adapter_application_b200 import run_case
    assert run_case.main(["decode_qproj", "--base", "bf16", "--experts", "8", "--reps", "2"]) == 0
    assert run_case.main(["tiny", "--base", "bf16", "--experts", "3", "--reps", "1"]) == 0


# ------------------------------------------------------------------------ sum: order
@pytest.mark.parametrize("T", [3, 4099])
@pytest.mark.parametrize("d", [264, 259])
def test_sum_adds_the_residual_last(cuda_lib, T, d):
    """Eight halves and 2^24: 2^24 + 4, where adding them to 2^24 one by one leaves it as it is (0.5 is a quarter of its last place)."""
    k = 8
    x, w = torch.ones(T * k, d, device="cuda"), torch.full((T, k), 0.5, device="cuda")
    y = torch.full((T, d), 2.0 ** 24, device="cuda")
    lora.lora_expert_sum(y, x, torch.zeros(T, k, dtype=torch.int32, device="cuda"), w, 1, residual=y)
    assert (y == 2.0 ** 24 + 4).all()


@pytest.mark.parametrize("T", [3, 4099])
@pytest.mark.parametrize("d", [264, 259])
@pytest.mark.parametrize("dtype", DTYPES)
def test_sum_leaves_tokens_without_experts_bit_for_bit(cuda_lib, T, d, dtype):
    """A residual of -0 stays -0 where no slot adds to it; without a residual the sum of nothing is 0."""
    k = 3
    ids = torch.where(torch.arange(T) % 2 == 0, -1, 0).int()[:, None].expand(T, k).contiguous().cuda()
    x, w = torch.ones(T * k, d, dtype=dtype, device="cuda"), torch.zeros(T, k, device="cuda")
    y = torch.full((T, d), -0.0, dtype=dtype, device="cuda")
    lora.lora_expert_sum(y, x, ids, w, 1, residual=y)
    assert torch.equal(torch.signbit(y), (ids[:, :1] < 0).expand(T, d)) and (y == 0).all()   # 0 * 1 + -0 = 0
    lora.lora_expert_sum(y, x, ids, w, 1)
    assert not torch.signbit(y).any() and (y == 0).all()
