"""The experts' calls over operands with strides, at addresses off 16 bytes and in place, groupings of other parameters, and
sums of enough tokens that a warp takes several (tolerances: dense_helpers)."""
import math

import pytest
import torch

import lora_adapter_application_b200 as lora
from dense_helpers import ACTS, assert_close, dense64, whole
from test_experts_gpu import _group_ids, _status, test_sum as check_sum

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


def _spread(t, pad, off):
    """A copy of t whose rows lie pad + off elements further apart, among NaN, from element off on."""
    buf = torch.full((t.shape[0], t.shape[1] + pad + off), math.nan, dtype=t.dtype, device="cuda")
    v = buf[:, off:off + t.shape[1]]
    v.copy_(t)
    return v


def _case(seed, slots, N, d, n, gated, x_div, dtype):
    """(ids, operands in fp64, the same in dtype), some slots without an expert."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = _group_ids("out", slots, N, torch.Generator().manual_seed(seed)).clamp(min=-1)
    n_w = 2 * n if gated else n
    o = {"x": whole(g, (-(-slots // x_div), d), 2), "w": whole(g, (N, n_w, d), 2, 2.0 ** -round(math.log2(d) / 2)),
         "bias": whole(g, (N, n_w), 8, 0.25), "addend": whole(g, (slots, n_w), 8, 0.25), "residual": whole(g, (slots, n), 64, 0.5)}
    return ids, o, {k: v.to(dtype) for k, v in o.items()}


def _grouped(ids, N, rows_per_tile=16, min_run=0, static=False):
    meta, st = lora.Meta(ids.numel(), N, rows_per_tile, min_run), _status()
    (lora.lora_build_segments_static if static else lora.lora_build_segments)(ids.cuda(), meta, st)
    assert int(st.item()) == 0
    return meta


def _check(y, before, ids, o, act, gated, x_div, dtype, what=""):
    """Slots with an expert hold its product, the others what they held before."""
    for e in range(-1, o["w"].shape[0]):
        mine = (ids == e).nonzero()[:, 0].cuda()
        if mine.numel() == 0:
            continue
        if e < 0:
            assert torch.equal(y[mine], before[mine]), what
            continue
        want, tol = dense64(o["x"][mine // x_div], o["w"][e], o["bias"][e], o["addend"][mine], o["residual"][mine], act, gated, dtype)
        assert_close(y[mine], want, tol, f"{what} expert {e}")


# few and many rows a group; 333: rows off 16-byte steps however they lie
SHAPES = [(24, 5, 256, 136, 2), (300, 5, 256, 264, 3), (1500, 4, 192, 520, 1), (200, 3, 333, 130, 2)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("slots,N,d,n,x_div", SHAPES)
def test_operands_with_strides_and_off_16_bytes(cuda_lib, slots, N, d, n, x_div, dtype, gated):
    ids, o, s = _case(slots, slots, N, d, n, gated, x_div, dtype)
    meta, st = _grouped(ids, N), _status()

    def run(x, addend, residual, what):
        y = torch.full((slots, n), 7.0, dtype=dtype, device="cuda")
        before = y.clone()
        lora.lora_expert_linear(y, x, s["w"], meta, st, x_div=x_div, bias=s["bias"], addend=addend, residual=residual,
                                act=lora.ACT_SILU, gated=gated)
        assert int(st.item()) == 0
        _check(y, before, ids, o, lora.ACT_SILU, gated, x_div, dtype, what)
    for pad, off in [(64, 0), (56, 8), (3, 0), (8, 1), (2, 2)]:
        run(*(_spread(s[k], pad, off) for k in ("x", "addend", "residual")), f"pad {pad} off {off}")
    for one in ("x", "addend", "residual"):
        run(*(_spread(s[k], 7, 1) if k == one else s[k] for k in ("x", "addend", "residual")), one)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("slots,N,d,n,x_div", SHAPES)
def test_in_place(cuda_lib, slots, N, d, n, x_div, dtype):
    """y over the residual, over the addend; a gated y over the residual."""
    for gated, over in [(False, "residual"), (False, "addend"), (True, "residual")]:
        ids, o, s = _case(slots + 1, slots, N, d, n, gated, x_div, dtype)
        meta, st = _grouped(ids, N), _status()
        y = s[over].clone()
        before = y.clone()
        lora.lora_expert_linear(y, s["x"], s["w"], meta, st, x_div=x_div, bias=s["bias"], act=lora.ACT_GELU, gated=gated,
                                **{**{k: s[k] for k in ("addend", "residual")}, over: y})
        assert int(st.item()) == 0
        _check(y, before, ids, o, lora.ACT_GELU, gated, x_div, dtype, over)


@pytest.mark.parametrize("rows_per_tile,min_run,static", [(1, 0, False), (64, 1, False), (16, 4, False), (8, 64, True)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_groupings_of_any_parameters(cuda_lib, dtype, rows_per_tile, min_run, static):
    """Runs of one expert that the grouping sets apart for the adapters' kernels, and the grouping without scratch."""
    slots, N, d, n = 700, 6, 128, 136
    ids, o, s = _case(9, slots, N, d, n, True, 1, dtype)
    ids[100:420] = 3
    meta, st = _grouped(ids, N, rows_per_tile, min_run, static), _status()
    y = torch.full((slots, n), 7.0, dtype=dtype, device="cuda")
    before = y.clone()
    lora.lora_expert_linear(y, s["x"], s["w"], meta, st, bias=s["bias"], addend=s["addend"], residual=s["residual"],
                            act=lora.ACT_SILU, gated=True)
    assert int(st.item()) == 0
    _check(y, before, ids, o, lora.ACT_SILU, True, 1, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("slots,N,d,n", [(24, 5, 4096, 136), (300, 5, 512, 264), (3000, 4, 200, 520), (200, 3, 333, 130)])
def test_a_call_repeated_gives_the_same_bits(cuda_lib, slots, N, d, n, dtype):
    g = torch.Generator(device="cuda").manual_seed(slots)
    ids = _group_ids("skewed", slots, N, torch.Generator().manual_seed(1))
    x, w = torch.randn(slots, d, generator=g, device="cuda").to(dtype), torch.randn(N, n, d, generator=g, device="cuda").to(dtype)
    meta, st = _grouped(ids, N), _status()
    ys = [torch.zeros(slots, n, dtype=dtype, device="cuda") for _ in range(4)]
    for y in ys:
        lora.lora_expert_linear(y, x, w, meta, st, act=ACTS[1])
    assert all(torch.equal(y, ys[0]) for y in ys) and int(st.item()) == 0


# ------------------------------------------------------------------------ sum
@pytest.mark.parametrize("residual", [None, "own", "in place"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,d", [(4095, 8, 264), (4096, 1, 16), (4097, 8, 264), (4099, 4, 1003), (4098, 10, 64), (4097, 16, 72),
                                   (4097, 17, 40), (5001, 32, 24), (4101, 3, 1032), (6000, 9, 7)])
def test_sum_of_many_tokens(cuda_lib, T, k, d, dtype, residual):
    """From 4096 tokens on a warp takes up to four of them, as many as its lanes hold the slots of; the last one fewer."""
    check_sum(cuda_lib, T, k, d, dtype, residual)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [5, 4099])
@pytest.mark.parametrize("pad,off", [(8, 0), (24, 8), (3, 0), (8, 1)])
def test_sum_of_strided_rows(cuda_lib, T, pad, off, dtype):
    k, d, N = 3, 264, 4
    g = torch.Generator(device="cuda").manual_seed(T + pad)
    ids = torch.randint(-1, N, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w, x, res = whole(g, (T, k), 4, 0.25), whole(g, (T * k, d), 8), whole(g, (T, d), 8)
    want = res + torch.where((ids >= 0)[:, :, None], w[:, :, None] * x.view(T, k, d), torch.zeros((), dtype=torch.float64, device="cuda")).sum(1)
    want = want.to(dtype)   # quarters up to 32: fp32 holds every sum, one rounding into y
    for xs, rs, y in [(_spread(x.to(dtype), pad, off), _spread(res.to(dtype), pad, off), None), (_spread(x.to(dtype), pad, off), res.to(dtype), None),
                      (x.to(dtype), _spread(res.to(dtype), pad, off), None), (x.to(dtype), _spread(res.to(dtype), pad, off), "in place")]:
        y = rs if y else torch.empty(T, d, dtype=dtype, device="cuda")
        lora.lora_expert_sum(y, xs, ids, w.float(), N, residual=rs)
        assert torch.equal(y, want)
