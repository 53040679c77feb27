"""Host-side refusals of lora_linear and the experts' calls: through the C ABI, before anything reaches a GPU, and in
the binding.  Runs without a GPU."""
import ctypes

import pytest
import torch

import lora_adapter_application_b200 as lora
from lora_adapter_application_b200 import LoraError

NULL, DTYPE, SHAPE, CAPACITY = -1, -2, -3, -7
P, Q, R = 4096, 8192, 16384   # addresses that no call may touch


@pytest.fixture(scope="module")
def lib():
    from lora_adapter_application_b200 import build
    build.build()
    return lora.load()


def _ep(**kw):
    e = lora.lora_epilogue()
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def _ref(e):
    return None if e is None else ctypes.addressof(e)


def test_linear_refusals(lib):
    ok = dict(y=P, ld_y=96, x=Q, ld_x=64, w=R, ld_w=64, T=4, d=64, n=96, ep=None, dt=0, st=P)

    def call(**over):
        f = dict(ok, **over)
        return lib.lora_linear(f["y"], f["ld_y"], f["x"], f["ld_x"], f["w"], f["ld_w"], f["T"], f["d"], f["n"], _ref(f["ep"]),
                               f["dt"], f["st"], None)
    assert call(T=0) == 0 and call(T=0, y=None, x=None, w=None) == 0
    for over, want in [(dict(dt=2), DTYPE), (dict(T=-1), SHAPE), (dict(T=131073), SHAPE), (dict(d=0), SHAPE), (dict(n=0), SHAPE),
                       (dict(d=(1 << 20) + 1, ld_x=1 << 22, ld_w=1 << 22), SHAPE), (dict(n=(1 << 20) + 1, ld_y=1 << 22), SHAPE),
                       (dict(ld_x=63), SHAPE), (dict(ld_w=63), SHAPE), (dict(ld_y=95), SHAPE), (dict(st=None), NULL),
                       (dict(y=None), NULL), (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=Q), SHAPE),
                       (dict(ep=_ep(act=5)), SHAPE), (dict(ep=_ep(act=-1)), SHAPE),
                       (dict(ep=_ep(addend=R, ld_addend=95)), SHAPE), (dict(ep=_ep(addend=R, ld_addend=191, gated=1)), SHAPE),
                       (dict(ep=_ep(residual=R, ld_residual=95)), SHAPE), (dict(ep=_ep(residual=P, ld_residual=97)), SHAPE),
                       (dict(ep=_ep(addend=P, ld_addend=97)), SHAPE), (dict(ep=_ep(addend=P, ld_addend=192, gated=1)), SHAPE),
                       (dict(n=(1 << 19) + 1, ld_y=1 << 22, ep=_ep(gated=1)), SHAPE)]:
        assert call(**over) == want, over


def _meta(T=8, N=3, **kw):
    mg, mc = lora.lora_meta_capacity(T, N, 16, 0)
    f = dict(T=T, N=N, rows_per_tile=16, min_run=0, long_tile=128, max_gather_tiles=mg, max_contig_tiles=mc, perm=P, seg_start=P,
             seg_adapter=P, counts=P, grow=P, gather_tiles=P, contig_tiles=P)
    f.update(kw)
    return lora.lora_meta(*f.values())


def test_expert_linear_refusals(lib):
    ok = dict(y=P, ld_y=96, x=Q, ld_x=64, rows=4, div=2, w=R, d=64, n=96, meta=_meta(), ep=None, dt=0, st=P)

    def call(**over):
        f = dict(ok, **over)
        m = None if f["meta"] is None else ctypes.byref(f["meta"])
        return lib.lora_expert_linear(f["y"], f["ld_y"], f["x"], f["ld_x"], f["rows"], f["div"], f["w"], f["d"], f["n"], m,
                                      _ref(f["ep"]), f["dt"], f["st"], None)
    assert call(meta=_meta(T=0), rows=0) == 0
    for over, want in [(dict(meta=None), NULL), (dict(meta=_meta(N=1025)), SHAPE), (dict(meta=_meta(perm=None)), NULL),
                       (dict(meta=_meta(max_gather_tiles=0)), CAPACITY), (dict(div=0), SHAPE), (dict(rows=3), SHAPE),
                       (dict(rows=-1), SHAPE), (dict(dt=3), DTYPE), (dict(ld_x=63), SHAPE), (dict(ld_y=95), SHAPE), (dict(st=None), NULL),
                       (dict(y=None), NULL), (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=Q), SHAPE),
                       (dict(ep=_ep(act=9)), SHAPE), (dict(ep=_ep(addend=P, ld_addend=192, gated=1)), SHAPE)]:
        assert call(**over) == want, over


def test_route_refusals(lib):
    ok = dict(ids=P, w=Q, l=R, ld=64, T=4, n=64, k=8, score=0, dt=0)

    def call(**over):
        f = dict(ok, **over)
        return lib.lora_expert_route(f["ids"], f["w"], f["l"], f["ld"], f["T"], f["n"], f["k"], f["score"], 1, 1.0, f["dt"], None)
    assert call(T=0) == 0
    for over, want in [(dict(dt=2), DTYPE), (dict(T=-1), SHAPE), (dict(T=131073), SHAPE), (dict(n=0, k=0), SHAPE), (dict(ld=63), SHAPE),
                       (dict(n=1025, ld=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(n=4, k=5), SHAPE),
                       (dict(score=2), SHAPE), (dict(score=-1), SHAPE), (dict(ids=None), NULL), (dict(w=None), NULL), (dict(l=None), NULL)]:
        assert call(**over) == want, over


def test_sum_refusals(lib):
    ok = dict(y=P, ld_y=64, x=Q, ld_x=64, ids=R, w=R, N=8, T=4, k=2, d=64, r=None, ld_r=0, dt=0)

    def call(**over):
        f = dict(ok, **over)
        return lib.lora_expert_sum(f["y"], f["ld_y"], f["x"], f["ld_x"], f["ids"], f["w"], f["N"], f["T"], f["k"], f["d"], f["r"],
                                   f["ld_r"], f["dt"], None)
    assert call(T=0) == 0
    for over, want in [(dict(dt=2), DTYPE), (dict(T=-1), SHAPE), (dict(T=131073), SHAPE), (dict(N=0), SHAPE), (dict(N=1025), SHAPE),
                       (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(d=0), SHAPE), (dict(d=(1 << 20) + 1, ld_y=1 << 22, ld_x=1 << 22), SHAPE),
                       (dict(ld_x=63), SHAPE), (dict(ld_y=63), SHAPE), (dict(r=R, ld_r=63), SHAPE), (dict(r=P, ld_r=65), SHAPE),
                       (dict(y=Q), SHAPE), (dict(y=None), NULL), (dict(x=None), NULL), (dict(ids=None), NULL), (dict(w=None), NULL)]:
        assert call(**over) == want, over


# ------------------------------------------------------------------- binding refusals
def _cpu_meta(T, N):
    return lora.Meta(T, N, min_run=0, device="cpu")


def test_binding_refuses_cpu_and_mismatched_operands(lib):
    x, w, y, st = torch.zeros(4, 64), torch.zeros(96, 64), torch.zeros(4, 96), torch.zeros(1, dtype=torch.int32)
    ok = dict(y=y, x=x, w=w, status=st)
    for over, msg in [({}, "CUDA"), (dict(w=w.bfloat16()), "dtype"), (dict(w=torch.zeros(96, 63)), "w must be"),
                      (dict(w=torch.zeros(95, 64), gated=True), "even"), (dict(x=x.t()), "2-D"), (dict(x=x[0]), "2-D"),
                      (dict(x=x[:1].expand(4, 64)), "overlap"), (dict(w=torch.zeros(0, 64)), "1 to"), (dict(x=torch.zeros(4, 0), w=torch.zeros(9, 0)), "1 to")]:
        with pytest.raises(LoraError, match=msg):
            lora.lora_linear(**{**ok, **over})
    m, w3 = _cpu_meta(8, 3), torch.zeros(3, 96, 64)
    ok = dict(y=torch.zeros(8, 96), x=torch.zeros(4, 64), w=w3, meta=m, status=st, x_div=2)
    for over, msg in [({}, "CUDA"), (dict(w=w), "w must be"), (dict(w=torch.zeros(2, 96, 64)), "w must be"), (dict(x_div=1), "every slot"),
                      (dict(w=torch.zeros(3, 64, 96).transpose(1, 2)), "w must be"), (dict(x_div=0), "every slot"),
                      (dict(w=torch.zeros(3, 95, 64), gated=True), "even")]:
        with pytest.raises(LoraError, match=msg):
            lora.lora_expert_linear(**{**ok, **over})
    ids, wt, lg = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(4, 8)
    for a, k, msg in [((ids, wt, lg), {}, "CUDA"), ((ids[:3], wt, lg), {}, "ids"), ((ids, wt, lg[:, :1]), {}, "at most"),
                      ((ids, wt, lg), dict(score=2), "score"), ((torch.zeros(4, 0, dtype=torch.int32), wt, lg), {}, "at most"),
                      ((ids, wt, torch.zeros(4, 1025)), {}, "at most")]:
        with pytest.raises(LoraError, match=msg):
            lora.lora_expert_route(*a, **k)
    for a, msg in [((y, torch.zeros(8, 96), ids, wt, 8), "CUDA"), ((y, torch.zeros(8, 96), ids[:3], wt, 8), "ids"),
                   ((y, torch.zeros(8, 96), ids, wt, 0), "at most"), ((y, torch.zeros(8, 96), ids, wt, 1025), "at most")]:
        with pytest.raises(LoraError, match=msg):
            lora.lora_expert_sum(*a)


def test_sizes_past_the_limits_are_refused(lib):
    """ctypes would pass them modulo 2^32."""
    big, st = 1 << 32, torch.zeros(1, dtype=torch.int32)
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="meta")
    for T, d, n in [(131073, 8, 8), (big + 1, 8, 8), (1, big + 8, 8), (1, 8, big + 8), (1, (1 << 20) + 1, 8), (1, 8, (1 << 20) + 1)]:
        with pytest.raises(LoraError, match="at most"):
            lora.lora_linear(e(T, n), e(T, d), e(n, d), st)
    m = _cpu_meta(8, 3)
    for R_, d, n in [((1 << 20) + 1, 8, 8), (8, big + 8, 8), (8, 8, big + 8)]:
        with pytest.raises(LoraError, match="at most"):
            lora.lora_expert_linear(e(8, n), e(R_, d), e(3, n, d), m, st)
    with pytest.raises(LoraError, match="every slot"):
        lora.lora_expert_linear(e(8, 8), e(8, 8), e(3, 8, 8), m, st, x_div=big + 1)


# ------------------------------------------------------------------- addresses off their elements' size
ALIGN = -5


@pytest.mark.parametrize("dt,off", [(0, 1), (1, 1), (1, 2), (1, 3)])
def test_addresses_off_their_elements_are_refused(lib, dt, off):
    """Odd addresses of bf16 data, and fp32 data, ids, weights and a status off four bytes: no kernel can read those."""
    ep = {}

    def linear(y=P, x=Q, w=R, st=P):
        return lib.lora_linear(y, 96, x, 64, w, 64, 4, 64, 96, _ref(ep.get("e")), dt, st, None)

    def experts(y=P, x=Q, w=R, st=P, **meta):
        m = _meta(**meta)
        return lib.lora_expert_linear(y, 96, x, 64, 4, 2, w, 64, 96, ctypes.byref(m), _ref(ep.get("e")), dt, st, None)
    for call in (linear, experts):
        for over in (dict(y=P + off), dict(x=Q + off), dict(w=R + off), dict(st=P + 2)):
            assert call(**over) == ALIGN, (call.__name__, over)
        for over in (dict(bias=R + off), dict(addend=R + off, ld_addend=96), dict(residual=R + off, ld_residual=96)):
            ep["e"] = _ep(**over)
            assert call() == ALIGN, (call.__name__, over)
        ep.clear()
    assert experts(perm=P + 2) == ALIGN and experts(seg_start=P + 2) == ALIGN

    def route(ids=P, w=Q, logits=R):
        return lib.lora_expert_route(ids, w, logits, 64, 4, 64, 8, 0, 1, 1.0, dt, None)
    for over in (dict(ids=P + off), dict(w=Q + off), dict(logits=R + off)):
        assert route(**over) == ALIGN, over

    def total(y=P, x=Q, ids=R, w=R, r=None):
        return lib.lora_expert_sum(y, 64, x, 64, ids, w, 8, 4, 2, 64, r, 64, dt, None)
    for over in (dict(y=P + off), dict(x=Q + off), dict(ids=R + off), dict(w=R + off), dict(r=R + off)):
        assert total(**over) == ALIGN, over


def test_current_device_is_asked_for_in_public(lib, monkeypatch):
    """The helper behind every call goes by torch.cuda.current_device(): the call is made at once where it is the operands'."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    got = []
    lora._call_on(3, 17, lambda *a: got.append(a) or 0, "a", "b")
    assert got == [("a", "b", 17)]
    with pytest.raises(LoraError):
        lora._call_on(3, 17, lambda *a: SHAPE)
