"""64-bit statement of the dense products' epilogue, and how far a kernel's result may be
from it.

Whole inputs: x and W hold whole numbers (bias and addend halves), so that every partial sum is held by fp32 exactly
in any order: z is exact, whatever the kernel's order.  Then y is off by its activation's arithmetic and the one rounding
(finfo(dtype).eps / 2 of y):
    none, relu        nothing more
    silu, gelu_tanh   z / (1 + e^-u).  e^-u: bf16 results use ex2.approx of -u log2 e (2 units of 2^-23, and two roundings of
                      the argument, |u| 2^-23 together: less than 2 + 1.16 |u| units), fp32 ones expf, 2; u itself 4
                      roundings, which e^-u multiplies by |u|: 4 |u| units of 2^-24; sum, reciprocal or quotient (1 to 2
                      units) and the rest 5 units: (9 + 3.2 |u|) 2^-23
    gelu              z erfc(v) / 2, v = -z / sqrt 2 rounded twice; erfc changes by at most (2 v^2 + 2) of a relative change
                      of v: (2 v^2 + 2) units; erfcf 4 units (CUDA's bound), two products: (8 + 2 v^2) 2^-23 = (8 + z^2) 2^-23.
                      bf16 results: the exponent -z^2 / 2 rounded twice, z^2 / 2 units of 2^-24 each, exponential and reciprocal 2
                      each, the fit 1, three products: within the same
    gated             one product more, residual one sum more: 2^-24 each of their results
and, where fp32 cannot hold e^-u or a quotient (below 2^-126), 2^-120.
Any inputs, no activation: fp32 accumulation of K exact products in any order is off by at most K 2^-23 sum |x w| (2^-23: a
hardware adder may truncate)."""
import math

import torch

import lora_adapter_application_b200 as lora

ACTS = [lora.ACT_NONE, lora.ACT_SILU, lora.ACT_GELU, lora.ACT_GELU_TANH, lora.ACT_RELU]


def act64(z, act):
    """(act(z), its relative error bound in units of 2^-23)"""
    if act == lora.ACT_SILU:
        return z * torch.sigmoid(z), 9 + 3.2 * z.abs()
    if act == lora.ACT_GELU:
        return z * torch.special.erfc(-z * math.sqrt(0.5)) / 2, 8 + z * z
    if act == lora.ACT_GELU_TANH:
        u = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
        return z * torch.sigmoid(u), 9 + 3.2 * u.abs()
    return (z.clamp(min=0) if act == lora.ACT_RELU else z), torch.zeros_like(z)


def dense64(x, w, bias=None, addend=None, residual=None, act=lora.ACT_NONE, gated=False, dtype=torch.bfloat16, dz=None):
    """(y, tolerance) in fp64, from fp64 operands; dz: how far z may be off before the activation (none: exact)."""
    z = x @ w.T
    if bias is not None:
        z = z + bias
    if addend is not None:
        z = z + addend
    n = z.shape[1] // 2 if gated else z.shape[1]
    y, rel = act64(z[:, :n], act)
    err = rel * 2.0 ** -23 * y.abs()
    if dz is not None:
        err = err + 1.13 * dz[:, :n]     # the steepest activation's slope
    if gated:
        if dz is not None:
            err = err * z[:, n:].abs() + y.abs() * dz[:, n:] + err * dz[:, n:]
        else:
            err = err * z[:, n:].abs()
        y = y * z[:, n:]
        err = err + 2.0 ** -24 * y.abs()
    if residual is not None:
        y = y + residual
        err = err + 2.0 ** -24 * (y.abs() + err)
    return y, err + (y.abs() + err) * torch.finfo(dtype).eps / 2 + 2.0 ** -120


def whole(g, shape, most=3, step=1.0):
    """Multiples of step up to `most` steps, on the GPU, fp64."""
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").double() * step


def assert_close(got, want, tol, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    if bad.any():
        at = bad.nonzero()[:5].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond tolerance, first at {at}: "
                             f"{[(got[tuple(i)].item(), want[tuple(i)].item()) for i in at]}")


def nan_frame(shape, dtype, pad=8):
    """A view of a larger buffer of NaN: (whole buffer, view whose rows are `pad` elements longer than it)."""
    buf = torch.full((shape[0] + 2, shape[1] + pad), math.nan, dtype=dtype, device="cuda")
    return buf, buf[1:-1, :shape[1]]


def assert_frame(buf, shape):
    """Nothing outside the view was written."""
    out = torch.ones_like(buf, dtype=torch.bool)
    out[1:-1, :shape[1]] = False
    assert torch.isnan(buf[out]).all()
