"""64-bit statement of the microscaled formats and the operators around them, in
numpy: the element tables of the OCP Microscaling formats v1.0 (e4m3, e2m1), a
block's scale, nearest element with ties to the even code, the storage of
include/lora_delta.h (lora_mx), the root-mean-square norm and the base product.
Test infrastructure: the library shares no code with it."""
import numpy as np

MXFP8, MXFP4 = 0, 1
EMAX = {MXFP8: 8, MXFP4: 2}


def table(fmt):
    """The magnitudes of codes 0, 1, 2, ... (sign bit clear, NaN left out)."""
    if fmt == MXFP4:
        return np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    return np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                     for e in range(16) for m in range(8)][:127])


def padded(cols):
    return -(-cols // 128) * 128


def quantize(v, fmt):
    """(codes [rows, padded], scale bytes [rows, padded / 32]) of fp64 rows."""
    rows, cols = v.shape
    b = np.zeros((rows, padded(cols)))
    b[:, :cols] = v
    b = b.reshape(rows, -1, 32)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        top = np.abs(b).max(2)
        bad = ~np.isfinite(top)
        _, ex = np.frexp(np.where(bad, 0, top))            # top = m 2^ex, m in [0.5, 1)
        e = np.where(top > 0, ex - 1 - EMAX[fmt], -127)
        e = np.clip(e, -127, None) + 127
        m = np.where(bad[:, :, None], 0, np.abs(b)) / 2.0 ** (e - 127.0)[:, :, None]
    t = table(fmt)
    hi = np.clip(np.searchsorted(t, m), 0, len(t) - 1)
    lo = np.clip(hi - 1, 0, None)
    up, down = t[hi] - m, m - t[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    sign = np.signbit(b) & ~bad[:, :, None]
    code = code + sign * (128 if fmt == MXFP8 else 8)
    return code.reshape(rows, -1).astype(np.uint8), np.where(bad, 255, e).astype(np.uint8)


def values(codes, scales, fmt, cols):
    """The fp64 values of codes and scale bytes."""
    t = np.append(table(fmt), [np.nan] if fmt == MXFP8 else [])
    half = len(t)
    q = np.where(codes >= half, -1.0, 1.0) * t[codes % half]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (q.reshape(len(q), -1, 32) * s[:, :, None]).reshape(len(q), -1)[:, :cols]


def pack(codes, fmt):
    """Stored bytes of codes [rows, padded]."""
    return codes if fmt == MXFP8 else (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(data, fmt):
    if fmt == MXFP8:
        return data
    out = np.empty((data.shape[0], data.shape[1] * 2), np.uint8)
    out[:, 0::2], out[:, 1::2] = data & 15, data >> 4
    return out


def scale_index(rows, n_blocks):
    """Where the scale byte of row r, block b is stored: [rows, n_blocks]."""
    r, b = np.arange(rows)[:, None], np.arange(n_blocks)[None, :]
    return ((r // 128) * (n_blocks // 4) + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4


def pack_scales(s):
    rows, n = s.shape
    out = np.zeros(-(-rows // 128) * (n // 4) * 512, np.uint8)
    out[scale_index(rows, n)] = s
    return out


def unpack_scales(data, rows, cols):
    return data[scale_index(rows, padded(cols) // 32)]


def rms_norm(r, weight, eps):
    return r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * weight
