"""Microscaled (MX) formats, the product on them, and the residual + RMS norm
that feeds it, in float64 numpy.  Test infrastructure only (see
``oracle/__init__.py``).

The format is that of the published OCP Microscaling Formats specification:
blocks of 32 along a row, a power-of-two scale 2^(byte - 127) each (0xFF is
NaN), E2M1 or E4M3 elements.  The scale is the largest power of two that is at
most amax / 2^emax (emax: the exponent of the element format's top binade),
the elements are rounded to nearest even and saturate.

``quantize_mx(x, fmt)`` works on float64 copies of float32 input, where the
division by the scale is exact over the whole float32 range.
"""

from __future__ import annotations

import numpy as np

from .codecs import E2M1_MAG_VALUES, e2m1_round_mag, e4m3_all_values

FP4, FP8 = 0, 1
EMAX = {FP4: 2, FP8: 8}
LARGEST = {FP4: 6.0, FP8: 448.0}


def _magnitudes(fmt):
    """Ascending magnitudes of the element format; the index is the code."""
    return E2M1_MAG_VALUES if fmt == FP4 else np.asarray(e4m3_all_values(), dtype=np.float64)[:127]


def quantize_mx(x, fmt):
    """(element codes uint8 [m, k], one per entry; scale bytes uint8 [m, k/32])."""
    x = np.asarray(x, dtype=np.float64)
    m, k = x.shape
    b = x.reshape(m, k // 32, 32)
    amax = np.abs(b).max(-1)  # NaN if any entry is
    nan = ~np.isfinite(amax)
    a = np.where(nan | (amax == 0), 1.0, amax)
    _, e = np.frexp(a)  # a = f 2^e, f in [1/2, 1)
    byte = np.clip(e - 1 - EMAX[fmt] + 127, 0, 254)
    byte = np.where(amax == 0, 0, byte)
    v = np.where(nan[..., None], 0.0, b / np.ldexp(1.0, byte - 127)[..., None])
    mag = np.minimum(np.abs(v), LARGEST[fmt])
    if fmt == FP4:
        c = e2m1_round_mag(mag)
        sign = 8
    else:
        grid = _magnitudes(FP8)
        lo = np.searchsorted(grid, mag, side="right") - 1
        hi = np.minimum(lo + 1, 126)
        dl, dh = mag - grid[lo], grid[hi] - mag
        c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        sign = 128
    c = np.where(np.signbit(b) & ~nan[..., None], c | sign, np.where(nan[..., None], 0, c))
    return c.astype(np.uint8).reshape(m, k), np.where(nan, 255, byte).astype(np.uint8)


def pack(codes, fmt):
    """The stored bytes of element codes: MXFP4 two per byte, the even one low."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)) if fmt == FP4 else codes


def unpack(stored, fmt):
    if fmt == FP8:
        return stored
    return np.stack((stored & 15, stored >> 4), -1).reshape(stored.shape[0], -1)


def dequant_mx(stored, scales, fmt):
    """Values, float64, of a stored MX matrix."""
    c = unpack(np.asarray(stored), fmt).astype(np.int64)
    grid = np.append(_magnitudes(fmt), np.nan) if fmt == FP8 else _magnitudes(fmt)
    top = 128 if fmt == FP8 else 8
    v = np.where(c >= top, -1.0, 1.0) * grid[c % top]
    s = np.asarray(scales).astype(np.int64)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, np.minimum(s, 254) - 127))
    return v * np.repeat(f, 32, axis=-1)


def add_rmsnorm(x, residual, weight, eps):
    """(s, rstd float32, h float32) with the roundings of the definition; x and
    residual are float arrays that hold bf16 values, s is one too."""
    s = np.asarray(x, dtype=np.float32)
    if residual is not None:
        s = round_bf16(s + np.asarray(residual, dtype=np.float32))
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        mean = np.mean(np.square(s.astype(np.float64)), axis=-1)
        rstd = (1.0 / np.sqrt(mean + np.float64(np.float32(eps)))).astype(np.float32)
        h = (s * rstd[:, None]) * np.asarray(weight, dtype=np.float32)
    return s, rstd, h


def round_bf16(v):
    """float32 rounded to nearest even bf16, as float32 (NaN kept)."""
    v = np.asarray(v, dtype=np.float32)
    b = v.view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(v), np.float32(np.nan), r)


def add_rmsnorm_backward(dh, s, weight, rstd, ds=None):
    """(dx, dweight) float64: the gradient of h = s rstd(s) weight, rstd given."""
    z, r = np.asarray(s, dtype=np.float64), np.asarray(rstd, dtype=np.float64)[:, None]
    g = np.asarray(dh, dtype=np.float64) * np.asarray(weight, dtype=np.float64)
    dx = r * g - z * r ** 3 * np.mean(g * z, axis=-1, keepdims=True)
    if ds is not None:
        dx = dx + np.asarray(ds, dtype=np.float64)
    return dx, np.sum(np.asarray(dh, dtype=np.float64) * z * r, axis=0)
