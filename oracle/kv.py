"""The NVFP4 key/value cache and attention over it: the CPU oracle.

Test infrastructure only (see ``oracle/__init__.py``).

K1 Rotation: for a pair (a, b) of a head's first rope_dim elements and its
   position's cosine c and sine s, a' = fl32(fl32(a c) - fl32(b s)) and b' =
   fl32(fl32(b c) + fl32(a s)); pairs (i, i + rope_dim / 2), or (2 i, 2 i + 1)
   if interleaved.
K2 Quantization: the activations' contract (A2 of ``w4a4``) along head_dim,
   with the head's scale in the place of the tensor's.  A head's key and value
   of a token are both NaN if either holds an infinity or a NaN.
K3 out = sum_j p_j v_j / sum_j p_j, lse = log sum_j p_j, p_j = exp(scale q.k_j)
   over the visible tokens; nothing visible: 0 and -inf.
"""

from __future__ import annotations

import numpy as np

from .codecs import E2M1_MAG_VALUES, e4m3_decode, e4m3_encode
from .fos import BLOCK, E4M3_MAX, _candidate

F32 = np.float32


def rotate(x, positions, rope, interleaved) -> np.ndarray:
    """K1 of float32 x [tokens, heads, d]; rope float32 [positions, rope_dim]."""
    x = np.array(x, dtype=F32)
    half = rope.shape[1] // 2
    c, s = rope[positions][:, None, :half], rope[positions][:, None, half:]
    i = np.arange(half)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[..., first], x[..., second]
    out = x.copy()
    out[..., first] = a * c - b * s
    out[..., second] = b * c + a * s
    return out


def quantize(x, scale) -> np.ndarray:
    """K2's values, float32, of finite float32 x [tokens, heads, d] with scale float32 [heads]."""
    out = np.empty_like(x, dtype=F32)
    t, _, d = x.shape
    for h, st in enumerate(scale):
        xb = np.ascontiguousarray(x[:, h], dtype=F32).reshape(t, d // BLOCK, BLOCK)
        a = np.max(np.abs(xb), axis=-1) if t else np.zeros((t, d // BLOCK), F32)
        code, _ = e4m3_encode(np.minimum(a / (F32(6.0) * st), E4M3_MAX))
        sigma = e4m3_decode(code).astype(F32)
        mag, _ = _candidate(xb, sigma, st)
        v = E2M1_MAG_VALUES.astype(F32)[mag] * sigma[..., None]  # exact
        out[:, h] = (np.where(np.signbit(xb), -v, v) * st).reshape(t, d)
    return out


def cached(k, v, k_scale, v_scale):
    """K2 of keys (rotated) and values: what the cache holds for them."""
    bad = ~(np.isfinite(k).all(-1) & np.isfinite(v).all(-1))
    kz, vz = np.where(bad[..., None], F32(0), k), np.where(bad[..., None], F32(0), v)
    kq, vq = quantize(kz, k_scale), quantize(vz, v_scale)
    kq[bad], vq[bad] = np.nan, np.nan
    return kq, vq


def visible(n, new, causal=True, window=0) -> np.ndarray:
    """bool [new, n]: which tokens the last `new` of n see."""
    i = np.arange(n - new, n)[:, None]
    j = np.arange(n)[None]
    if not causal:
        return np.ones((new, n), bool)
    return (j <= i) & (j > i - window) if window else np.broadcast_to(j <= i, (new, n))


def attention(q, k, v, scale, seen):
    """K3 in float64 of q [new, q_heads, d] over k, v [n, heads, d].

    Returns out, lse and, for error bounds, weight = sum p |v| / sum p and
    size = the largest scale * sum |q| |k| of a row's visible tokens."""
    new, q_heads, d = q.shape
    group = q_heads // k.shape[1]
    out, weight = np.zeros((new, q_heads, d)), np.zeros((new, q_heads, d))
    lse, size = np.full((new, q_heads), -np.inf), np.zeros((new, q_heads))
    for h in range(q_heads):
        kh, vh = k[:, h // group].astype(np.float64), v[:, h // group].astype(np.float64)
        w = scale * (q[:, h].astype(np.float64) @ kh.T)
        big = abs(scale) * (np.abs(q[:, h].astype(np.float64)) @ np.abs(kh).T)
        for i in range(new):
            at = seen[i]
            if not at.any():
                continue
            top = w[i, at].max()
            p = np.exp(w[i, at] - top)
            out[i, h] = p @ vh[at] / p.sum()
            weight[i, h] = p @ np.abs(vh[at]) / p.sum()
            lse[i, h] = top + np.log(p.sum())
            size[i, h] = big[i, at].max()
    return out, lse, weight, size
