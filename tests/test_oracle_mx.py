"""Pins of oracle/mx.py against things other than itself: torch's E4M3 cast,
brute force over all codes, exact powers of two, finite differences."""

import numpy as np
import pytest
import torch

import oracle.mx as mx
from mx_cases import rows, special_rows


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_fp8_elements_are_torchs_cast(dtype):
    x = torch.cat([rows(40, 64, 1, dtype), special_rows(dtype)])
    c, s = mx.quantize_mx(x.double().numpy(), mx.FP8)
    ok = s != 255
    v = x.double().numpy().reshape(-1, 2, 32) / np.ldexp(1.0, np.where(ok, s, 127).astype(int) - 127)[..., None]
    v = torch.from_numpy(np.where(ok[..., None], v, 0.0)).clamp(-448, 448).float()
    want = v.to(torch.float8_e4m3fn).view(torch.uint8).numpy().reshape(c.shape)
    keep = np.repeat(ok, 32, axis=-1)
    assert np.array_equal(c[keep], want[keep])
    assert np.all(c[~keep] == 0)


def test_fp4_elements_are_the_nearest_of_all_codes():
    x = rows(30, 64, 2, torch.float32).double().numpy()
    c, s = mx.quantize_mx(x, mx.FP4)
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    v = np.abs(x) / np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=-1)
    d = np.abs(v[..., None] - grid)
    best = d.min(-1)
    took = np.take_along_axis(d, (c & 7).astype(int)[..., None], -1)[..., 0]
    assert np.array_equal(took, best)
    tie = (d == best[..., None]).sum(-1) > 1
    assert tie.any() and np.all((c & 7)[tie] % 2 == 0)
    assert np.array_equal((c & 8) != 0, np.signbit(x))


@pytest.mark.parametrize("fmt,top", [(mx.FP4, 4.0), (mx.FP8, 256.0)])
def test_scale_puts_the_maximum_into_the_top_binade(fmt, top):
    x = rows(30, 64, 3, torch.float32, 30).double().numpy()
    _, s = mx.quantize_mx(x, fmt)
    a = np.abs(x).reshape(30, 2, 32).max(-1)
    q = a / np.ldexp(1.0, s.astype(int) - 127)
    assert np.all((q[a > 0] >= top) & (q[a > 0] < 2 * top))
    # zeros, NaN and infinity, subnormals
    sp = special_rows(torch.float32).double().numpy()
    _, s = mx.quantize_mx(sp, fmt)
    assert np.all(s[0] == 0) and s[1, 0] == 255 and s[1, 1] == 0 and s[2, 1] == 255 and s[3, 0] == 255
    assert np.all(s[4] == 0) and s[13, 1] == 255


@pytest.mark.parametrize("fmt", [mx.FP4, mx.FP8])
def test_representable_values_round_trip(fmt):
    g = np.random.default_rng(4)
    mags = mx._magnitudes(fmt)
    v = mags[g.integers(0, len(mags), (20, 64))] * np.where(g.random((20, 64)) < 0.5, -1, 1)
    v[:, ::32] = mags[-1]  # the block's maximum in the top binade
    v *= np.repeat(2.0 ** g.integers(-60, 60, (20, 2)), 32, axis=-1)
    c, s = mx.quantize_mx(v, fmt)
    assert np.array_equal(mx.dequant_mx(mx.pack(c, fmt), s, fmt), v)


def test_norm_gradient_is_the_difference_quotient():
    g = np.random.default_rng(5)
    m, k, eps = 3, 64, 1e-3
    s, w = g.standard_normal((m, k)), 1 + 0.3 * g.standard_normal(k)
    dh, ds = g.standard_normal((m, k)), g.standard_normal((m, k))

    def loss(s, w):
        r = 1 / np.sqrt(np.mean(s * s, -1, keepdims=True) + eps)
        return np.sum(dh * s * r * w) + np.sum(ds * s)

    rstd = 1 / np.sqrt(np.mean(s * s, -1) + eps)
    dx, dw = mx.add_rmsnorm_backward(dh, s, w, rstd, ds)
    step = 1e-6
    for i, j in [(0, 0), (1, 17), (2, 63), (0, 31)]:
        d = np.zeros_like(s)
        d[i, j] = step
        assert abs((loss(s + d, w) - loss(s - d, w)) / (2 * step) - dx[i, j]) < 1e-7
        d = np.zeros_like(w)
        d[j] = step
        assert abs((loss(s, w + d) - loss(s, w - d)) / (2 * step) - dw[j]) < 1e-7


def test_round_bf16_is_torchs():
    x = np.concatenate([np.random.default_rng(6).standard_normal(1000) * 1e3, [0.0, -0.0, np.inf, 1e-40, 3e38]]).astype(np.float32)
    assert np.array_equal(mx.round_bf16(x).view(np.uint32), torch.from_numpy(x).bfloat16().float().numpy().view(np.uint32))
