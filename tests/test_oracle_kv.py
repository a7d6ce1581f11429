"""The key/value cache's oracle against other statements of the same things."""

import math

import numpy as np
import pytest
import torch

import oracle
import oracle.kv as okv
from kv_cases import rope_table


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,d", [(32, 64), (64, 64), (128, 128)])
def test_rotation_is_a_complex_product(rot, d, interleaved):
    rng = np.random.default_rng(rot)
    x = rng.standard_normal((5, 3, d)).astype(np.float32)
    pos = np.array([0, 1, 77, 4000, 12])
    table = rope_table(4096, rot)
    y = okv.rotate(x, pos, table, interleaved).astype(np.float64)
    z = x.astype(np.float64)[..., :rot]
    pairs = z.reshape(5, 3, rot // 2, 2) if interleaved else np.stack((z[..., : rot // 2], z[..., rot // 2:]), -1)
    angle = pos[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    w = (pairs[..., 0] + 1j * pairs[..., 1]) * np.exp(1j * angle)[:, None]
    got = y[..., :rot].reshape(5, 3, rot // 2, 2) if interleaved else np.stack((y[..., : rot // 2], y[..., rot // 2: rot]), -1)
    # the table, two products and a sum are rounded: 3 half steps of |x|
    assert np.abs(got[..., 0] - w.real).max() <= 4 * 2.0 ** -24 * np.abs(pairs).max() * 2
    assert np.abs(got[..., 1] - w.imag).max() <= 4 * 2.0 ** -24 * np.abs(pairs).max() * 2
    assert np.array_equal(y[..., rot:], x[..., rot:])
    assert np.array_equal(okv.rotate(x, np.zeros(5, int), table, interleaved), x)


def test_quantization_is_the_activations_with_a_head_scale():
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.standard_normal((6, 2, 64)).astype(np.float32)).bfloat16()
    scale = np.array([5.0, 2.5], np.float32) / np.float32(2688.0)
    got = okv.quantize(x.float().numpy(), scale)
    for h, amax in enumerate((5.0, 2.5)):
        r = oracle.quantize_act(x[:, h].contiguous(), amax)
        want = oracle.act_blockscaled(r) * r.tensor_scale
        assert r.tensor_scale == scale[h] and np.array_equal(got[:, h], want)


def test_poison():
    k, v = np.ones((3, 2, 64), np.float32), np.ones((3, 2, 64), np.float32)
    k[0, 1, 5], v[2, 0, 63] = np.inf, np.nan
    kq, vq = okv.cached(k, v, np.ones(2, np.float32), np.ones(2, np.float32))
    bad = np.zeros((3, 2), bool)
    bad[0, 1] = bad[2, 0] = True
    assert np.array_equal(np.isnan(kq).all(-1), bad) and np.array_equal(np.isnan(vq).any(-1), bad)


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 3), (False, 0)])
def test_attention_term_by_term(causal, window):
    rng = np.random.default_rng(5)
    n, new, d = 9, 4, 64
    q, k, v = (rng.standard_normal(s) for s in ((new, 4, d), (n, 2, d), (n, 2, d)))
    out, lse, weight, size = okv.attention(q, k, v, 0.3, okv.visible(n, new, causal, window))
    for i in range(new):
        at = n - new + i
        js = [j for j in range(n) if not causal or (j <= at and (not window or j > at - window))]
        for h in range(4):
            e = [math.exp(0.3 * sum(q[i, h, x] * k[j, h // 2, x] for x in range(d))) for j in js]
            assert lse[i, h] == pytest.approx(math.log(sum(e)), rel=1e-12)
            for x in (0, 17, 63):
                assert out[i, h, x] == pytest.approx(sum(a * v[j, h // 2, x] for a, j in zip(e, js)) / sum(e), rel=1e-9, abs=1e-12)
    # more new tokens than context: the first rows see nothing
    seen = okv.visible(2, 5)
    assert seen.sum(1).tolist() == [0, 0, 0, 1, 2]
    out, lse, _, _ = okv.attention(rng.standard_normal((5, 2, d)), k[:2], v[:2], 1.0, seen)
    assert (out[:3] == 0).all() and np.isneginf(lse[:3]).all() and np.isfinite(lse[3:]).all()
