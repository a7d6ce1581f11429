"""Inputs and tolerances shared by the microscaled operators' tests."""

import numpy as np
import torch

import oracle.mx as mx

U32, UBF16 = 2.0 ** -24, 2.0 ** -8  # half a rounding step, relative


def rows(m, k, seed, dtype=torch.bfloat16, spread=8):
    """[m, k] values whose blocks of 32 differ in size by up to 2^spread, with zeros, signed zeros and exact ties."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((m, k)) * np.repeat(2.0 ** g.integers(-spread, spread + 1, (m, k // 32)), 32, axis=-1)
    x[g.random((m, k)) < 0.03] = 0.0
    x[g.random((m, k)) < 0.02] *= -0.0
    x = np.where(g.random((m, k)) < 0.1, np.sign(x) * 2.0 ** np.round(np.log2(np.abs(x) + 1e-30)) * 1.25, x)
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def special_rows(dtype):
    """Rows that hold what a quantizer can get wrong: all zeros, one infinity or
    NaN in a block, subnormals, the largest finite values, block maxima on both
    sides of a power of two, values that saturate, and every rounding midpoint."""
    tiny = 2.0 ** -133 if dtype == torch.bfloat16 else 2.0 ** -149
    top = float(torch.finfo(dtype).max)
    r = np.zeros((14, 64), dtype=np.float64)
    r[1, 3] = np.inf
    r[2, 40] = -np.inf
    r[3, 7] = np.nan
    r[4] = tiny * np.arange(64)
    r[5] = 2.0 ** -126 * (np.arange(64) % 7 - 3)
    r[6] = top * np.where(np.arange(64) % 2, 1, -1)
    r[7, ::3] = top / 2
    r[8] = np.linspace(-7.96875, 7.96875, 64)
    r[9, :32] = np.repeat([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5], 4) * np.tile([1, -1, 1, -1], 8)
    r[9, 0] = 6.0
    r[9, 32:] = (np.arange(32) + 0.5) * 2.0 ** -9
    r[9, 32] = 448.0
    r[10, :32] = 256 + 8 + 16 * np.arange(32) % 256
    r[10, 32:] = 464.0
    r[11, 5] = 2.0 ** -120
    r[11, 36] = 1.9921875
    r[12] = -0.0
    r[13, 0], r[13, 1] = 2.0 ** 100, 2.0 ** -100
    r[13, 32:] = np.nan
    return torch.from_numpy(r.astype(np.float32)).to(dtype)


def weights(n, k, seed):
    """(stored codes, scales) of an MXFP4 [n, k] matrix, from the oracle."""
    c, s = mx.quantize_mx(rows(n, k, seed, torch.float32, 4).numpy(), mx.FP4)
    return mx.pack(c, mx.FP4), s


def product_bound(a, w, fmt, out_dtype):
    """(float64 a @ w.T, elementwise bound on the kernels' error).

    Products are exact.  Sums are in fp32: an output passes at most k / 8 + 64
    additions (the instruction's groups of 8, then waves or planes), each off by
    at most one step 2^-23 (two half steps: the instruction may cut instead of
    round) of a partial sum that is at most sum |products|.  MXFP8 with bf16 output adds the
    instruction's cut: 7 of each group's 8 products lose less than 2^-14 of
    the largest.  Then one rounding to the output."""
    ref, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    bound = (a.shape[1] / 8 + 64) * 2 * U32 * mag
    if fmt == mx.FP8 and out_dtype == torch.bfloat16:
        bound = bound + 7 * 2.0 ** -14 * mag
    half = UBF16 if out_dtype == torch.bfloat16 else U32
    return ref, bound * (1 + half) + half * np.abs(ref)


# (format of a, path, K split over workgroups, m, n, k): every kernel and tile of
# mx_gemm, whole and split, with remainders in m, n and k; for the tiles rows of
# n even, odd and a multiple of 8 (each stored its own way).  MXFP4 never splits
# the 256 tile.  test_mx_host.py holds the paths to the library's plan.
GEMM_PATHS = [
    (mx.FP4, 0, False, 5, 83, 992), (mx.FP4, 0, False, 13, 4131, 4640), (mx.FP4, 16, False, 1, 4215, 4096),
    (mx.FP4, 16, False, 15, 4200, 4096), (mx.FP4, 16, False, 16, 133, 4096), (mx.FP4, 16, False, 4, 4503, 4608),
    (mx.FP4, 16, False, 3, 70, 7680), (mx.FP4, 16, False, 5, 4100, 5120), (mx.FP4, 16, False, 16, 97, 14336),
    (mx.FP4, 64, False, 67, 131, 1056), (mx.FP4, 64, False, 142, 138, 96), (mx.FP4, 64, True, 50, 1715, 6592),
    (mx.FP4, 64, True, 20, 16, 2368), (mx.FP4, 128, False, 388, 4739, 1056), (mx.FP4, 128, False, 342, 5632, 1056),
    (mx.FP4, 128, False, 323, 5441, 32), (mx.FP4, 128, True, 17, 2103, 14880), (mx.FP4, 128, True, 66, 4104, 8320),
    (mx.FP4, 224, False, 1046, 7244, 1088), (mx.FP4, 224, False, 1951, 4231, 1056), (mx.FP4, 224, False, 1542, 5136, 1184),
    (mx.FP4, 224, True, 3345, 577, 15264), (mx.FP4, 224, True, 2421, 872, 16064), (mx.FP4, 256, False, 3862, 3659, 1056),
    (mx.FP4, 256, False, 2172, 6632, 1088), (mx.FP4, 256, False, 2278, 6394, 288),
    (mx.FP8, 0, False, 5, 83, 992), (mx.FP8, 0, False, 13, 4131, 4640), (mx.FP8, 16, False, 1, 4215, 4096),
    (mx.FP8, 16, False, 15, 4200, 4096), (mx.FP8, 16, False, 16, 133, 4096), (mx.FP8, 16, False, 4, 4503, 4608),
    (mx.FP8, 16, False, 3, 70, 7680), (mx.FP8, 16, False, 5, 4100, 5120), (mx.FP8, 16, False, 16, 97, 14336),
    (mx.FP8, 64, False, 67, 131, 1056), (mx.FP8, 64, False, 142, 138, 96), (mx.FP8, 64, True, 50, 1715, 6592),
    (mx.FP8, 64, True, 17, 16, 1888), (mx.FP8, 128, False, 1573, 1923, 1568), (mx.FP8, 128, False, 472, 6232, 1632),
    (mx.FP8, 128, False, 650, 4484, 1664), (mx.FP8, 128, True, 70, 2077, 9440), (mx.FP8, 128, True, 2068, 72, 11424),
    (mx.FP8, 224, False, 1860, 4474, 1056), (mx.FP8, 224, False, 1447, 5843, 1056), (mx.FP8, 224, False, 1215, 7176, 1088),
    (mx.FP8, 224, True, 4197, 69, 13216), (mx.FP8, 224, True, 585, 784, 16032), (mx.FP8, 256, False, 3862, 3659, 1056),
    (mx.FP8, 256, False, 2615, 5320, 1056), (mx.FP8, 256, True, 262, 3826, 11808), (mx.FP8, 256, True, 271, 4016, 13632),
]
# (tile, n split over workgroups, m, n, k) of mx_gemm_dx; rows of dy that are no whole 16-byte pieces have a kernel of their own
DX_PATHS = [
    (128, False, 129, 264, 96), (128, False, 300, 331, 2080), (128, False, 600, 72, 4128), (128, True, 131, 1001, 1056),
    (128, True, 65, 4104, 4128), (128, True, 3, 2050, 64), (256, False, 1050, 776, 12192), (256, False, 2209, 904, 5472),
    (256, False, 1000, 1000, 14304), (256, True, 149, 6432, 8800), (256, True, 1246, 6072, 1568),
]
