"""GPU parity of the microscaled operators against the float64 oracle:
quantization, dequantization, the residual + RMS norm bit-exact; the products
and the norm's gradient within bounds on the sums' roundings."""

import numpy as np
import pytest
import torch

import bit_gemm_amd as nv
import oracle.mx as mx
from mx_cases import DX_PATHS, GEMM_PATHS, U32, UBF16, product_bound, rows, special_rows, weights

pytestmark = pytest.mark.gpu

FMTS = pytest.mark.parametrize("fmt", [nv.MXFP4, nv.MXFP8], ids=["fp4", "fp8"])
DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])


def _np(t):
    return t.double().cpu().numpy()


def _mx(stored, scales, fmt):
    return nv.MXTensor(torch.from_numpy(stored).cuda(), torch.from_numpy(scales).cuda(), fmt)


def _same_bits(a, b):
    """Equal fp32 bit patterns, any NaN equal to any other."""
    a, b = a.astype(np.float32), b.astype(np.float32)
    return np.array_equal(np.where(np.isnan(a), 0x7FC00000, a.view(np.uint32)), np.where(np.isnan(b), 0x7FC00000, b.view(np.uint32)))


@FMTS
@DTYPES
@pytest.mark.parametrize("m,k", [(1, 32), (3, 96), (2, 2048), (17, 1056), (130, 544), (1, 65568), (0, 64), (5, 0)])
def test_quantize_and_dequantize(fmt, dtype, m, k):
    print("mx quantize", fmt, dtype, m, k, flush=True)
    x = torch.cat([rows(m, k, 10 + m, dtype), special_rows(dtype)]) if k == 64 else rows(m, k, 10 + m, dtype)
    if m * k == 0:
        x = torch.zeros((m, k), dtype=dtype)
    q = nv.quantize_mx(x.cuda(), fmt)
    if m * k:
        c, s = mx.quantize_mx(x.double().numpy(), fmt)
        assert np.array_equal(q.scales.cpu().numpy(), s)
        assert np.array_equal(q.codes.cpu().numpy(), mx.pack(c, fmt))
        want = mx.dequant_mx(mx.pack(c, fmt), s, fmt).astype(np.float32)
        assert _same_bits(nv.dequant_mx(q).cpu().numpy(), want)
        assert _same_bits(nv.dequant_mx(q, torch.bfloat16).float().cpu().numpy(), mx.round_bf16(want))
    else:
        assert q.shape == (m, k) and nv.dequant_mx(q).shape == (m, k)


@FMTS
@DTYPES
def test_quantize_special_values(fmt, dtype):
    x = special_rows(dtype)
    q = nv.quantize_mx(x.cuda(), fmt)
    c, s = mx.quantize_mx(x.double().numpy(), fmt)
    assert np.array_equal(q.scales.cpu().numpy(), s)
    assert np.array_equal(q.codes.cpu().numpy(), mx.pack(c, fmt))


@FMTS
def test_dequantize_every_code_at_every_scale(fmt):
    # 256 rows, one per scale byte, holding every stored byte
    stored = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    per = stored.shape[1] * (2 if fmt == nv.MXFP4 else 1) // 32
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], per, axis=1)
    with np.errstate(over="ignore"):  # the largest scales pass fp32's range
        want = mx.dequant_mx(stored, scales, fmt).astype(np.float32)
    q = _mx(stored, scales, fmt)
    assert _same_bits(nv.dequant_mx(q).cpu().numpy(), want)
    assert _same_bits(nv.dequant_mx(q, torch.bfloat16).float().cpu().numpy(), mx.round_bf16(want))


def test_quantize_writes_only_its_rows():
    x = rows(5, 96, 3)
    for fmt in (nv.MXFP4, nv.MXFP8):
        big = nv.MXTensor.empty(9, 96, fmt, "cuda")
        big.codes.fill_(0xA5), big.scales.fill_(0x5A)
        part = nv.MXTensor(big.codes[:5], big.scales[:5], fmt)
        nv.quantize_mx(x.cuda(), fmt, out=part)
        assert bool((big.codes[5:] == 0xA5).all()) and bool((big.scales[5:] == 0x5A).all())
        assert torch.equal(part.codes, nv.quantize_mx(x.cuda(), fmt).codes)


# (m, n, k): one row; sizes around the 16-row tiles; k below, at and past one
# instruction's 128 and one wave's 512; odd sizes; many rows; more than one
# tile of every kind
PRODUCTS = [(1, 1, 32), (1, 17, 64), (2, 16, 96), (15, 33, 128), (16, 100, 160), (17, 64, 512), (33, 48, 544),
            (48, 31, 1056), (49, 16, 4128), (64, 272, 2048), (65, 64, 96), (100, 300, 1056), (129, 257, 320),
            (257, 129, 256), (300, 515, 4192), (1, 4096, 4096), (16, 1001, 14336), (130, 1024, 2048),
            (520, 1056, 1312), (64, 80, 33 * 512), (130, 90, 320), (300, 518, 288), (700, 2046, 160),
            (3, 4200, 4096), (16, 5000, 4096), (4, 700, 5120), (2, 4500, 4608), (9, 4500, 4608), (13, 50, 8192)]


@FMTS
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_gemm(fmt, m, n, k):
    print("mx gemm", fmt, m, n, k, flush=True)
    c, s = mx.quantize_mx(rows(m, k, 20 + m, torch.float32, 6).numpy(), fmt)
    wc, ws = weights(n, k, 21 + n)
    a, w = mx.dequant_mx(mx.pack(c, fmt), s, fmt), mx.dequant_mx(wc, ws, mx.FP4)
    qa, qw = _mx(mx.pack(c, fmt), s, fmt), _mx(wc, ws, nv.MXFP4)
    for dt in (torch.bfloat16, torch.float32):
        ref, bound = product_bound(a, w, fmt, dt)
        y = _np(nv.mx_gemm(qa, qw, out_dtype=dt))
        assert np.all(np.abs(y - ref) <= bound), (dt, float((np.abs(y - ref) / bound).max()))


@FMTS
@pytest.mark.parametrize("m,n,k", [(3500, 3700, 544), (2300, 5000, 1024), (4096, 4224, 2080), (3990, 4090, 1056),
                                   (2045, 7159, 544)])
def test_gemm_many_tiles(fmt, m, n, k):
    # enough outputs for every workgroup tile the library has; sampled rows against the oracle
    print("mx gemm", fmt, m, n, k, flush=True)
    g = torch.Generator(device="cuda").manual_seed(m)
    a = nv.quantize_mx(torch.randn(m, k, generator=g, device="cuda"), fmt)
    w = nv.quantize_mx(torch.randn(n, k, generator=g, device="cuda"))
    pick = np.unique(np.concatenate([[0, 31, 32, 63, 64, 127, 128, 255, 256, m - 1], np.random.default_rng(m).integers(0, m, 30)]))
    av = mx.dequant_mx(a.codes.cpu().numpy()[pick], a.scales.cpu().numpy()[pick], fmt)
    wv = mx.dequant_mx(w.codes.cpu().numpy(), w.scales.cpu().numpy(), mx.FP4)
    for dt in (torch.bfloat16, torch.float32):
        ref, bound = product_bound(av, wv, fmt, dt)
        y = _np(nv.mx_gemm(a, w, out_dtype=dt)[torch.from_numpy(pick).cuda()])
        assert np.all(np.abs(y - ref) <= bound), (dt, float((np.abs(y - ref) / bound).max()))


@FMTS
@pytest.mark.parametrize("m,n", [(7, 19), (70, 140), (300, 520)])
def test_gemm_exact_sums(fmt, m, n):
    # small codes and scales: every partial sum is an integer multiple of one
    # unit below 2^24 of them, so fp32 output has no rounding at all; every
    # element and block has its own value, so a misplaced operand shows
    g = np.random.default_rng(30 + m)
    k = 1312
    w = g.integers(-3, 4, (n, k)).astype(np.float32) * np.repeat(2.0 ** g.integers(0, 3, (n, k // 32)), 32, axis=-1)
    hi = 4 if fmt == nv.MXFP4 else 16
    a = g.integers(-hi + 1, hi, (m, k)).astype(np.float32) * np.repeat(2.0 ** g.integers(0, 3, (m, k // 32)), 32, axis=-1)
    (ac, as_), (wc, ws) = mx.quantize_mx(a, fmt), mx.quantize_mx(w, mx.FP4)
    av, wv = mx.dequant_mx(mx.pack(ac, fmt), as_, fmt), mx.dequant_mx(mx.pack(wc, mx.FP4), ws, mx.FP4)
    y = _np(nv.mx_gemm(_mx(mx.pack(ac, fmt), as_, fmt), _mx(mx.pack(wc, mx.FP4), ws, nv.MXFP4), out_dtype=torch.float32))
    assert np.array_equal(y, av @ wv.T)


@pytest.mark.parametrize("m,n", [(5, 40), (150, 300)])
def test_gemm_fp8_keeps_small_products_in_fp32(m, n):
    # each group of 8 holds one product of 448 * 6 and seven of 2^-9 * 0.5, and
    # the large ones cancel in pairs of groups: what is left is the small ones
    k = 512
    c = np.full((m, k), 0x01, dtype=np.uint8)
    c[:, 0::16], c[:, 8::16] = 0x7E, 0xFE
    wc = np.full((n, k), 0x1, dtype=np.uint8)
    wc[:, 0::8] = 0x7
    s = np.full((m, k // 32), 127, dtype=np.uint8)
    sw = np.full((n, k // 32), 127, dtype=np.uint8)
    y = nv.mx_gemm(_mx(c, s, nv.MXFP8), _mx(mx.pack(wc, mx.FP4), sw, nv.MXFP4), out_dtype=torch.float32)
    assert np.array_equal(_np(y), np.full((m, n), (k - k // 8) * 2.0 ** -10))


@FMTS
@pytest.mark.parametrize("m,n,k", [(3, 40, 160), (140, 300, 1056)])
def test_gemm_nan_blocks_reach_their_row_and_column_only(fmt, m, n, k):
    c, s = mx.quantize_mx(rows(m, k, 40, torch.float32, 2).numpy(), fmt)
    wc, ws = weights(n, k, 41)
    s[1, -1] = 255  # the last block of a row: what reads past the end must not spread it
    ws[n - 1, 0] = 255
    y = nv.mx_gemm(_mx(mx.pack(c, fmt), s, fmt), _mx(wc, ws, nv.MXFP4), out_dtype=torch.float32).cpu().numpy()
    want = np.zeros((m, n), dtype=bool)
    want[1], want[:, n - 1] = True, True
    assert np.array_equal(np.isnan(y), want)


@FMTS
def test_gemm_writes_only_its_output(fmt):
    for m, n in [(3, 17), (130, 300), (257, 259)]:
        k = 160
        c, s = mx.quantize_mx(rows(m, k, 50, torch.float32, 2).numpy(), fmt)
        qa, qw = _mx(mx.pack(c, fmt), s, fmt), _mx(*weights(n, k, 51), nv.MXFP4)
        for dt in (torch.bfloat16, torch.float32):
            big = torch.full((m * n + 4096,), 7.0, dtype=dt, device="cuda")
            y = nv.mx_gemm(qa, qw, out_dtype=dt, out=big[: m * n].view(m, n))
            assert bool((big[m * n:] == 7.0).all())
            assert torch.equal(y, nv.mx_gemm(qa, qw, out_dtype=dt))


@FMTS
@pytest.mark.parametrize("m,n", [(17, 5), (300, 70), (70000, 9)])
def test_gemm_over_nothing(fmt, m, n):
    a, w = (nv.quantize_mx(torch.zeros((r, 0), device="cuda"), f) for r, f in ((m, fmt), (n, nv.MXFP4)))
    for dt in (torch.bfloat16, torch.float32):
        y = nv.mx_gemm(a, w, out=torch.full((m, n), 7.0, dtype=dt, device="cuda"), out_dtype=dt)
        assert not bool(y.any())


def test_gemm_rows_longer_than_tiles_take():
    # k past the tiles' 32-bit offsets, more than 16 rows: the kernel of few rows in several groups.  Values 0,
    # 1/2, 1 of either sign: products are quarters, sums (random walks) stay far below 2^24 of them: exact in any order
    m, n, k = 17, 2, (1 << 22) + 32
    g = np.random.default_rng(26)
    code = np.array([0, 1, 2, 9, 10], dtype=np.uint8)
    ac, wc = (code[g.integers(0, 5, (r, k))] for r in (m, n))
    sa, sw = (np.full((r, k // 32), 127, dtype=np.uint8) for r in (m, n))
    a, w = mx.dequant_mx(mx.pack(ac, mx.FP4), sa, mx.FP4), mx.dequant_mx(mx.pack(wc, mx.FP4), sw, mx.FP4)
    y = _np(nv.mx_gemm(_mx(mx.pack(ac, mx.FP4), sa, nv.MXFP4), _mx(mx.pack(wc, mx.FP4), sw, nv.MXFP4),
                       out_dtype=torch.float32))
    assert np.array_equal(y, a @ w.T)


def test_gemm_empty():
    w = nv.quantize_mx(torch.zeros((6, 0), device="cuda"))
    y = nv.mx_gemm(nv.quantize_mx(torch.zeros((3, 0), device="cuda"), nv.MXFP8), w, out_dtype=torch.float32)
    assert y.shape == (3, 6) and float(y.abs().sum()) == 0.0
    w = nv.quantize_mx(torch.zeros((6, 64), device="cuda"))
    assert nv.mx_gemm(nv.quantize_mx(torch.zeros((0, 64), device="cuda")), w).shape == (0, 6)
    w0 = nv.quantize_mx(torch.zeros((0, 64), device="cuda"))
    assert nv.mx_gemm(nv.quantize_mx(torch.zeros((3, 64), device="cuda")), w0).shape == (3, 0)


@pytest.mark.parametrize("m,n,k", [(1, 64, 128), (17, 100, 96), (128, 256, 256), (300, 1001, 1056), (64, 4096, 1024),
                                   (5, 33, 32), (200, 1024, 384), (130, 72, 160), (3, 8, 32), (257, 584, 1312)])
def test_gemm_dx(m, n, k):
    print("mx gemm_dx", m, n, k, flush=True)
    wc, ws = weights(n, k, 60 + n)
    w = mx.dequant_mx(wc, ws, mx.FP4)
    dy = rows(m, 32 * ((n + 31) // 32), 61 + m, torch.bfloat16, 2)[:, :n].contiguous()
    d = dy.double().numpy()
    for dt, half in ((torch.bfloat16, UBF16), (torch.float32, U32)):
        # bf16 x bf16 products are exact, at most n + 64 fp32 additions per output, one rounding
        ref, mag = d @ w, np.abs(d) @ np.abs(w)
        bound = (n + 64) * 2 * U32 * mag * (1 + half) + half * np.abs(ref)
        y = _np(nv.mx_gemm_dx(dy.cuda(), _mx(wc, ws, nv.MXFP4), out_dtype=dt))
        assert np.all(np.abs(y - ref) <= bound), dt


@pytest.mark.parametrize("m,n,k", [(3500, 520, 3700 // 32 * 32), (4096, 64, 4128), (2600, 1000, 4096)])
def test_gemm_dx_many_tiles(m, n, k):
    # enough outputs for the large tile; sampled rows against the oracle
    print("mx gemm_dx", m, n, k, flush=True)
    g = torch.Generator(device="cuda").manual_seed(m)
    dy = torch.randn(m, n, generator=g, device="cuda").bfloat16()
    w = nv.quantize_mx(torch.randn(n, k, generator=g, device="cuda"))
    wv = mx.dequant_mx(w.codes.cpu().numpy(), w.scales.cpu().numpy(), mx.FP4)
    pick = np.unique(np.concatenate([[0, 31, 32, 127, 128, 255, 256, m - 1], np.random.default_rng(m).integers(0, m, 30)]))
    d = _np(dy[torch.from_numpy(pick).cuda()])
    ref, mag = d @ wv, np.abs(d) @ np.abs(wv)
    for dt, half in ((torch.bfloat16, UBF16), (torch.float32, U32)):
        bound = (n + 64) * 2 * U32 * mag * (1 + half) + half * np.abs(ref)
        y = _np(nv.mx_gemm_dx(dy, w, out_dtype=dt)[torch.from_numpy(pick).cuda()])
        assert np.all(np.abs(y - ref) <= bound), dt


def test_gemm_dx_rows_and_empty():
    # one-hot gradients give the weights' rows exactly; scales span the format, a NaN scale stays in its block
    n, k = 128, 256
    g = np.random.default_rng(62)
    wc = g.integers(0, 256, (n, k // 2)).astype(np.uint8)
    ws = g.integers(0, 252, (n, k // 32)).astype(np.uint8)
    w = mx.dequant_mx(wc, ws, mx.FP4).astype(np.float32)
    for rows_ in (n, n - 3, n - 8):  # every kernel: whole 64-row steps or not, rows of dy of whole 16 bytes or not
        dx = nv.mx_gemm_dx(torch.eye(rows_, device="cuda").bfloat16(), _mx(wc[:rows_], ws[:rows_], nv.MXFP4),
                           out_dtype=torch.float32).cpu().numpy()
        assert np.array_equal(dx, w[:rows_])
    ws[5, 2] = 255
    dx = nv.mx_gemm_dx(torch.ones((2, n), device="cuda").bfloat16(), _mx(wc, ws, nv.MXFP4), out_dtype=torch.float32)
    bad = np.zeros((2, k), dtype=bool)
    bad[:, 64:96] = True
    assert np.array_equal(np.isnan(dx.cpu().numpy()), bad)
    w0 = nv.quantize_mx(torch.zeros((0, 64), device="cuda"))
    z = nv.mx_gemm_dx(torch.zeros((3, 0), device="cuda").bfloat16(), w0, out_dtype=torch.float32)
    assert z.shape == (3, 64) and float(z.abs().sum()) == 0.0


def _norm_inputs(m, k, seed, wdtype, residual):
    x = rows(m, k, seed, torch.bfloat16, 3)
    r = rows(m, k, seed + 1, torch.bfloat16, 3) if residual else None
    w = (1.0 + 0.2 * torch.randn(k, generator=torch.Generator().manual_seed(seed))).to(wdtype)
    return x, r, w


def _check_norm(x, r, w, eps, fmt):
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    h, s, rstd = nv.add_rmsnorm_mx(cu(x), cu(w), residual=cu(r), eps=eps, fmt=fmt)
    want_s, want_r, want_h = mx.add_rmsnorm(x.float().numpy(), None if r is None else r.float().numpy(), w.float().numpy(), eps)
    assert _same_bits(s.float().cpu().numpy(), want_s)
    assert _same_bits(rstd.cpu().numpy(), want_r)
    c, sc = mx.quantize_mx(want_h, fmt)
    assert np.array_equal(h.scales.cpu().numpy(), sc)
    assert np.array_equal(h.codes.cpu().numpy(), mx.pack(c, fmt))


# k at and around every number of threads and pieces per row
NORMS = [(1, 32), (5, 96), (3, 512), (7, 544), (2, 2048), (3, 2080), (4, 4096), (3, 4128), (2, 8192), (2, 11008),
         (2, 16384), (2, 16416), (1, 32768), (1, 32800), (1, 65536), (1030, 64), (600, 1056)]


@FMTS
@pytest.mark.parametrize("m,k", NORMS)
def test_norm(fmt, m, k):
    print("norm", fmt, m, k, flush=True)
    for residual, wdtype in ((True, torch.bfloat16), (False, torch.float32)):
        _check_norm(*_norm_inputs(m, k, 70 + m, wdtype, residual), 1e-6, fmt)


@FMTS
@pytest.mark.parametrize("k", [64, 4096])
def test_norm_special_rows(fmt, k):
    x = special_rows(torch.bfloat16).repeat(1, k // 64)
    w = torch.ones(k)
    w[3], w[7] = 0.0, -2.0
    with np.errstate(all="ignore"):
        for eps in (1e-6, 0.0, 1.0):  # eps = 0: a row of zeros has no norm and comes out as NaN
            _check_norm(x, None, w, eps, fmt)
        _check_norm(x, x.flip(0).contiguous(), w, 1e-6, fmt)  # infinity + -infinity, overflow of the sum


def test_norm_in_place_and_guards():
    x, r, w = _norm_inputs(6, 1056, 80, torch.bfloat16, True)
    h, s, rstd = nv.add_rmsnorm_mx(x.cuda(), w.cuda(), residual=r.cuda())
    for which in ("residual", "x"):
        xd, rd = x.cuda(), r.cuda()
        big = nv.MXTensor.empty(8, 1056, nv.MXFP8, "cuda")
        big.codes.fill_(0xA5), big.scales.fill_(0x5A)
        rs = torch.full((8,), 3.0, device="cuda")
        h2, s2, r2 = nv.add_rmsnorm_mx(xd, w.cuda(), residual=rd, residual_out=rd if which == "residual" else xd,
                                       out=nv.MXTensor(big.codes[:6], big.scales[:6], nv.MXFP8), rstd=rs[:6])
        assert s2.data_ptr() == (rd if which == "residual" else xd).data_ptr()
        assert torch.equal(s2, s) and torch.equal(r2, rstd) and torch.equal(h2.codes, h.codes) and torch.equal(h2.scales, h.scales)
        assert bool((big.codes[6:] == 0xA5).all()) and bool((big.scales[6:] == 0x5A).all()) and bool((rs[6:] == 3.0).all())
    h, s, rstd = nv.add_rmsnorm_mx(x[:0].cuda(), w.cuda())
    assert h.shape == (0, 1056) and rstd.shape == (0,)


@pytest.mark.parametrize("m,k", [(1, 32), (5, 96), (3, 512), (7, 544), (2, 2080), (1200, 64), (700, 1056), (4, 4096),
                                 (3, 11008), (2, 16416), (2, 32800), (3, 65536)])
def test_norm_backward(m, k):
    print("norm backward", m, k, flush=True)
    for with_ds, wdtype in ((True, torch.float32), (False, torch.bfloat16)):
        x, _, w = _norm_inputs(m, k, 90 + m, wdtype, False)
        dh, ds = rows(m, k, 91 + m, torch.bfloat16, 2), rows(m, k, 92 + m, torch.bfloat16, 2)
        _, s, rstd = nv.add_rmsnorm_mx(x.cuda(), w.cuda())
        dx, dw = nv.add_rmsnorm_backward(dh.cuda(), s, w.cuda(), rstd, ds=ds.cuda() if with_ds else None)
        z, r = x.double().numpy(), _np(rstd)
        g = dh.double().numpy() * w.double().numpy()
        ref_dx, ref_dw = mx.add_rmsnorm_backward(dh.double().numpy(), z, w.double().numpy(), r,
                                                 ds.double().numpy() if with_ds else None)
        # xhat, g: one rounding each; the row's sum: at most 8 pieces of 8 per thread, 6 shuffles, 16 waves, the
        # division, on terms with 2 roundings; then 3 roundings of terms that large, and one to bf16
        xh = np.abs(z * r[:, None])
        c = np.mean(np.abs(g) * xh, -1, keepdims=True)
        size = r[:, None] * (np.abs(g) + xh * c)
        bound = (64 + 6 + 16 + 8) * U32 * size + 2 * U32 * np.abs(ref_dx)
        if with_ds:
            bound = bound + U32 * np.abs(ds.double().numpy())
        bound = bound * (1 + UBF16) + UBF16 * np.abs(ref_dx)
        assert np.all(np.abs(_np(dx) - ref_dx) <= bound)
        # a column's sum over m rows: one rounding per row and per partial sum, two in each term
        bound = (m + 600) * U32 * np.sum(np.abs(dh.double().numpy()) * xh, axis=0)
        assert np.all(np.abs(_np(dw) - ref_dw) <= bound)


def test_norm_backward_in_place_and_empty():
    x, _, w = _norm_inputs(9, 544, 95, torch.float32, False)
    dh, ds = rows(9, 544, 96), rows(9, 544, 97)
    _, s, rstd = nv.add_rmsnorm_mx(x.cuda(), w.cuda())
    dx, dw = nv.add_rmsnorm_backward(dh.cuda(), s, w.cuda(), rstd, ds=ds.cuda())
    buf = ds.cuda()
    dx2, dw2 = nv.add_rmsnorm_backward(dh.cuda(), s, w.cuda(), rstd, ds=buf, dx=buf)
    assert dx2.data_ptr() == buf.data_ptr() and torch.equal(dx, dx2) and torch.equal(dw, dw2)
    e = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    dw = torch.full((64,), 5.0, device="cuda")
    dx, dw = nv.add_rmsnorm_backward(e, e, torch.ones(64, device="cuda"), torch.zeros(0, device="cuda"), dweight=dw)
    assert dx.shape == (0, 64) and float(dw.abs().sum()) == 0.0


def _layer(x, r, wn, w1, w2):
    """A decoder block's MLP half as it is served: norm, product, quantize, product."""
    h, s, rstd = nv.add_rmsnorm_mx(x, wn, residual=r)
    u = nv.mx_gemm(h, w1)
    y = nv.mx_gemm(nv.quantize_mx(u, nv.MXFP4), w2)
    return h, s, rstd, u, y


@pytest.mark.parametrize("m", [1, 40, 200])
def test_operators_together(m):
    k, n = 512, 1056
    x, r, wn = _norm_inputs(m, k, 100, torch.bfloat16, True)
    w1, w2 = (weights(n, k, 101), weights(k, n, 102))
    q1, q2 = _mx(*w1, nv.MXFP4), _mx(*w2, nv.MXFP4)
    h, s, rstd, u, y = _layer(x.cuda(), r.cuda(), wn.cuda(), q1, q2)
    # each product against the oracle on the operands the step before it wrote
    hv = mx.dequant_mx(h.codes.cpu().numpy(), h.scales.cpu().numpy(), mx.FP8)
    ref, bound = product_bound(hv, mx.dequant_mx(*w1, mx.FP4), mx.FP8, torch.bfloat16)
    assert np.all(np.abs(_np(u) - ref) <= bound)
    c, sc = mx.quantize_mx(_np(u), mx.FP4)
    ref, bound = product_bound(mx.dequant_mx(mx.pack(c, mx.FP4), sc, mx.FP4), mx.dequant_mx(*w2, mx.FP4), mx.FP4, torch.bfloat16)
    assert np.all(np.abs(_np(y) - ref) <= bound)
    # backward: through the second product, the first, the norm
    dy = rows(m, k, 103, torch.bfloat16, 1).cuda()
    du = nv.mx_gemm_dx(dy, q2)
    dh = nv.mx_gemm_dx(du, q1)
    dx, dw = nv.add_rmsnorm_backward(dh, s, wn.cuda(), rstd, ds=dy)
    ref_dh = _np(du) @ mx.dequant_mx(*w1, mx.FP4)
    mag = np.abs(_np(du)) @ np.abs(mx.dequant_mx(*w1, mx.FP4))
    assert np.all(np.abs(_np(dh) - ref_dh) <= (n + 64) * 2 * U32 * mag * (1 + UBF16) + UBF16 * np.abs(ref_dh))
    assert dx.shape == (m, k) and bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all())


def test_captured_and_replayed_on_another_stream():
    m, k, n = 33, 512, 1056
    x, r, wn = _norm_inputs(m, k, 110, torch.bfloat16, True)
    q1, q2 = _mx(*weights(n, k, 111), nv.MXFP4), _mx(*weights(k, n, 112), nv.MXFP4)
    xd, rd, wd = x.cuda(), r.cuda(), wn.cuda()

    def step():
        h, s, rstd, u, y = _layer(xd, rd, wd, q1, q2)
        dh = nv.mx_gemm_dx(nv.mx_gemm_dx(y, q2), q1)
        return [h.codes, h.scales, s, rstd, u, y, dh, *nv.add_rmsnorm_backward(dh, s, wd, rstd, ds=y)]

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = step()
    for seed in (1, 2, 3):
        x2, r2, _ = _norm_inputs(m, k, 120 + seed, torch.bfloat16, True)
        xd.copy_(x2), rd.copy_(r2)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in got]
        for a, b in zip(replayed, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_calls_at_once_on_two_streams():
    # every operator under way on both streams at one time, own buffers each: the results of calls one by one
    x = [rows(m, 4096, 140 + m, torch.bfloat16, 3).cuda() for m in (3, 700)]
    w = _mx(*weights(600, 4096, 141), nv.MXFP4)
    gain = torch.ones(4096, device="cuda")

    def chain(x):
        h, s, rstd = nv.add_rmsnorm_mx(x, gain, residual=x)
        y = nv.mx_gemm(h, w)
        dh = nv.mx_gemm_dx(y, w)
        return [h.codes, y, nv.dequant_mx(nv.quantize_mx(y[:, :544].contiguous())), dh,
                *nv.add_rmsnorm_backward(dh, s, gain, rstd, ds=x)]

    want = [chain(t) for t in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    got = [[], []]
    for _ in range(4):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(chain(x[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(run, want[i]))


@pytest.mark.parametrize("m,k", [(16, 4096), (40, 1056)])
def test_gemm_of_a_matrix_with_itself(m, k):
    q = _mx(*weights(m, k, 150), nv.MXFP4)
    v = mx.dequant_mx(q.codes.cpu().numpy(), q.scales.cpu().numpy(), mx.FP4)
    ref, bound = product_bound(v, v, mx.FP4, torch.float32)
    assert np.all(np.abs(_np(nv.mx_gemm(q, q, out_dtype=torch.float32)) - ref) <= bound)


def test_refuses_views_off_sixteen_bytes():
    flat = torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    x, odd = flat[8:].view(4, 64), flat[4:-4].view(4, 64)
    w = nv.quantize_mx(x)
    for call in (lambda: nv.quantize_mx(odd), lambda: nv.add_rmsnorm_mx(odd, torch.ones(64, device="cuda")),
                 lambda: nv.mx_gemm(w, w, out=torch.zeros(24, device="cuda").bfloat16()[4:20].view(4, 4)),
                 lambda: nv.mx_gemm_dx(flat[4:20].view(4, 4), w)):
        with pytest.raises(RuntimeError, match="aligned"):
            call()
    assert nv.quantize_mx(x).shape == (4, 64)


def test_large_offsets():
    # codes past 2^31 bytes: a [m, k] MXFP8 matrix of 2.2e9 elements, its last rows against the oracle
    m, k = 33600, 65536
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    tail = rows(3, k, 130)
    x[-3:] = tail.cuda()
    q = nv.quantize_mx(x, nv.MXFP8)
    c, s = mx.quantize_mx(tail.double().numpy(), mx.FP8)
    assert np.array_equal(q.codes[-3:].cpu().numpy(), c) and np.array_equal(q.scales[-3:].cpu().numpy(), s)
    assert not bool(q.codes[:64].any())
    v = nv.dequant_mx(q, torch.bfloat16)
    assert torch.equal(v[-3:].cpu().float(), torch.from_numpy(mx.dequant_mx(c, s, mx.FP8)).float())
    del v
    w = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    h, _, rstd = nv.add_rmsnorm_mx(x, w)
    _, want_r, want_h = mx.add_rmsnorm(tail.float().numpy(), None, np.ones(k), 1e-6)
    c, s = mx.quantize_mx(want_h, mx.FP8)
    assert np.array_equal(h.codes[-3:].cpu().numpy(), c) and np.array_equal(h.scales[-3:].cpu().numpy(), s)
    # the last activation rows of a product
    wc, ws = weights(40, k, 131)
    y = nv.mx_gemm(nv.MXTensor(h.codes, h.scales, nv.MXFP8), _mx(wc, ws, nv.MXFP4), out_dtype=torch.float32)
    ref, bound = product_bound(mx.dequant_mx(c, s, mx.FP8), mx.dequant_mx(wc, ws, mx.FP4), mx.FP8, torch.float32)
    assert np.all(np.abs(_np(y[-3:]) - ref) <= bound)
    dx, _ = nv.add_rmsnorm_backward(x, x, w, rstd)
    z, r = tail.double().numpy(), _np(rstd[-3:])
    ref, _ = mx.add_rmsnorm_backward(z, z, np.ones(k), r)
    size = r[:, None] * (np.abs(z) + np.abs(z * r[:, None]) * np.mean(z * z, -1, keepdims=True) * r[:, None])
    assert np.all(np.abs(_np(dx[-3:]) - ref) <= (94 * U32 * size) * (1 + UBF16) + (UBF16 + 2 * U32) * np.abs(ref))


# every kernel of few rows (k below 4096, at it with many weight rows, past it in whole chunks of 512 or not) and tiles
@pytest.mark.parametrize("m,n,k", [(5, 40, 512), (5, 40, 4128), (3, 4200, 4096), (4, 70, 5120), (9, 45, 8192),
                                   (150, 300, 512), (700, 2046, 1056)])
def test_gemm_fp8_drops_nothing_in_either_output_type(m, n, k):
    # every group of 8 is led by +-448 * 6, which cancels over two groups; the other seven codes lie anywhere between
    # 2^-9 and 16.  All products are whole multiples of 2^-10 and the sums stay below 2^14: fp32 holds each of them
    # exactly in any order, and a bf16 output is the exact sum rounded once
    g = np.random.default_rng(160 + m)
    c = (g.integers(1, 0x51, (m, k)) | g.integers(0, 2, (m, k)) << 7).astype(np.uint8)
    c[:, 0::16], c[:, 8::16] = 0x7E, 0xFE
    wc = (g.integers(0, 2, (n, k)) * 2 + 1 | g.integers(0, 2, (n, k)) << 3).astype(np.uint8)  # +-0.5, +-1.5
    wc[:, 0::8] = 0x7
    s, ws = np.full((m, k // 32), 127, dtype=np.uint8), np.full((n, k // 32), 127, dtype=np.uint8)
    ref = mx.dequant_mx(c, s, mx.FP8) @ mx.dequant_mx(mx.pack(wc, mx.FP4), ws, mx.FP4).T
    a, w = _mx(c, s, nv.MXFP8), _mx(mx.pack(wc, mx.FP4), ws, nv.MXFP4)
    assert np.array_equal(_np(nv.mx_gemm(a, w, out_dtype=torch.float32)), ref)
    assert np.array_equal(_np(nv.mx_gemm(a, w)), mx.round_bf16(ref.astype(np.float32)).astype(np.float64))


def _exact_mx(rows_, k, fmt, gen):
    """Random elements (all E2M1 codes; E4M3 codes of 1/8 up to 15) with scales 1/2 and 1: a product of two such
    matrices has products of whole multiples of 2^-9, at most 90, and sums that stay far below 2^24 of those (random
    walks of at most 16064 steps of 10 in the mean): fp32 holds every partial sum in any order."""
    if fmt == nv.MXFP4:
        codes = torch.randint(0, 256, (rows_, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
    else:
        codes = torch.randint(0x20, 0x58, (rows_, k), generator=gen, device="cuda", dtype=torch.uint8)
        codes = codes | torch.randint(0, 2, (rows_, k), generator=gen, device="cuda", dtype=torch.uint8) << 7
    return nv.MXTensor(codes, torch.randint(126, 128, (rows_, k // 32), generator=gen, device="cuda", dtype=torch.uint8), fmt)


def _guarded(m, n, dtype):
    big = torch.full((m * n + 4096,), 7.0, dtype=dtype, device="cuda")
    return big, big[: m * n].view(m, n)


@pytest.mark.parametrize("fmt,path,split,m,n,k", GEMM_PATHS)
def test_every_gemm_kernel_to_the_last_bit(fmt, path, split, m, n, k):
    print("mx gemm", fmt, path, split, m, n, k, flush=True)
    assert nv.mx_gemm_path(m, n, k, fmt) == path and (nv.mx_gemm_workspace_size(m, n, k, fmt) > 0) == split
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    a, w = _exact_mx(m, k, fmt, gen), _exact_mx(n, k, nv.MXFP4, gen)
    a.scales[m - 1, -1] = 255  # the last row and column are NaN, and nothing else
    w.scales[n - 1, 0] = 255
    ref = nv.dequant_mx(a).double() @ nv.dequant_mx(w).double().t()
    for dt in (torch.float32, torch.bfloat16):
        big, out = _guarded(m, n, dt)
        y = nv.mx_gemm(a, w, out_dtype=dt, out=out)
        assert bool((y == ref.float().to(dt))[:-1, :-1].all()), dt
        assert bool(y[-1].isnan().all()) and bool(y[:, -1].isnan().all()) and bool((big[m * n:] == 7.0).all())


@pytest.mark.parametrize("path,split,m,n,k", DX_PATHS)
def test_every_gemm_dx_kernel_to_the_last_bit(path, split, m, n, k):
    # quarters up to 1 times weights as above: every partial sum is exact in fp32
    print("mx gemm_dx", path, split, m, n, k, flush=True)
    assert nv.mx_gemm_dx_path(m, n, k) == path and (nv.mx_gemm_dx_workspace_size(m, n, k) > 0) == split
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    w = _exact_mx(n, k, nv.MXFP4, gen)
    dy = (torch.randint(-4, 5, (m, n), generator=gen, device="cuda") / 4).bfloat16()
    dy[m - 1, n - 1] = float("nan")  # one row of NaN
    w.scales[n - 1, -1] = 255  # and one block of columns
    ref = dy.double() @ nv.dequant_mx(w).double()
    for dt in (torch.float32, torch.bfloat16):
        big, out = _guarded(m, k, dt)
        dx = nv.mx_gemm_dx(dy, w, out_dtype=dt, out=out)
        assert bool((dx == ref.float().to(dt))[:-1, :-32].all()), dt
        assert bool(dx[-1].isnan().all()) and bool(dx[:, -32:].isnan().all()) and bool((big[m * k:] == 7.0).all())


@pytest.mark.parametrize("fmt,path,split,m,n,k", [c for c in GEMM_PATHS if c[0] == nv.MXFP8 and c[1] >= 64])
def test_gemm_fp8_drops_nothing_in_any_tile(fmt, path, split, m, n, k):
    # the codes of test_gemm_fp8_drops_nothing_in_either_output_type, in every tile
    print("mx gemm", fmt, path, split, m, n, k, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    bits = lambda lo, hi, r: torch.randint(lo, hi, (r, k), generator=gen, device="cuda", dtype=torch.uint8)  # noqa: E731
    c, wc = bits(1, 0x51, m) | bits(0, 2, m) << 7, bits(0, 2, n) * 2 + 1 | bits(0, 2, n) << 3
    c[:, 0::16], c[:, 8::16], wc[:, 0::8] = 0x7E, 0xFE, 0x7
    ones = lambda r: torch.full((r, k // 32), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    a, w = nv.MXTensor(c, ones(m), nv.MXFP8), nv.MXTensor(wc[:, 0::2] | wc[:, 1::2] << 4, ones(n), nv.MXFP4)
    ref = (nv.dequant_mx(a).double() @ nv.dequant_mx(w).double().t()).float()
    assert torch.equal(nv.mx_gemm(a, w, out_dtype=torch.float32), ref)
    assert torch.equal(nv.mx_gemm(a, w), ref.bfloat16())


# more than 512 rows: rows that divide neither a workgroup's group nor 256 workgroups, up to five turns per
# workgroup, at widths of every number of threads and pieces per row
@pytest.mark.parametrize("m,k", [(9001, 64), (4099, 512), (2501, 544), (1030, 2048), (1029, 2080), (4099, 4096), (1027, 4128),
                                 (2051, 8192), (700, 11008), (1283, 16384), (515, 16416), (769, 32768), (515, 32800),
                                 (513, 65536)])
def test_norm_backward_many_rows(m, k):
    print("norm backward", m, k, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(m + k)
    R = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    for with_ds, wdtype in ((True, torch.bfloat16), (False, torch.float32)):
        dh, s, ds = (R(m, k).bfloat16() for _ in range(3))
        w, rstd = (1 + 0.2 * R(k)).to(wdtype), 0.5 + torch.rand(m, generator=gen, device="cuda")
        big = torch.full(((m + 2) * k,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = big[: m * k].view(m, k)
        if with_ds:
            out.copy_(ds)  # in place
        dx, dw = nv.add_rmsnorm_backward(dh, s, w, rstd, ds=out if with_ds else None, dx=out)
        assert bool((big[m * k:] == 7.0).all())
        r, g = rstd.double()[:, None], dh.double() * w.double()
        xh = s.double() * r
        ref = r * (g - xh * (g * xh).mean(-1, keepdim=True)) + (ds.double() if with_ds else 0)
        # dx: as in test_norm_backward
        size = r * (g.abs() + xh.abs() * (g * xh).abs().mean(-1, keepdim=True))
        bound = (64 + 6 + 16 + 8) * U32 * size + 2 * U32 * ref.abs() + (U32 * ds.double().abs() if with_ds else 0)
        assert bool(((dx.double() - ref).abs() <= bound * (1 + UBF16) + UBF16 * ref.abs()).all())
        # dweight: a workgroup adds m / (256 groups) rows, at most 16 groups and 256 planes (8 + 6 steps deep);
        # 2 roundings in a term
        terms = dh.double() * xh
        bound = (-(-m // 256) + 16 + 14 + 2) * U32 * terms.abs().sum(0)
        assert bool(((dw.double() - terms.sum(0)).abs() <= bound).all())


@pytest.mark.parametrize("scale", [0, 1, 126, 252, 253, 254])
def test_gemm_dx_of_one_weight_row(scale):
    # dy = 1 and n = 1: the weights as bf16, infinite where they pass its range
    w = nv.MXTensor(torch.arange(256, device="cuda").to(torch.uint8).view(1, 256),
                    torch.full((1, 16), scale, dtype=torch.uint8, device="cuda"), nv.MXFP4)
    want = nv.dequant_mx(w, torch.bfloat16)
    assert bool(want.isinf().any()) == (scale >= 253)
    for dt in (torch.bfloat16, torch.float32):
        assert torch.equal(nv.mx_gemm_dx(torch.ones((1, 1), device="cuda").bfloat16(), w, out_dtype=dt), want.to(dt))


@FMTS
@DTYPES
def test_quantize_special_rows_among_others(fmt, dtype):
    # in the middle of a wave's run, so that neighbouring blocks' lanes hold ordinary values
    x = torch.cat([rows(21, 64, 170, dtype), special_rows(dtype), rows(30, 64, 171, dtype)])
    q = nv.quantize_mx(x.cuda(), fmt)
    c, s = mx.quantize_mx(x.double().numpy(), fmt)
    assert np.array_equal(q.scales.cpu().numpy(), s) and np.array_equal(q.codes.cpu().numpy(), mx.pack(c, fmt))


@pytest.mark.parametrize("m,n,k", [(5, 83, 992), (13, 131, 4640), (15, 4200, 4096), (16, 97, 14336), (67, 131, 1056),
                                   (1573, 1923, 1568), (1860, 4474, 1056), (2615, 5320, 1056)])
def test_gemm_fp8_nan_codes_reach_their_row_only(m, n, k):
    # both NaN codes, at the first and the last place of a row, in every kernel (each lies whole in one of the two
    # parts that are multiplied)
    gen = torch.Generator(device="cuda").manual_seed(m)
    a, w = _exact_mx(m, k, nv.MXFP8, gen), _exact_mx(n, k, nv.MXFP4, gen)
    a.codes[0, k - 1], a.codes[m - 2, 0] = 0x7F, 0xFF
    bad = torch.zeros(m, dtype=torch.bool, device="cuda")
    bad[0] = bad[m - 2] = True
    for dt in (torch.bfloat16, torch.float32):
        y = nv.mx_gemm(a, w, out_dtype=dt).isnan()
        assert bool(y[bad].all()) and not bool(y[~bad].any())
