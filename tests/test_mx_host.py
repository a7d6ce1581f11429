"""Refusals of the microscaled operators: by the library on the host, before
any HIP call, and by the Python binding before the library is reached."""

import os

import pytest
import torch

import bit_gemm_amd as nv
from mx_cases import DX_PATHS, GEMM_PATHS

FAKE, ODD = 0x10000, 0x10008  # never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nv.LIB_PATH):
        from bit_gemm_amd import build
        build.build()
    return nv.lib()


def test_quantize_and_dequant(L):
    q = L.nvfp4_mx_quantize
    assert q(FAKE, 0, 4, 48, 0, FAKE, FAKE, None) == 2  # k % 32
    assert "multiple of 32" in L.nvfp4_last_error().decode()
    assert q(FAKE, 0, -1, 64, 0, FAKE, FAKE, None) == 1
    assert q(FAKE, 2, 4, 64, 0, FAKE, FAKE, None) == 1  # x type
    assert q(FAKE, 0, 4, 64, 2, FAKE, FAKE, None) == 1  # format
    assert q(None, 0, 4, 64, 0, FAKE, FAKE, None) == 1
    assert q(FAKE, 0, 4, 64, 0, ODD, FAKE, None) == 3
    assert q(FAKE, 0, 1 << 32, 64, 0, FAKE, FAKE, None) == 2  # more than one launch's work-items
    assert q(None, 0, 0, 64, 0, None, None, None) == 0 and q(None, 1, 5, 0, 1, None, None, None) == 0
    d = L.nvfp4_mx_dequant
    assert d(FAKE, FAKE, FAKE, 4, 40, 0, 0, None) == 2
    assert d(FAKE, FAKE, FAKE, 4, 64, -1, 0, None) == 1
    assert d(FAKE, FAKE, FAKE, 4, 64, 0, 5, None) == 1
    assert d(FAKE, None, FAKE, 4, 64, 0, 0, None) == 1
    assert d(FAKE, ODD, FAKE, 4, 64, 0, 0, None) == 3
    assert d(None, None, None, 0, 64, 0, 0, None) == 0


def test_gemm(L):
    def g(a=FAKE, s=FAKE, f=0, w=FAKE, ws=FAKE, y=FAKE, m=4, n=8, k=64, o=0, wsp=None, wsb=0):
        return L.nvfp4_mx_gemm(a, s, f, w, ws, y, m, n, k, o, wsp, wsb, None)

    assert g(k=48) == 2 and g(m=-1) == 1 and g(n=-2) == 1 and g(f=3) == 1 and g(o=2) == 1
    assert g(y=None) == 1 and g(a=None) == 1 and g(ws=None) == 1
    assert g(y=ODD) == 3 and g(w=ODD) == 3 and g(s=ODD) == 3
    assert g(m=(1 << 22) + 1) == 2 and g(n=1 << 27) == 2 and g(k=1 << 31) == 2
    assert g(m=0, a=None, y=None) == 0 and g(n=0, w=None, y=None) == 0
    # k = 0: planned like any other size (it needs no operands and no workspace), not divided by
    for m in (3, 100, 1 << 22):
        assert g(m=m, k=0, a=None, s=None, w=None, ws=None, y=ODD) == 3
        if not torch.cuda.is_available():  # past every check, no device here
            assert g(m=m, k=0, a=None, s=None, w=None, ws=None) > 4
    size = L.nvfp4_mx_gemm_workspace_size
    assert size(0, 8, 64, 0) == 0 and size(4, 8, 48, 0) == 0 and size(4, 8, 64, 7) == 0 and size(4, -8, 64, 0) == 0


def test_gemm_dx(L):
    def g(dy=FAKE, w=FAKE, s=FAKE, dx=FAKE, m=4, n=8, k=64, o=0, wsp=None, wsb=0):
        return L.nvfp4_mx_gemm_dx(dy, w, s, dx, m, n, k, o, wsp, wsb, None)

    assert g(k=48) == 2 and g(m=-1) == 1 and g(o=2) == 1 and g(dx=None) == 1 and g(dy=None) == 1
    assert g(dy=ODD) == 3 and g(dx=ODD) == 3 and g(m=0, dy=None, dx=None) == 0
    need = L.nvfp4_mx_gemm_dx_workspace_size(64, 4096, 4096)
    assert need > 0 and need % (64 * 4096 * 4) == 0
    big = dict(m=64, n=4096, k=4096)
    assert g(**big, wsp=FAKE, wsb=need - 1) == 4 and g(**big, wsp=None, wsb=need) == 1 and g(**big, wsp=ODD, wsb=need) == 3
    assert L.nvfp4_mx_gemm_dx_workspace_size(64, 4096, 4080) == 0


def test_norm(L):
    def f(x=FAKE, r=None, w=FAKE, wt=0, eps=1e-6, m=4, k=64, fmt=1, ro=None, rs=FAKE, c=FAKE, s=FAKE):
        return L.nvfp4_add_rmsnorm_mx(x, r, w, wt, eps, m, k, fmt, ro, rs, c, s, None)

    assert f(k=48) == 2 and f(k=0) == 2 and f(k=65568) == 2 and f(m=-1) == 1 and f(m=(1 << 22) + 1) == 2
    assert f(m=1 << 22, k=16416) == 2  # 2^32 work-items
    assert f(wt=4) == 1 and f(fmt=9) == 1 and f(eps=-1.0) == 1 and f(eps=float("nan")) == 1 and f(eps=float("inf")) == 1
    assert f(r=FAKE) == 1 and f(ro=FAKE) == 1 and f(x=None) == 1 and f(c=None) == 1 and f(w=None) == 1
    assert f(x=ODD) == 3 and f(w=ODD) == 3 and f(rs=FAKE + 2) == 3 and f(r=FAKE, ro=ODD) == 3
    assert f(m=0, x=None, w=None, c=None, s=None, rs=None) == 0

    def b(dh=FAKE, s=FAKE, w=FAKE, wt=0, rs=FAKE, ds=None, dx=FAKE + 16, dw=FAKE, m=4, k=64, wsp=FAKE, wsb=1 << 30):
        return L.nvfp4_add_rmsnorm_backward(dh, s, w, wt, rs, ds, dx, dw, m, k, wsp, wsb, None)

    assert b(k=48) == 2 and b(k=0) == 2 and b(m=-1) == 1 and b(wt=2) == 1 and b(dw=None) == 1 and b(dx=None) == 1
    assert b(rs=None) == 1 and b(dh=ODD) == 3 and b(ds=ODD) == 3 and b(dw=ODD) == 3
    assert b(dx=FAKE + 64, dh=FAKE + 64) == 1 and b(dx=FAKE + 64, s=FAKE + 64) == 1  # only ds may be dx
    assert L.nvfp4_add_rmsnorm_backward_workspace_size(4, 64) == 0  # few rows: one launch
    need = L.nvfp4_add_rmsnorm_backward_workspace_size(9000, 64)
    big = dict(m=9000, dx=FAKE + 64)
    assert need >= 64 * 4 and b(**big, wsb=need - 1) == 4
    assert b(**big, wsp=None, wsb=need) == 1 and b(**big, wsp=ODD, wsb=need) == 3
    assert L.nvfp4_add_rmsnorm_backward_workspace_size(0, 64) == 0


def test_norm_refuses_overlaps(L):
    """Outputs that share memory with what other workgroups read: at any offset, the largest included."""
    m, k = 6, 96
    row = 2 * m * k
    at = {n: (1 << 24) + (1 << 16) * i for i, n in enumerate(["x", "r", "w", "ro", "rs", "c", "s", "dh", "ds", "dx", "dw"])}

    def f(**o):
        p = {**at, **o}
        return L.nvfp4_add_rmsnorm_mx(p["x"], p["r"], p["w"], 1, 1e-6, m, k, 1, p["ro"], p["rs"], p["c"], p["s"], None)

    def b(**o):
        p = {**at, **o}
        return L.nvfp4_add_rmsnorm_backward(p["dh"], p["s"], p["w"], 1, p["rs"], p["ds"], p["dx"], p["dw"], m, k, None,
                                            0, None)

    for call, out, inputs in ((f, "ro", ("x", "r")), (b, "dx", ("dh", "s", "ds"))):
        for name in inputs:
            for off in (-row + 16, -16, 16, row - 16):
                assert call(**{out: at[name] + off}) == 1, (out, name, off)
                assert f"{out.replace('ro', 'residual_out')} overlaps" in L.nvfp4_last_error().decode()
    assert b(dx=at["dh"]) == 1 and b(dx=at["s"]) == 1 and b(dx=at["w"]) == 1 and b(dx=at["rs"] - 16) == 1
    assert b(dw=at["w"]) == 1 and b(dw=at["dx"] + 32) == 1 and b(dw=at["dh"] + row - 16) == 1 and b(dw=at["ds"]) == 1
    assert f(c=at["x"]) == 1 and f(c=at["ro"] + 16) == 1 and f(s=at["c"]) == 1 and f(rs=at["r"] + 4) == 1
    assert f(ro=at["w"] + 16) == 1 and f(rs=at["ro"] + row - 4) == 1
    if not torch.cuda.is_available():  # past every check, no device here: whole buffers in place, neighbours
        for ok in (f(), f(ro=at["x"]), f(ro=at["r"]), f(r=at["x"], ro=at["x"]), f(ro=at["x"] + row), f(r=None, ro=None, rs=None),
                   b(), b(dx=at["ds"]), b(ds=None), b(dx=at["dh"] - row), b(dx=at["s"] + row), b(dw=at["w"] + 4 * k)):
            assert ok > 4


def _mx(m, k, fmt):
    return nv.MXTensor.empty(m, k, fmt, "cpu")


def test_binding_refuses():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        nv.quantize_mx(x)
    with pytest.raises(ValueError, match="2-D"):
        nv.quantize_mx(x[0])
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        nv.quantize_mx(x.half())
    with pytest.raises(ValueError, match="contiguous"):
        nv.quantize_mx(x.t())
    with pytest.raises(ValueError, match="format"):
        nv.quantize_mx(x, nv.MXFP8, out=_mx(4, 64, nv.MXFP4))
    with pytest.raises(ValueError, match="multiple of 32"):
        nv.MXTensor.empty(4, 48, nv.MXFP4, "cpu")
    with pytest.raises(ValueError, match="MXFP4 or MXFP8"):
        nv.MXTensor.empty(4, 64, 2, "cpu")
    with pytest.raises(ValueError, match="GPU"):
        nv.dequant_mx(_mx(4, 64, nv.MXFP8))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        nv.dequant_mx(_mx(4, 64, nv.MXFP8), torch.float16)
    bad = _mx(4, 64, nv.MXFP4)
    bad.scales = bad.scales[:3]
    with pytest.raises(ValueError, match="w.scales must have shape"):
        nv.mx_gemm(_mx(2, 64, nv.MXFP8), bad)
    with pytest.raises(ValueError, match="w must be in MXFP4"):
        nv.mx_gemm(_mx(2, 64, nv.MXFP8), _mx(4, 64, nv.MXFP8))
    with pytest.raises(ValueError, match="k=96"):
        nv.mx_gemm(_mx(2, 96, nv.MXFP8), _mx(4, 64, nv.MXFP4))
    with pytest.raises(ValueError, match="out must have shape"):
        nv.mx_gemm(_mx(2, 64, nv.MXFP8), _mx(4, 64, nv.MXFP4), out=torch.zeros(2, 5, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="GPU"):
        nv.mx_gemm(_mx(2, 64, nv.MXFP8), _mx(4, 64, nv.MXFP4))
    with pytest.raises(ValueError, match="dy must be"):
        nv.mx_gemm_dx(x, _mx(5, 64, nv.MXFP4))
    with pytest.raises(ValueError, match="GPU"):
        nv.mx_gemm_dx(x, _mx(64, 64, nv.MXFP4))
    w = torch.ones(64)
    with pytest.raises(ValueError, match="residual_out without"):
        nv.add_rmsnorm_mx(x, w, residual_out=x)
    with pytest.raises(ValueError, match="weight must have shape"):
        nv.add_rmsnorm_mx(x, w[:32])
    with pytest.raises(ValueError, match="residual must be torch.bfloat16"):
        nv.add_rmsnorm_mx(x, w, residual=x.float())
    with pytest.raises(ValueError, match="GPU"):
        nv.add_rmsnorm_mx(x, w, residual=x)
    with pytest.raises(ValueError, match="rstd must have shape"):
        nv.add_rmsnorm_backward(x, x, w, torch.ones(3))
    with pytest.raises(ValueError, match="GPU"):
        nv.add_rmsnorm_backward(x, x, w, torch.ones(4))


def test_paths(L):
    """Every kernel and tile of the products is on the list that the GPU tests run, at a size that the plan gives it."""
    for fmt, path, split, m, n, k in GEMM_PATHS:
        assert nv.mx_gemm_path(m, n, k, fmt) == path, (fmt, m, n, k)
        assert (nv.mx_gemm_workspace_size(m, n, k, fmt) > 0) == split, (fmt, m, n, k)
    for path, split, m, n, k in DX_PATHS:
        assert nv.mx_gemm_dx_path(m, n, k) == path and (nv.mx_gemm_dx_workspace_size(m, n, k) > 0) == split, (m, n, k)
    forms = {(fmt, path, split) for fmt, path, split, *_ in GEMM_PATHS}
    tiles = {(f, t, z) for f in (nv.MXFP4, nv.MXFP8) for t in (64, 128, 224, 256) for z in (False, True)}
    assert forms == {(f, t, False) for f in (nv.MXFP4, nv.MXFP8) for t in (0, 16)} | tiles - {(nv.MXFP4, 256, True)}
    assert {(t, z, n % 8 == 0) for t, z, _, n, _ in DX_PATHS} == \
        {(128, z, w) for z in (False, True) for w in (False, True)} | {(256, False, True), (256, True, True)}
    for bad in ((0, 8, 64), (4, 0, 64), (4, 8, 0), (4, 8, 48), (-1, 8, 64), (4, 1 << 27, 64)):
        assert nv.mx_gemm_path(*bad, nv.MXFP4) == -1 and nv.mx_gemm_dx_path(*bad) == -1
    assert nv.mx_gemm_path(4, 8, 64, 5) == -1


def test_binding_refuses_what_is_no_mx_matrix():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), _mx(4, 64, nv.MXFP4)
    for bad in (x, None, (w.codes, w.scales), 3):
        for call, name in ((lambda: nv.dequant_mx(bad), "q"), (lambda: nv.mx_gemm(bad, w), "a"),
                           (lambda: nv.mx_gemm(w, bad), "w"), (lambda: nv.mx_gemm_dx(x, bad), "w")):
            with pytest.raises(ValueError, match=f"^{name} must be an MXTensor"):
                call()
