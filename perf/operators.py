"""Cases of the microscaled (MX) operators: what is timed and compared.

The operators: quantization to MXFP4 / MXFP8 (an E8M0 power-of-two scale per
32 consecutive elements of a row), the product of an MX activation matrix with
MXFP4 weights, its input gradient, the residual addition with a root mean
square norm whose output is MX, and that norm's gradient.

``run`` computes them with elementary torch operations where ``own`` is false,
and with this package's entry points where it is true.
"""

import math

import torch

own = False

EPS = 1e-6
FP4_MAX, FP8_MAX = 6.0, 448.0
FP4_EMAX, FP8_EMAX = 2, 8  # exponent of the element format's largest binade


def listed():
    return [
        # a stacked down projection's fp32 master weights to MXFP4 and back to
        # bf16 (what a quantized checkpoint costs to write and to check)
        {"name": "quantize_fp4_fp32_4096x14336", "op": "quantize", "fmt": "fp4", "dtype": "fp32", "m": 4096, "k": 14336},
        # activations of a ragged prompt to MXFP8 for the next product
        {"name": "quantize_fp8_bf16_1000x5120", "op": "quantize", "fmt": "fp8", "dtype": "bf16", "m": 1000, "k": 5120},
        # one new token through a square attention projection: latency
        {"name": "gemm_fp8_1x4096x4096", "op": "gemm", "fmt": "fp8", "out": "bf16", "m": 1, "n": 4096, "k": 4096},
        # a batch of new tokens through the down projection: weight streaming
        {"name": "gemm_fp4_16x4096x14336", "op": "gemm", "fmt": "fp4", "out": "bf16", "m": 16, "n": 4096, "k": 14336},
        # a short ragged prompt, sizes that divide nothing, fp32 logits-like output
        {"name": "gemm_fp8_333x4100x1056", "op": "gemm", "fmt": "fp8", "out": "fp32", "m": 333, "n": 4100, "k": 1056},
        # a long prompt through the up projection: matrix rate
        {"name": "gemm_fp4_4096x14336x4096", "op": "gemm", "fmt": "fp4", "out": "bf16", "m": 4096, "n": 14336, "k": 4096},
        # the norm in front of a projection for one new token: latency
        {"name": "norm_1x4096", "op": "norm", "m": 1, "k": 4096, "residual": True, "weight": "bf16"},
        # the same for a long prompt: bandwidth
        {"name": "norm_4096x4096", "op": "norm", "m": 4096, "k": 4096, "residual": True, "weight": "bf16"},
        # a training step's norm gradient at the layer's width, with the
        # residual stream's own gradient
        {"name": "norm_grad_4096x4096", "op": "norm_grad", "m": 4096, "k": 4096, "residual": True, "weight": "fp32"},
        # a small ragged batch of wide rows, no residual branch
        {"name": "norm_grad_333x11008", "op": "norm_grad", "m": 333, "k": 11008, "residual": False, "weight": "bf16"},
        # a training step's input gradient through the down projection
        {"name": "gemm_dx_1024x4096x14336", "op": "gemm_dx", "out": "bf16", "m": 1024, "n": 4096, "k": 14336},
        # a ragged batch through an odd-sized layer, fp32 gradients
        {"name": "gemm_dx_100x1001x1056", "op": "gemm_dx", "out": "fp32", "m": 100, "n": 1001, "k": 1056},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "norm", "norm_grad", "gemm_dx"])
    if op == "quantize":
        return {"op": op, "fmt": rng.choice(["fp4", "fp8"]), "dtype": rng.choice(["fp32", "bf16"]),
                "m": _log_int(rng, 1, 4096), "k": 32 * _log_int(rng, 1, 448)}
    if op == "gemm":
        return {"op": op, "fmt": rng.choice(["fp4", "fp8"]), "out": rng.choice(["bf16", "bf16", "fp32"]),
                "m": _log_int(rng, 1, 2048), "n": _log_int(rng, 48, 14336), "k": 32 * _log_int(rng, 4, 256)}
    if op == "gemm_dx":
        return {"op": op, "out": rng.choice(["bf16", "bf16", "fp32"]), "m": _log_int(rng, 1, 2048),
                "n": _log_int(rng, 48, 8192), "k": 32 * _log_int(rng, 4, 256)}
    return {"op": op, "m": _log_int(rng, 1, 4096), "k": 32 * _log_int(rng, 4, 448),
            "residual": rng.random() < 0.75, "weight": rng.choice(["bf16", "fp32"])}


def _dtype(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _weights(gen, n, k):
    """Layer weights: standard deviation 0.02, one entry in a thousand 20 times as large."""
    w = 0.02 * _randn(gen, n, k)
    return torch.where(torch.rand(n, k, generator=gen, device="cuda") < 0.001, 20.0 * w, w)


def _activations(gen, m, k):
    """Activations with channels of different sizes."""
    return _randn(gen, m, k) * (0.5 + 2.0 * torch.rand(k, generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, m, k = case["op"], case["m"], case["k"]
    s = {"case": case}
    if op == "quantize":
        x = _weights(gen, m, k) if case["dtype"] == "fp32" else _activations(gen, m, k)
        s["x"] = x.to(_dtype(case["dtype"]))
    elif op == "gemm":
        # activations come from a quantizer or a norm, weights were quantized once
        s["a"] = _quantize(_activations(gen, m, k).bfloat16(), case["fmt"])
        s["w"] = _quantize(_weights(gen, case["n"], k), "fp4")
    elif op == "gemm_dx":
        s["dy"] = (0.01 * _randn(gen, m, case["n"])).bfloat16()
        s["w"] = _quantize(_weights(gen, case["n"], k), "fp4")
    else:
        s["x"] = _activations(gen, m, k).bfloat16()
        s["residual"] = (4.0 * _randn(gen, m, k)).bfloat16() if case["residual"] else None
        s["weight"] = (1.0 + 0.1 * _randn(gen, k)).to(_dtype(case["weight"]))
        if op == "norm_grad":  # what the forward pass left, and the gradients that arrive
            s["s"], s["rstd"] = _residual_and_rstd(s.pop("x"), s.pop("residual"))
            s["dh"] = (0.01 * _randn(gen, m, k)).bfloat16()
            s["ds"] = (0.01 * _randn(gen, m, k)).bfloat16() if case["residual"] else None
    return s


# ---------------------------------------------------------------- plain forms


def _quantize(x, fmt):
    """(codes, scales) of the rows of x: scale 2^(floor(log2(amax)) - emax) per 32, codes rounded to nearest even."""
    m, k = x.shape
    b = x.float().reshape(m, k // 32, 32)
    amax = b.abs().amax(-1)
    e = torch.frexp(amax)[1] - 1 - (FP4_EMAX if fmt == "fp4" else FP8_EMAX)
    e = torch.where(amax > 0, e, -127).clamp(min=-127)
    v = torch.ldexp(b, -e[..., None])  # exact: a power of two
    scales = (e + 127).to(torch.uint8)
    if fmt == "fp8":
        return v.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8).reshape(m, k), scales
    a = v.abs()
    mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c = (mag | (torch.signbit(v).to(torch.uint8) << 3)).reshape(m, k // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), scales


def _values(codes, scales, fmt):
    """The fp32 values of packed codes with their scales."""
    m, nb = scales.shape
    if fmt == "fp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                            device=codes.device)
        c = torch.stack((codes & 15, codes >> 4), -1)
        v = grid[c.reshape(m, nb * 32).int()]
    return torch.ldexp(v.reshape(m, nb, 32), scales.int()[..., None] - 127).reshape(m, nb * 32)


def _residual_and_rstd(x, residual):
    s = x if residual is None else (x.float() + residual.float()).bfloat16()
    # long sums of squares, next to rounding borders of the 8-bit output
    return s, (s.double().square().mean(-1) + EPS).rsqrt().float()


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        codes, scales = _quantize(s["x"], c["fmt"])
        if c["fmt"] == "fp4":
            return {"values": _values(codes, scales, "fp4").bfloat16()}
        return {"elements": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}
    if op == "gemm":
        y = _values(*s["a"], c["fmt"]) @ _values(*s["w"], "fp4").t()
        return {"y": y.to(_dtype(c["out"]))}
    if op == "gemm_dx":
        return {"dx": (s["dy"].float() @ _values(*s["w"], "fp4")).to(_dtype(c["out"]))}
    if op == "norm":
        r, rstd = _residual_and_rstd(s["x"], s["residual"])
        h = r.float() * rstd[:, None] * s["weight"].float()
        codes, scales = _quantize(h, "fp8")
        return {"elements": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu),
                "residual": r, "rstd": rstd}
    xhat = s["s"].float() * s["rstd"][:, None]
    dh = s["dh"].float()
    g = dh * s["weight"].float()
    dx = s["rstd"][:, None] * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
    return {"dx": dx.bfloat16(), "dweight": (dh * xhat).sum(0)}


# ------------------------------------------------------------ the entry points


def _own(s):
    import bit_gemm_amd as nv

    c = s["case"]
    op = c["op"]
    if op == "quantize":
        if c["fmt"] == "fp4":
            return {"values": nv.dequant_mx(nv.quantize_mx(s["x"], nv.MXFP4), torch.bfloat16)}
        q = nv.quantize_mx(s["x"], nv.MXFP8)
        return {"elements": q.codes.view(torch.float8_e4m3fn), "scales": q.scales.view(torch.float8_e8m0fnu)}
    if op == "gemm":
        a = nv.MXTensor(*s["a"], nv.MXFP4 if c["fmt"] == "fp4" else nv.MXFP8)
        return {"y": nv.mx_gemm(a, nv.MXTensor(*s["w"], nv.MXFP4), out_dtype=_dtype(c["out"]))}
    if op == "gemm_dx":
        return {"dx": nv.mx_gemm_dx(s["dy"], nv.MXTensor(*s["w"], nv.MXFP4), out_dtype=_dtype(c["out"]))}
    if op == "norm":
        q, r, rstd = nv.add_rmsnorm_mx(s["x"], s["weight"], residual=s["residual"], eps=EPS, fmt=nv.MXFP8)
        return {"elements": q.codes.view(torch.float8_e4m3fn), "scales": q.scales.view(torch.float8_e8m0fnu),
                "residual": r, "rstd": rstd}
    dx, dweight = nv.add_rmsnorm_backward(s["dh"], s["s"], s["weight"], s["rstd"], ds=s["ds"])
    return {"dx": dx, "dweight": dweight}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    if op == "quantize":
        size = 4 if case["dtype"] == "fp32" else 2
        packed = m * k * (0.5 if case["fmt"] == "fp4" else 1.0) + m * k / 32
        # fp4: the packed tensor is written, read again and its bf16 values written
        return {"bytes": m * k * size + (2 * packed + 2 * m * k if case["fmt"] == "fp4" else packed), "flops": 4 * m * k}
    if op == "gemm":
        n = case["n"]
        a = m * k * (0.5 if case["fmt"] == "fp4" else 1.0) + m * k / 32
        return {"bytes": a + n * k * (0.5 + 1 / 32) + m * n * (4 if case["out"] == "fp32" else 2), "flops": 2 * m * n * k}
    if op == "gemm_dx":
        n = case["n"]
        return {"bytes": 2 * m * n + n * k * (0.5 + 1 / 32) + m * k * (4 if case["out"] == "fp32" else 2),
                "flops": 2 * m * n * k}
    w = k * (4 if case["weight"] == "fp32" else 2)
    if op == "norm":  # x, and with a residual it and the new one; 8-bit elements with scales; rstd
        return {"bytes": m * k * (2 + (4 if case["residual"] else 0) + 1 + 1 / 32) + 4 * m + w, "flops": 6 * m * k}
    return {"bytes": m * k * (2 + 2 + 2 + (2 if case["residual"] else 0)) + 4 * m + w + 4 * k, "flops": 10 * m * k}


# ------------------------------------------------- the definitions in 64 bits


def _nearest(v, magnitudes):
    """Index of the entry of the ascending `magnitudes` nearest to each v >= 0; a tie goes to the even index."""
    mid = (magnitudes[1:] + magnitudes[:-1]) / 2
    up, down = torch.searchsorted(mid, v, right=True), torch.searchsorted(mid, v, right=False)
    return torch.where(up == down, up, up - up % 2)


def _exact_blocks(x, fmt):
    """(element values, scale values), float64, of float64 x."""
    m, k = x.shape
    if fmt == "fp4":
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
        top = 4.0
    else:  # 8 subnormal steps of 2^-9, then 8 values in each binade from 2^-6, up to 448
        grid = torch.tensor([i * 2.0 ** -9 for i in range(8)]
                            + [(1 + i / 8) * 2.0 ** e for e in range(-6, 9) for i in range(8)][:-1],
                            dtype=torch.float64, device=x.device)
        top = 256.0
    out, scales = [], []
    for part in x.split(max(1, (1 << 24) // k)):  # rows in pieces: bounded memory
        b = part.reshape(-1, k // 32, 32)
        amax = b.abs().amax(-1, keepdim=True)
        # the power of two that puts amax into the binade that starts at `top`
        p = torch.exp2(torch.floor(torch.log2(amax / top)))
        p = torch.where(amax / p >= 2 * top, 2 * p, torch.where(amax / p < top, p / 2, p))
        p = torch.where(amax > 0, p, torch.zeros_like(p)).clamp(min=2.0 ** -127)
        r = b / p
        v = grid[_nearest(r.abs().contiguous(), grid)]
        out.append(torch.copysign(v, r).reshape(-1, k))
        scales.append(p[..., 0])
    return torch.cat(out), torch.cat(scales)


def _exact_values(codes, scales, fmt):
    if fmt == "fp8":
        c = codes.int()
        e, f = (c >> 3) & 15, (c & 7).double()
        v = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2(e.double() - 10))
        v = torch.where(c >= 128, -v, v)
    else:
        c = torch.stack((codes.int() % 16, codes.int() // 16), -1).reshape(codes.shape[0], -1)
        e, f = (c >> 1) & 3, (c & 1).double()
        v = torch.where(e == 0, f / 2, (2 + f) * torch.exp2(e.double() - 2))
        v = torch.where(c >= 8, -v, v)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        v, p = _exact_blocks(s["x"].double(), case["fmt"])
        if case["fmt"] == "fp4":
            return {"values": v * p.repeat_interleave(32, -1)}
        return {"elements": v, "scales": p}
    if op == "gemm":
        return {"y": _exact_values(*s["a"], case["fmt"]) @ _exact_values(*s["w"], "fp4").t()}
    if op == "gemm_dx":
        return {"dx": s["dy"].double() @ _exact_values(*s["w"], "fp4")}
    w = s["weight"].double()
    if op == "norm":
        r = s["x"].double()
        if s["residual"] is not None:  # the residual stream is kept in bf16
            r = (r + s["residual"].double()).float().bfloat16().double()
        rstd = 1 / torch.sqrt((r * r).sum(-1) / case["k"] + EPS)
        v, p = _exact_blocks(r * rstd[:, None] * w, "fp8")
        return {"elements": v, "scales": p, "residual": r, "rstd": rstd}
    z = s["s"].double()
    rstd = s["rstd"].double()[:, None]
    g = s["dh"].double() * w
    dx = rstd * g - z * rstd ** 3 * (g * z).sum(-1, keepdim=True) / case["k"]
    if s["ds"] is not None:
        dx = dx + s["ds"].double()
    return {"dx": dx, "dweight": (s["dh"].double() * z * rstd).sum(0)}
