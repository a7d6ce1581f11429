"""Cases of the NVFP4 key/value cache: what is timed and compared.

The operators: appending keys and values to a paged cache held in NVFP4 (E2M1
codes, one E4M3 scale per 16 elements of a head, one fp32 scale per head), with
the position rotation of queries and keys on the way; reading cached tokens
back; and attention of new tokens, from one per sequence to whole prompts, over
that cache.

``run`` computes them with elementary torch operations where ``own`` is false,
and with this package's entry points where it is true.
"""

import math

import torch

own = False

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _text(numbers):
    return " ".join(str(n) for n in numbers)


def _numbers(text):
    return [int(n) for n in text.split()]


def listed():
    return [
        # one new token of a layer with 32 heads of 128 (4096 wide): latency
        {"name": "append_1_32x128", "op": "append", "tokens": 1, "hq": 32, "hkv": 32, "d": 128, "rot": 128,
         "interleaved": False, "page": 64, "out": "bf16"},
        # a batch of new tokens, four query heads to a key head
        {"name": "append_48_32to8x128", "op": "append", "tokens": 48, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "page": 64, "out": "bf16"},
        # a ragged prompt of a narrow model that rotates half of each head in neighbouring pairs
        {"name": "append_1001_20to5x64", "op": "append", "tokens": 1001, "hq": 20, "hkv": 5, "d": 64, "rot": 32,
         "interleaved": True, "page": 32, "out": "fp32"},
        # a long prompt of the 4096 wide layer: bandwidth
        {"name": "append_4096_32x128", "op": "append", "tokens": 4096, "hq": 32, "hkv": 32, "d": 128, "rot": 128,
         "interleaved": False, "page": 256, "out": "bf16"},
        # a few tokens of wide heads out of scattered pages
        {"name": "read_777_2x256", "op": "read", "tokens": 777, "hkv": 2, "d": 256, "page": 32, "out": "fp32"},
        # a long shared prefix, to be moved to a cache of another type
        {"name": "read_32768_8x128", "op": "read", "tokens": 32768, "hkv": 8, "d": 128, "page": 64, "out": "bf16"},
        # one new token of the 4096 wide layer over a short context: latency
        {"name": "decode_1x4096_32x128", "op": "attend", "lens": "4096", "new": "1", "hq": 32, "hkv": 32, "d": 128,
         "page": 64, "window": 0},
        # a batch of sequences of very different lengths, one new token each
        {"name": "decode_16xragged_32to8x128", "op": "attend",
         "lens": "8191 17 4096 777 2500 1 6001 333 8192 1024 3071 5555 64 129 7000 1999", "new": _text([1] * 16),
         "hq": 32, "hkv": 8, "d": 128, "page": 64, "window": 0},
        # one new token over a very long context, eight query heads to a key head: bandwidth
        {"name": "decode_1x131072_64to8x128", "op": "attend", "lens": "131072", "new": "1", "hq": 64, "hkv": 8, "d": 128,
         "page": 256, "window": 0},
        # drafted tokens to be verified, a sliding window, narrow heads, small pages
        {"name": "verify_24x5_20to5x64", "op": "attend", "lens": _text(299 + 163 * i for i in range(24)),
         "new": _text(1 + (5 * i) % 8 for i in range(24)), "hq": 20, "hkv": 5, "d": 64, "page": 32, "window": 1024},
        # a step that mixes pieces of prompts with new tokens, wide heads
        {"name": "mixed_8_8to2x256", "op": "attend", "lens": "10001 700 4097 513 9000 33 2048 7777",
         "new": "700 700 1 33 250 33 1 5", "hq": 8, "hkv": 2, "d": 256, "page": 64, "window": 0},
        # a whole long prompt: matrix rate
        {"name": "prompt_4096_32to8x128", "op": "attend", "lens": "4096", "new": "4096", "hq": 32, "hkv": 8, "d": 128,
         "page": 64, "window": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "attend", "attend", "attend", "attend"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 5, 8]) if d > 64 else rng.choice([2, 5, 8, 16])
    hq = hkv * rng.choice([1, 2, 3, 4, 7, 8] if hkv < 8 else [1, 2, 4, 8])
    page = rng.choice([32, 64, 128, 256])
    if op == "append":
        return {"op": op, "tokens": _log_int(rng, 1, 4096), "hq": hq, "hkv": hkv, "d": d,
                "rot": rng.choice([32, d // 2, d, d]), "interleaved": rng.random() < 0.3, "page": page,
                "out": rng.choice(["bf16", "fp32"])}
    if op == "read":
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "hkv": hkv, "d": d, "page": page,
                "out": rng.choice(["bf16", "fp32"])}
    kind = rng.choice(["decode", "decode", "verify", "prompt"])
    if kind == "prompt":  # one to three prompts, each with or without tokens cached before it
        new = [_log_int(rng, 16, 1500) for _ in range(rng.randint(1, 3))]
        lens = [n + rng.choice([0, _log_int(rng, 1, 8000)]) for n in new]
    else:
        b = _log_int(rng, 1, 48)
        new = [1 if kind == "decode" else rng.randint(1, 8) for _ in range(b)]
        top = rng.choice([512, 4096, 16384 if b > 4 else 100000])
        lens = [n + _log_int(rng, 1, top) for n in new]
    return {"op": op, "lens": _text(lens), "new": _text(new), "hq": hq, "hkv": hkv, "d": d, "page": page,
            "window": rng.choice([0, 0, 0, _log_int(rng, 1, 4096)])}


# ------------------------------------------------------------------ the cache
#
# A page holds, for each key head, units of 32 tokens; a unit the codes of the
# keys, of the values, the keys' scales and the values' scales, each in the
# order in which the matrix instructions take them.


def _unit_bytes(d):
    return 32 * (d + d // 8)


def _offsets(d, device):
    """Byte offsets within a unit of the 32 tokens' key codes [32, d/2], value codes [32, d/2], key scales and
    value scales [32, d/16], where byte j of a token's codes holds elements 2j and 2j + 1."""
    i = torch.arange(_unit_bytes(d), device=device)
    n = 16 * d
    kc, vc, ks, vs = i[:n], i[n:2 * n], i[2 * n:2 * n + 2 * d], i[2 * n + 2 * d:]
    order = torch.tensor([0, 2, 1, 3], device=device)  # where the four tokens of a quad lie
    if d == 64:
        kc = kc.view(4, 16, 2, 8).permute(2, 1, 0, 3)  # [half, token, piece of 16, byte]
        vc = vc.view(4, 16, 2, 4, 2)[:, :, :, order].permute(2, 0, 3, 1, 4)  # [half, quad, token, piece of 4, byte]
        ks = ks.view(4, 16, 2).permute(2, 1, 0)
        vs = vs.view(4, 4, 2, 4)[..., order].permute(2, 0, 3, 1)
    else:
        p = d // 128
        kc = kc.view(p, 2, 4, 16, 16).permute(1, 3, 0, 2, 4)  # [half, token, panel, piece of 32, byte]
        vc = vc.view(p, 2, 4, 16, 4, 4).permute(1, 2, 4, 0, 3, 5)  # [half, quad, token, panel, piece of 8, byte]
        ks = ks.view(p, 4, 16, 2, 2).permute(3, 2, 0, 1, 4)
        vs = vs.view(p, 4, 8, 2, 4)[..., order].permute(3, 1, 4, 0, 2)
    return kc.reshape(32, d // 2), vc.reshape(32, d // 2), ks.reshape(32, d // 16), vs.reshape(32, d // 16)


def _units(slots, heads, page):
    """[tokens, heads] index of the unit that holds each slot's token."""
    unit = (slots // page)[:, None] * heads + torch.arange(heads, device=slots.device)
    return unit * (page // 32) + (slots % page // 32)[:, None]


def _write(data, d, page, slots, k, v):
    """k, v: (codes uint8 [tokens, heads, d/2], scales uint8 [tokens, heads, d/16])."""
    flat = data.view(-1, _unit_bytes(d))
    unit = _units(slots, k[0].shape[1], page)[..., None]
    for off, part in zip(_offsets(d, data.device), (k[0], v[0], k[1], v[1])):
        flat[unit, off[slots % 32][:, None]] = part


def _gather(data, d, page, heads, slots):
    flat = data.view(-1, _unit_bytes(d))
    unit = _units(slots, heads, page)[..., None]
    kc, vc, ks, vs = (flat[unit, off[slots % 32][:, None]] for off in _offsets(d, data.device))
    return (kc, ks), (vc, vs)


def _sequence(data, d, page, heads, pages, n):
    """The codes and scales of the first n tokens on these pages, [tokens, heads, ...]."""
    x = data[pages].view(len(pages), heads, page // 32, _unit_bytes(d)).transpose(1, 2)
    x = x.reshape(-1, heads, _unit_bytes(d))[: (n + 31) // 32]
    kc, vc, ks, vs = (x[:, :, off.reshape(-1)].view(x.shape[0], heads, 32, -1).transpose(1, 2).reshape(
        -1, heads, off.shape[1])[:n] for off in _offsets(d, data.device))
    return (kc, ks), (vc, vs)


# ------------------------------------------------------------------ the inputs


def _dtype(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _heads(gen, tokens, heads, d):
    """Keys or values: channels of different sizes, a few far larger."""
    size = 0.5 + torch.rand(heads, d, generator=gen, device="cuda")
    size = torch.where(torch.rand(heads, d, generator=gen, device="cuda") < 0.03, 4.0 * size, size)
    return _randn(gen, tokens, heads, d) * size


def _rope(positions, rot, base=10000.0):
    """cos and sin of every position, side by side."""
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), -1).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, heads, d, page = case["op"], case["hkv"], case["d"], case["page"]
    # calibrated scales: the largest magnitude of a head over 2688 = 6 * 448
    s = {"case": case, "k_scale": (16.0 + 16.0 * torch.rand(heads, generator=gen, device="cuda")) / 2688.0,
         "v_scale": (16.0 + 16.0 * torch.rand(heads, generator=gen, device="cuda")) / 2688.0}
    lens = _numbers(case["lens"]) if op == "attend" else [case["tokens"]]
    per = [-(-n // page) for n in lens]
    total = sum(per) + 3
    pages = torch.randperm(total, generator=gen, device="cuda")[: sum(per)]  # scattered over the cache
    s["data"] = torch.zeros(total, heads * (page // 32) * _unit_bytes(d), dtype=torch.uint8, device="cuda")
    if op != "attend":
        n = case["tokens"]
        i = torch.arange(n, device="cuda")
        s["slots"] = (pages[i // page] * page + i % page).int()
    if op == "append":
        # one projection's output holds q, k and v side by side
        qkv = torch.cat((_randn(gen, n, case["hq"], d), _heads(gen, n, heads, d), _heads(gen, n, heads, d)), 1)
        qkv = qkv.bfloat16()
        s["q"], s["k"], s["v"] = qkv.split((case["hq"], heads, heads), 1)
        s["rope"] = _rope(8192, case["rot"])
        first = int(torch.randint(0, 8192 - n, (1,), generator=gen, device="cuda"))
        s["positions"] = (first + i).int()
        return s
    for b, n in enumerate(lens):  # the context: appended before
        p = pages[sum(per[:b]):sum(per[: b + 1])]
        i = torch.arange(n, device="cuda")
        k = _quantize(_heads(gen, n, heads, d).bfloat16().float(), s["k_scale"])
        v = _quantize(_heads(gen, n, heads, d).bfloat16().float(), s["v_scale"])
        _write(s["data"], d, page, p[i // page] * page + i % page, k, v)
    if op == "read":
        return s
    s["table"] = torch.full((len(lens), max(per)), -1, dtype=torch.int32, device="cuda")
    for b in range(len(lens)):
        s["table"][b, : per[b]] = pages[sum(per[:b]):sum(per[: b + 1])].int()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    new = _numbers(case["new"])
    if max(new) > 1:
        s["starts"] = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    else:
        s["starts"] = None
    s["q"] = (1.5 * _randn(gen, sum(new), case["hq"], d)).bfloat16()
    return s


# ---------------------------------------------------------------- plain forms


def _e4m3(c):
    return c.view(torch.float8_e4m3fn).float()


def _quantize(x, scale):
    """NVFP4 (codes, scales) of fp32 x [tokens, heads, d], blocks of 16 along d; scale fp32 [heads]."""
    t, h, d = x.shape
    st = scale[None, :, None]
    b = x.reshape(t, h, d // 16, 16)
    sigma = (b.abs().amax(-1) / (6.0 * st)).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = sigma.float()
    r = torch.where(f == 0, torch.zeros_like(f), (1.0 / (f * st)).clamp(max=torch.finfo(torch.float32).max))
    v = b * r[..., None]
    a = v.abs()
    mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c = (mag | (torch.signbit(v).to(torch.uint8) << 3)).reshape(t, h, d // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), sigma.view(torch.uint8)


def _values(codes, scales, scale):
    """fp32 [tokens, heads, d]: E2M1 value times E4M3 block scale (exact) times the head's scale."""
    t, h, nb = scales.shape
    grid = torch.tensor(E2M1 + [-x for x in E2M1], device=codes.device)
    v = grid[torch.stack((codes & 15, codes >> 4), -1).reshape(t, h, nb, 16).int()]
    return ((v * _e4m3(scales.contiguous())[..., None]) * scale[None, :, None, None]).reshape(t, h, nb * 16)


def _rotate(x, cos, sin, interleaved):
    """fp32 x [tokens, heads, d]; cos, sin [tokens, rot/2]: its first rot elements rotated in pairs."""
    half = cos.shape[-1]
    r, rest = x[..., : 2 * half], x[..., 2 * half:]
    c, s = cos[:, None], sin[:, None]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    a, b = a * c - b * s, b * c + a * s
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _visible(n, new, window, device):
    """[new, n]: whether the i-th of the last `new` tokens of n sees token j."""
    i = torch.arange(n - new, n, device=device)[:, None]
    j = torch.arange(n, device=device)
    return (j <= i) & (j > i - window) if window else j <= i


def _plain(s):
    c = s["case"]
    heads, d, page = c["hkv"], c["d"], c["page"]
    if c["op"] == "append":
        cos, sin = s["rope"][s["positions"].long()].split(c["rot"] // 2, -1)
        slots = s["slots"].long()
        k = _quantize(_rotate(s["k"].float(), cos, sin, c["interleaved"]), s["k_scale"])
        _write(s["data"], d, page, slots, k, _quantize(s["v"].float(), s["v_scale"]))
        k, v = _gather(s["data"], d, page, heads, slots)
        return {"q": _rotate(s["q"].float(), cos, sin, c["interleaved"]).bfloat16(),
                "k": _values(*k, s["k_scale"]).to(_dtype(c["out"])), "v": _values(*v, s["v_scale"]).to(_dtype(c["out"]))}
    if c["op"] == "read":
        k, v = _gather(s["data"], d, page, heads, s["slots"].long())
        return {"k": _values(*k, s["k_scale"]).to(_dtype(c["out"])), "v": _values(*v, s["v_scale"]).to(_dtype(c["out"]))}
    out, lse, at, group = [], [], 0, c["hq"] // heads
    for b, (n, new) in enumerate(zip(_numbers(c["lens"]), _numbers(c["new"]))):
        k, v = _sequence(s["data"], d, page, heads, s["table"][b, : -(-n // page)].long(), n)
        k = _values(*k, s["k_scale"]).permute(1, 2, 0).contiguous()  # [heads, d, n]
        v = _values(*v, s["v_scale"]).transpose(0, 1).contiguous()
        q = s["q"][at:at + new].float().view(new, heads, group, d).permute(1, 0, 2, 3).reshape(heads, new * group, d)
        w = (q @ k).view(heads, new, group, n) / math.sqrt(d)
        w.masked_fill_(~_visible(n, new, c["window"], w.device)[:, None], -math.inf)
        top = w.amax(-1, keepdim=True)
        w = w.sub_(top).exp_()
        total = w.sum(-1, keepdim=True)
        o = (w.view(heads, new * group, n) @ v).view(heads, new, group, d) / total
        out.append(o.permute(1, 0, 2, 3).reshape(new, heads * group, d))
        lse.append((total.log() + top).permute(1, 0, 2, 3).reshape(new, heads * group))
        at += new
    return {"out": torch.cat(out).bfloat16(), "lse": torch.cat(lse)}


# ------------------------------------------------------------ the entry points


def _own(s):
    import bit_gemm_amd as nv

    c = s["case"]
    cache = nv.KVCache(s["data"], s["k_scale"], s["v_scale"], c["d"], c["page"])
    if c["op"] == "append":
        q = nv.kv_append(cache, s["k"], s["v"], s["slots"], q=s["q"], positions=s["positions"], rope=s["rope"],
                         interleaved=c["interleaved"])
        k, v = nv.kv_read(cache, s["slots"], _dtype(c["out"]))
        return {"q": q, "k": k, "v": v}
    if c["op"] == "read":
        k, v = nv.kv_read(cache, s["slots"], _dtype(c["out"]))
        return {"k": k, "v": v}
    out, lse = nv.kv_attention(s["q"], cache, s["table"], s["lens"], q_starts=s["starts"], window=c["window"],
                               return_lse=True)
    return {"out": out, "lse": lse}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    heads, d = case["hkv"], case["d"]
    packed = heads * d * 2 * (0.5 + 1 / 16)  # a token's key and value in the cache
    if case["op"] != "attend":
        n, size = case["tokens"], 4 if case["out"] == "fp32" else 2
        read = n * (packed + 2 * heads * d * size)
        if case["op"] == "read":
            return {"bytes": read, "flops": 2 * n * heads * 2 * d}
        rope = n * case["rot"] * 4
        return {"bytes": n * (2 * (case["hq"] + 2 * heads) * d + 2 * case["hq"] * d + packed) + rope + read,
                "flops": n * d * (3 * case["hq"] + 12 * heads)}
    seen = pairs = 0
    for n, new in zip(_numbers(case["lens"]), _numbers(case["new"])):
        w = case["window"] or n
        seen += min(n, w + new - 1)
        pairs += sum(min(n - new + 1 + i, w) for i in range(new))
    rows = sum(_numbers(case["new"])) * case["hq"]
    return {"bytes": seen * packed + rows * (4 * d + 4), "flops": 4 * d * pairs * case["hq"]}


# ------------------------------------------------- the definitions in 64 bits


def _nearest(v, magnitudes):
    """Index of the entry of the ascending `magnitudes` nearest to each v >= 0; a tie goes to the even index."""
    mid = (magnitudes[1:] + magnitudes[:-1]) / 2
    up, down = torch.searchsorted(mid, v, right=True), torch.searchsorted(mid, v, right=False)
    return torch.where(up == down, up, up - up % 2)


def _exact_quantized(x, scale):
    t, h, d = x.shape
    e4m3 = torch.tensor([i * 2.0 ** -9 for i in range(8)]
                        + [(1 + i / 8) * 2.0 ** e for e in range(-6, 9) for i in range(8)][:-1],
                        dtype=torch.float64, device=x.device)
    e2m1 = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    b = x.reshape(t, h, d // 16, 16)
    s = scale.double()[None, :, None]
    sigma = e4m3[_nearest((b.abs().amax(-1) / (6 * s)).contiguous(), e4m3)]
    unit = (sigma * s)[..., None]
    v = e2m1[_nearest(torch.where(unit > 0, b.abs() / unit, torch.zeros_like(b)).contiguous(), e2m1)]
    return (torch.copysign(v, b) * unit).reshape(t, h, d)


def _exact_values(codes, scales, scale):
    c = torch.stack((codes.int() % 16, codes.int() // 16), -1).flatten(-2)
    e, f = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, f / 2, (2 + f) * torch.exp2(e.double() - 2))
    v = torch.where(c >= 8, -v, v)
    e, f = (scales.int() >> 3) & 15, (scales.int() & 7).double()
    sigma = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2(e.double() - 10))
    return v * sigma.repeat_interleave(16, -1) * scale.double()[None, :, None]


def _exact_rotated(x, angle_cos, angle_sin, interleaved):
    half = angle_cos.shape[-1]
    i = torch.arange(half, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
    out = x.clone()
    z = torch.complex(x[..., first], x[..., second]) * torch.complex(angle_cos, angle_sin)[:, None]
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    heads, d, page = case["hkv"], case["d"], case["page"]
    if case["op"] == "append":
        cs = s["rope"].double()[s["positions"].long()]
        half = case["rot"] // 2
        q, k = (_exact_rotated(s[n].double(), cs[:, :half], cs[:, half:], case["interleaved"]) for n in "qk")
        return {"q": q, "k": _exact_quantized(k, s["k_scale"]), "v": _exact_quantized(s["v"].double(), s["v_scale"])}
    if case["op"] == "read":
        k, v = _gather(s["data"], d, page, heads, s["slots"].long())
        return {"k": _exact_values(*k, s["k_scale"]), "v": _exact_values(*v, s["v_scale"])}
    group = case["hq"] // heads
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, new) in enumerate(zip(_numbers(case["lens"]), _numbers(case["new"]))):
        i = torch.arange(n, device="cuda")
        slots = s["table"][b].long()[i // page] * page + i % page
        k, v = _gather(s["data"], d, page, heads, slots)
        k, v = _exact_values(*k, s["k_scale"]), _exact_values(*v, s["v_scale"])
        seen = _visible(n, new, case["window"], "cuda")
        for h in range(heads * group):  # a head at a time: bounded memory
            w = s["q"][at:at + new, h].double() @ k[:, h // group].t().contiguous() / math.sqrt(d)
            w = torch.where(seen, w, torch.full_like(w, -math.inf))
            norm = torch.logsumexp(w, -1, keepdim=True)
            out[at:at + new, h] = torch.exp(w - norm) @ v[:, h // group].contiguous()
            lse[at:at + new, h] = norm[:, 0]
        at += new
    return {"out": out, "lse": lse}
