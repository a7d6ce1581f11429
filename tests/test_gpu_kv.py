"""GPU parity of the key/value cache: append and read bit-exact with the
oracle, attention against float64 within bounds on its roundings."""

import numpy as np
import pytest
import torch

import bit_gemm_amd as nv
import oracle.kv as okv
from kv_cases import Sequences, bf16, check_attention, heads, queries, rope_table, starts

pytestmark = pytest.mark.gpu

DIMS = pytest.mark.parametrize("d", [64, 128, 256])


def _same(a, b):
    """Equal values bit for bit, any NaN equal to any other."""
    a, b = a.astype(np.float32), b.astype(np.float32)
    return np.array_equal(np.where(np.isnan(a), 0x7FC00000, a.view(np.uint32)), np.where(np.isnan(b), 0x7FC00000, b.view(np.uint32)))


def _np(t):
    return t.float().cpu().numpy()


# ------------------------------------------------------------- append and read


@DIMS
@pytest.mark.parametrize("tokens,hq,hkv,page,rot,interleaved", [
    (1, 4, 1, 32, "d", False), (3, 3, 3, 64, "d", True), (37, 8, 2, 32, 32, False), (130, 5, 5, 256, 32, True),
    (65, 2, 1, 128, "half", False), (33, 7, 7, 32, 0, False), (300, 1, 1, 32, "d", False)])
def test_append_and_read(d, tokens, hq, hkv, page, rot, interleaved):
    print("kv append", d, tokens, hq, hkv, page, rot, interleaved, flush=True)
    rot = d if rot == "d" else d // 2 if rot == "half" else rot
    rng = np.random.default_rng(tokens + d)
    pages = -(-tokens // page) + 2
    ks, vs = ((rng.uniform(4, 40, hkv) / 2688).astype(np.float32) for _ in "kv")
    cache = nv.KVCache.empty(pages, page, hkv, d, "cuda", torch.from_numpy(ks).cuda(), torch.from_numpy(vs).cuda())
    cache.data.fill_(0xA5)
    # q, k and v as columns of one matrix
    fused = torch.cat((heads(rng, tokens, hq, d), heads(rng, tokens, hkv, d), heads(rng, tokens, hkv, d)), 1)
    q, k, v = fused.cuda().split((hq, hkv, hkv), 1)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int32)
    table = rope_table(500, rot)
    pos = rng.integers(0, 500, tokens).astype(np.int32)
    before = cache.data.clone()
    args = dict(positions=torch.from_numpy(pos).cuda(), rope=torch.from_numpy(table).cuda()) if rot else {}
    got = nv.kv_append(cache, k, v, torch.from_numpy(slots).cuda(), q=q, interleaved=interleaved, **args)
    f = fused.float().numpy()
    kf, qf = f[:, hq:hq + hkv], f[:, :hq]
    if rot:
        kf, qf = okv.rotate(kf, pos, table, interleaved), okv.rotate(qf, pos, table, interleaved)
    assert _same(_np(got), bf16(qf).float().numpy())
    want_k, want_v = okv.cached(kf, f[:, hq + hkv:], ks, vs)
    for dtype in (torch.float32, torch.bfloat16):
        gk, gv = nv.kv_read(cache, torch.from_numpy(slots).cuda(), dtype)
        assert gk.shape == gv.shape == (tokens, hkv, d)
        assert _same(_np(gk), torch.from_numpy(want_k).to(dtype).float().numpy())
        assert _same(_np(gv), torch.from_numpy(want_v).to(dtype).float().numpy())
    # bytes of the tokens alone changed: as many as a token's key and value hold, at most
    rest = np.setdiff1d(np.arange(pages * page), slots).astype(np.int32)
    after = cache.data.clone()
    assert int((after != before).sum()) <= tokens * hkv * (d + d // 8)
    cache.data.copy_(before)
    rk, rv = nv.kv_read(cache, torch.from_numpy(rest).cuda())
    cache.data.copy_(after)
    sk, sv = nv.kv_read(cache, torch.from_numpy(rest).cuda())
    assert _same(_np(rk), _np(sk)) and _same(_np(rv), _np(sv))
    # in q's place
    same = nv.kv_append(cache, k, v, torch.from_numpy(slots).cuda(), q=q, q_out=q, interleaved=interleaved, **args)
    assert same.data_ptr() == q.data_ptr() and _same(_np(q), _np(got))
    assert torch.equal(cache.data, after)


@DIMS
def test_blocks_of_every_kind(d):
    """Zeros of both signs, magnitudes from subnormal to past the scales' range, ties of codes and scales."""
    rng = np.random.default_rng(d)
    rows = [np.zeros(d), -np.zeros(d), np.full(d, 1e-38), rng.standard_normal(d) * 1e-4, rng.standard_normal(d) * 1e5,
            np.full(d, 3e38), np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], d // 8),
            -np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], d // 8) / 64, np.repeat(2.0 ** -np.arange(d // 16), 16),
            np.eye(d)[3] * 1e-3]
    x = bf16(np.stack(rows)[:, None])
    one = np.ones(1, np.float32)
    cache = nv.KVCache.empty(1, 32, 1, d)
    slots = torch.arange(len(rows), dtype=torch.int32, device="cuda")
    nv.kv_append(cache, x.cuda(), x.flip(0).cuda(), slots)
    k, v = nv.kv_read(cache, slots, torch.float32)
    want = okv.cached(x.float().numpy(), x.flip(0).float().numpy(), one, one)
    assert _same(_np(k), want[0]) and _same(_np(v), want[1])


@DIMS
def test_infinities_and_nans_stay_with_their_token_and_head(d):
    rng = np.random.default_rng(1)
    k, v = heads(rng, 40, 3, d), heads(rng, 40, 3, d)
    k[3, 0, 5], k[7, 1, d - 1], v[9, 2, 0], v[33, 1, 17] = float("inf"), float("nan"), float("-inf"), float("nan")
    cache = nv.KVCache.empty(2, 32, 3, d)
    slots = torch.arange(5, 45, dtype=torch.int32, device="cuda")
    nv.kv_append(cache, k.cuda(), v.cuda(), slots)
    gk, gv = nv.kv_read(cache, slots, torch.float32)
    one = np.ones(3, np.float32)
    want = okv.cached(k.float().numpy(), v.float().numpy(), one, one)
    assert np.isnan(want[0]).any((-1,)).sum() == 4
    assert _same(_np(gk), want[0]) and _same(_np(gv), want[1])
    # a position outside the table, a rotation past fp32's range
    big = bf16(np.full((4, 3, d), 3.3e38))
    table = torch.from_numpy(rope_table(4, d)).cuda()
    pos = torch.tensor([0, 4, -1, 1], dtype=torch.int32, device="cuda")
    q = nv.kv_append(cache, big.cuda(), v[:4].cuda(), slots[:4], q=big.cuda(), positions=pos, rope=table)
    gk, gv = nv.kv_read(cache, slots[:4], torch.float32)
    assert torch.isfinite(gk[0]).all() and torch.isnan(gk[1:]).all() and torch.isnan(gv[1:]).all()
    assert torch.isnan(q[1:3]).all() and torch.isfinite(q[0]).all() and torch.isinf(q[3]).any()


def test_slots_outside_the_cache_are_left_out():
    rng = np.random.default_rng(2)
    k, v, q = heads(rng, 8, 2, 64).cuda(), heads(rng, 8, 2, 64).cuda(), heads(rng, 8, 4, 64).cuda()
    cache = nv.KVCache.empty(2, 32, 2, 64)
    cache.data.fill_(0x11)
    slots = torch.tensor([0, -1, 63, 64, 2 ** 31 - 1, -2 ** 31, 7, 9], dtype=torch.int32, device="cuda")
    out = torch.full((8, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    nv.kv_append(cache, k, v, slots, q=q, q_out=out)
    kept = torch.tensor([0, 2, 6, 7], device="cuda")
    gone = torch.tensor([1, 3, 4, 5], device="cuda")
    assert torch.equal(out[kept], q[kept]) and (out[gone] == 9.0).all()
    gk, gv = nv.kv_read(cache, slots, torch.float32)
    assert (gk[gone] == 0).all() and (gv[gone] == 0).all()
    want = okv.cached(_np(k), _np(v), np.ones(2, np.float32), np.ones(2, np.float32))
    assert _same(_np(gk[kept]), want[0][kept.cpu()]) and _same(_np(gv[kept]), want[1][kept.cpu()])
    # nothing at all
    assert nv.kv_append(cache, k[:0], v[:0], slots[:0], q=q[:0]).shape == (0, 4, 64)
    assert nv.kv_read(cache, slots[:0])[0].shape == (0, 2, 64)


# ------------------------------------------------------------------- attention

CASES = [
    # lens, new, q heads, heads, page, causal, window
    ([1], [1], 1, 1, 32, True, 0),
    ([31, 32, 33, 64, 65], [1] * 5, 4, 4, 32, True, 0),
    ([129, 1, 2000, 400], [1] * 4, 8, 2, 64, True, 0),
    ([700, 5, 0, 1300], [1] * 4, 16, 1, 128, True, 0),
    ([257, 90], [1] * 2, 34, 2, 32, True, 0),
    ([600, 1025, 31], [1] * 3, 64, 1, 64, True, 0),
    ([1000, 640], [2, 1], 3, 3, 32, True, 700),
    ([40, 300, 5, 77], [3, 8, 5, 1], 6, 2, 32, True, 0),
    ([40, 300, 5, 77], [3, 0, 5, 0], 6, 2, 32, True, 0),
    ([3, 0, 64], [7, 4, 64], 3, 1, 32, True, 0),
    ([100, 333], [100, 45], 4, 2, 64, True, 0),
    ([257], [257], 2, 1, 32, True, 0),
    ([640, 95], [130, 95], 5, 1, 256, True, 0),
    ([900, 333, 20], [1] * 3, 4, 2, 32, True, 100),
    ([900, 333, 20], [40, 3, 20], 4, 2, 32, True, 1),
    ([900, 333, 20], [200, 3, 20], 4, 2, 32, True, 65),
    ([500, 30], [20, 30], 2, 2, 64, False, 0),
    ([5, 200], [9, 300], 2, 1, 64, False, 0),
    ([700, 0, 33, 500], [300, 0, 1, 77], 4, 1, 64, True, 0),
    ([512, 1000], [256, 513], 2, 1, 32, True, 0),
]
# head_dim, rows of a workgroup
PATHS = [(64, 16), (64, 32), (128, 16), (128, 32), (128, 256), (256, 16), (256, 128)]


def _table_for(rows, lens, new, hq, hkv, d, page, window):
    """Pages of a table with which the call is planned with blocks of that many rows; None where it never is."""
    need = max([-(-n // page) for n in lens] + [1])
    one = min(new) == max(new) == 1
    for pages in sorted({need} | {need * 2 ** i for i in range(1, 22)}):
        if pages * page < 2 ** 31 and len(lens) * pages < 2 ** 22 and nv.kv_attention_path(
                len(lens), sum(new), hq, hkv, d, page, pages, window, one) == rows:
            return pages
    return None


@pytest.mark.parametrize("d,rows", PATHS)
@pytest.mark.parametrize("lens,new,hq,hkv,page,causal,window", CASES)
def test_attention(d, rows, lens, new, hq, hkv, page, causal, window):
    """Every kernel: a wide page table makes the call look like more work than it is."""
    pages = _table_for(rows, lens, new, hq, hkv, d, page, window)
    if pages is None:
        pytest.skip("few rows or a short window: never so many rows in a workgroup")
    print("kv attention", d, rows, lens, new, hq, hkv, page, causal, window, flush=True)
    s = Sequences(len(lens) + d, lens, hkv, d, page, table_pages=pages).append()
    q = queries(7, sum(new), hq, d)
    one = max(new) == 1 == min(new)
    out, lse = nv.kv_attention(q.cuda(), s.cache, s.table, s.kv_lens, None if one else starts(new), causal=causal,
                               window=window, return_lse=True)
    check_attention(s, new, q, out, lse, d ** -0.5, causal, window)
    again = nv.kv_attention(q.cuda(), s.cache, s.table, s.kv_lens, starts(new), causal=causal, window=window)
    if not one:
        assert torch.equal(out, again)  # the order of the sums is fixed, lse or not


@pytest.mark.parametrize("d,rows", PATHS)
@pytest.mark.parametrize("lens,new,hq,hkv", [([5000], [1], 8, 1), ([9000, 100, 3000], [1, 1, 1], 3, 1),
                                             ([2500, 2300], [4, 60], 8, 2), ([20000], [2], 2, 1),
                                             ([6000, 40, 3300], [300, 40, 1], 4, 1)])
def test_attention_split_contexts(d, rows, lens, new, hq, hkv):
    pages = _table_for(rows, lens, new, hq, hkv, d, 32, 0)
    if pages is None:
        pytest.skip("few rows: never so many in a workgroup")
    print("kv attention split", d, rows, lens, new, hq, hkv, flush=True)
    s = Sequences(3, lens, hkv, d, 32, table_pages=pages).append()
    q = queries(8, sum(new), hq, d)
    assert nv.kv_attention_workspace_size(len(lens), sum(new), hq, hkv, d, 32, pages, 0, False) > 0
    out, lse = nv.kv_attention(q.cuda(), s.cache, s.table, s.kv_lens, starts(new), return_lse=True)
    check_attention(s, new, q, out, lse, d ** -0.5)


@pytest.mark.parametrize("d,rows", PATHS)
@pytest.mark.parametrize("fill", [0x00, 0x7F, 0xFF])
def test_attention_does_not_see_what_is_masked(d, rows, fill):
    """Unwritten places of any content, pages past the length, NaN tokens behind a row's own, bad page numbers."""
    new = [40, 150]
    pages = _table_for(rows, [70, 200], new, 4, 2, d, 64, 0)
    s = Sequences(9, [70, 200], 2, d, 64, fill=fill, table_pages=max(pages, 9))
    s.k[1][190, 0, 3] = float("nan")  # seen by the last 10 tokens, through both query heads of its group
    s.v[1][195, 1, 3] = float("inf")
    s.append()
    q = queries(1, sum(new), 4, d)
    table = s.table.clone()
    table[0, 2:] = 2 ** 31 - 1
    table[1, 4:] = -1
    out, lse = nv.kv_attention(q.cuda(), s.cache, table, s.kv_lens, starts(new), return_lse=True)
    bad = torch.zeros(sum(new), 4, dtype=torch.bool)
    bad[-10:, :2] = True
    bad[-5:, 2:] = True
    assert torch.equal(torch.isnan(out).all(-1).cpu(), bad) and torch.equal(torch.isnan(out).any(-1).cpu(), bad)
    assert torch.equal(torch.isnan(lse).cpu(), bad)
    # the rest as with finite stand-ins for these tokens
    s.k[1][190, 0, 3] = 0.0
    s.v[1][195, 1, 3] = 0.0
    at = 0
    for b, m in enumerate(new):
        k, v = s.held(b)
        ref = okv.attention(q[at:at + m].float().numpy(), k, v, d ** -0.5, okv.visible(s.lens[b], m))
        ok = ~bad[at:at + m].numpy()
        assert np.abs(out[at:at + m].double().cpu().numpy() - ref[0])[ok].max() <= 2.0 ** -7 * np.abs(ref[0]).max()
        at += m


@pytest.mark.parametrize("d,rows", PATHS)
def test_attention_leaves_out_pages_that_are_not_in_the_cache(d, rows):
    n, new = 330, 70
    pages = _table_for(rows, [n], [new], 2, 1, d, 32, 0)
    s = Sequences(11, [n], 1, d, 32, table_pages=pages).append()
    table = s.table.clone()
    table[0, 1], table[0, 3] = s.cache.pages, -5  # tokens 32..63 and 96..127
    q = queries(3, new, 2, d)
    out, lse = nv.kv_attention(q.cuda(), s.cache, table, s.kv_lens, starts([new]), return_lse=True)
    k, v = s.held(0)
    seen = okv.visible(n, new).copy()
    seen[:, 32:64] = seen[:, 96:128] = False
    ref = okv.attention(q.float().numpy(), k, v, d ** -0.5, seen)
    assert np.abs(out.double().cpu().numpy() - ref[0]).max() <= 2.0 ** -7 * np.abs(ref[0]).max()
    assert np.abs(lse.double().cpu().numpy() - ref[1]).max() <= 1e-4
    table.fill_(-1)
    out, lse = nv.kv_attention(q.cuda(), s.cache, table, s.kv_lens, starts([new]), return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("b,longest", [(70, 300), (150, 40), (257, 900)])
def test_attention_of_many_sequences(b, longest):
    rng = np.random.default_rng(b)
    lens = [int(x) for x in rng.integers(0, longest, b)]
    new = [int(x) for x in rng.integers(0, 4, b)]
    s = Sequences(b, lens, 1, 64, 32).append()
    q = queries(4, sum(new), 2, 64)
    out, lse = nv.kv_attention(q.cuda(), s.cache, s.table, s.kv_lens, starts(new), return_lse=True)
    check_attention(s, new, q, out, lse, 0.125)


@pytest.mark.parametrize("d,rows", PATHS)
@pytest.mark.parametrize("size,scale", [(0.0, 1.0), (1e-30, 1.0), (30.0, None), (1.0, -0.3), (1.0, 0.0), (2e38, 1e-38), (1.0, 1e-30), (1e-39, 1e37)])
def test_attention_of_small_and_large_logits(d, rows, size, scale):
    lens, new = [150, 700], [40, 33]
    pages = _table_for(rows, lens, new, 3, 1, d, 32, 0)
    s = Sequences(5, lens, 1, d, 32, table_pages=pages).append()
    q = queries(2, sum(new), 3, d, size)
    q.clamp_(-3e38, 3e38)
    scale = d ** -0.5 if scale is None else scale
    out, lse = nv.kv_attention(q.cuda(), s.cache, s.table, s.kv_lens, starts(new), scale=scale, return_lse=True)
    check_attention(s, new, q, out, lse, scale)


@pytest.mark.parametrize("d,rows", PATHS)
@pytest.mark.parametrize("logit", [3e4, 1e6, -1e6, 7e8, -7e8, 3e12, -1e20, 2e37, -2e37, -2e38])
def test_attention_of_logits_past_the_steps_of_fp32(d, rows, logit):
    """Logits whose neighbours in fp32 are further apart than exponentials tell: the largest ones share the row alike,
    in whichever units they lie.  Keys are 4 (held as 6 * 0.6875) or 6 in one element and a logit's rounding is common to equal
    keys; the p of the others are 0.  The larger ones' p are equal but for p's rounding to fp16 (2^-11) and what an
    exponential is off (2^-16, as in `bounds`); the quotient is rounded to bf16 (2^-8)."""
    n, new = 1500, 70
    pages = _table_for(rows, [n], [new], 4, 1, d, 32, 0)
    print("kv attention logits", d, rows, logit, flush=True)
    rng = np.random.default_rng(6)
    k, v = np.zeros((n, 1, d)), rng.choice([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], (n, 1, d)) * rng.choice([-1.0, 1.0], (n, 1, d))
    v[:, 0, ::16] = 6.0  # every block's scale is 1
    large = rng.random(n) < 0.03
    large[:40], large[41] = False, True  # (the first of them behind the first unit)
    best = 6.0 if logit > 0 else 4.0
    k[:, 0, 5] = np.where(large, best, 10.0 - best)
    cache = nv.KVCache.empty(-(-n // 32), 32, 1, d)
    nv.kv_append(cache, bf16(k).cuda(), bf16(v).cuda(), torch.arange(n, dtype=torch.int32, device="cuda"))
    table = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    table[0, : cache.pages] = torch.arange(cache.pages)
    q = torch.zeros(new, 4, d, dtype=torch.bfloat16)
    q[:, :, 5] = torch.tensor([logit / 6.0, logit / 5.0, logit / 4.0, logit / 3.0]).bfloat16()
    scale = 0.75
    out, lse = nv.kv_attention(q.cuda(), cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), starts([new]),
                               scale=scale, return_lse=True)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    held = {6.0: 6.0, 4.0: 4.125}[best]
    for t in range(new):
        at = np.flatnonzero(large[: n - new + t + 1])
        want = v[at, 0].mean(0)
        rounded = (2.0 ** -11 + 2.0 ** -16) * np.abs(v[at, 0]).mean(0)
        assert (np.abs(out[t] - want) <= rounded + 2.0 ** -8 * (np.abs(want) + rounded)).all(), t
        top = q[t, :, 5].double().numpy() * held * scale
        assert (np.abs(lse[t] - top - np.log(len(at))) <= 2.0 ** -21 * np.abs(top) + 2.0 ** -20).all(), t


@DIMS
@pytest.mark.parametrize("b,hq,hkv", [(300, 2, 1), (600, 40, 1)])
def test_attention_of_many_single_tokens(d, b, hq, hkv):
    rng = np.random.default_rng(b + d)
    lens = [int(x) for x in rng.integers(0, 90, b)]
    s = Sequences(b, lens, hkv, d, 32).append()
    q = queries(9, b, hq, d)
    out, lse = nv.kv_attention(q.cuda(), s.cache, s.table, s.kv_lens, return_lse=True)
    check_attention(s, [1] * b, q, out, lse, d ** -0.5)


def test_attention_keeps_many_small_probabilities():
    """One token of probability 1 and 60000 whose own is about 2^-24 each: together 2^-8 of the row's sum, which fp16
    probabilities below 2^-24 would lose."""
    n = 60001
    k = np.zeros((n, 1, 64))
    k[0, 0, 0] = 6.0  # representable as they are: 6 * 1
    v = np.full((n, 1, 64), 6.0)
    v[0] = 0.0
    cache = nv.KVCache.empty(n // 64 + 1, 64, 1, 64)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    nv.kv_append(cache, bf16(k).cuda(), bf16(v).cuda(), slots)
    table = torch.arange(n // 64 + 1, dtype=torch.int32, device="cuda")[None]
    for exponent in (20.0, 24.0, 24.7, 28.0):
        q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
        q[0, 0, 0] = 1.0
        scale = exponent * np.log(2) / 6
        out = nv.kv_attention(q.cuda(), cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), scale=scale)
        p = float(np.exp(-np.float64(np.float32(scale)) * 6))
        want = 6.0 * 60000 * p / (1 + 60000 * p)
        assert abs(float(out[0, 0, 5]) - want) <= want * (2.0 ** -8 + 2.0 ** -10), exponent


def test_attention_cuts_lengths_and_starts_to_their_tables():
    s = Sequences(12, [64, 64], 1, 64, 32).append()
    q = queries(3, 2, 2, 64)
    want = nv.kv_attention(q.cuda(), s.cache, s.table, s.kv_lens)
    long = torch.tensor([64 + 1000, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    assert torch.equal(nv.kv_attention(q.cuda(), s.cache, s.table, long), want)
    none = nv.kv_attention(q.cuda(), s.cache, s.table, torch.tensor([-3, -2 ** 31], dtype=torch.int32, device="cuda"))
    assert (none == 0).all()
    st = torch.tensor([-4, 1, 900], dtype=torch.int32, device="cuda")
    assert torch.equal(nv.kv_attention(q.cuda(), s.cache, s.table, s.kv_lens, st), want)
    # a table without pages
    out, lse = nv.kv_attention(q.cuda(), s.cache, s.table[:, :0].contiguous(), s.kv_lens, return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_attention_of_starts_in_disorder_stays_in_bounds():
    """Row numbers that decrease or leave the call's tokens: unspecified rows, but none outside its own buffers."""
    s = Sequences(22, [4000, 3000, 2000], 1, 64, 32).append()
    q = queries(5, 50, 20, 64).cuda()
    need = nv.kv_attention_workspace_size(3, 50, 20, 1, 64, 32, s.table.shape[1], 0, False)
    assert need > 0
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.full((60, 20, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((60, 20), 7.0, device="cuda")
    for st in ([0, 50, 0, 50], [50, 0, 50, 0], [-9, 70, -9, 70], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 50]):
        st = torch.tensor(st, dtype=torch.int32, device="cuda")
        nv.kv_attention(q, s.cache, s.table, s.kv_lens, st, out=out[:50], lse=lse[:50], workspace=ws[:need])
        assert (ws[need:] == 0x5A).all() and (out[50:] == 7.0).all() and (lse[50:] == 7.0).all()


def test_attention_windows_past_every_context():
    """A window as long as int32 goes, contexts shorter than the new tokens: as without a window."""
    s = Sequences(23, [5, 300], 1, 64, 32).append()
    q = queries(6, 120, 2, 64).cuda()
    want = nv.kv_attention(q, s.cache, s.table, s.kv_lens, starts([40, 80]))
    for window in (300, 2 ** 31 - 2, 2 ** 31 - 1, 2 ** 40):
        assert torch.equal(nv.kv_attention(q, s.cache, s.table, s.kv_lens, starts([40, 80]), window=window), want)


def test_attention_leaves_other_rows_as_they_were():
    """A padded batch: rows before the first sequence, behind the last one and between them belong to nobody."""
    s = Sequences(13, [50, 600, 80], 2, 128, 32).append()
    q = queries(5, 40, 4, 128)
    st = torch.tensor([2, 5, 5, 29], dtype=torch.int32, device="cuda")
    out = torch.full((40, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((40, 4), 7.0, device="cuda")
    got = nv.kv_attention(q.cuda(), s.cache, s.table, s.kv_lens, st, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    for x in (out, lse):
        assert (x[:2] == 7.0).all() and (x[29:] == 7.0).all()
    check_attention(s, [3, 0, 24], q[2:29], out[2:29], lse[2:29], 128 ** -0.5)
    empty = nv.kv_attention(q[:0].cuda(), s.cache, s.table[:0], s.kv_lens[:0])
    assert empty.shape == (0, 4, 128)


def test_attention_of_queries_beside_other_columns():
    s = Sequences(14, [90, 33], 2, 128, 32).append()
    wide = queries(6, 2, 10, 128).cuda()
    q = wide[:, 3:7]
    assert torch.equal(nv.kv_attention(q, s.cache, s.table, s.kv_lens),
                       nv.kv_attention(q.contiguous(), s.cache, s.table, s.kv_lens))
    with pytest.raises(ValueError, match="heads of a token"):
        nv.kv_attention(wide[:, ::2], s.cache, s.table, s.kv_lens)
    with pytest.raises(ValueError, match="not a multiple"):
        nv.kv_attention(wide[:, :3], s.cache, s.table, s.kv_lens)
    with pytest.raises(ValueError, match="kv_lens"):
        nv.kv_attention(q, s.cache, s.table, s.kv_lens.long())
    with pytest.raises(nv.NVFP4Error):  # one token in another's place
        nv.kv_attention(wide[:1].expand(2, 10, 128)[:, :4], s.cache, s.table, s.kv_lens)
    with pytest.raises(nv.NVFP4Error) as e:
        nv.kv_attention(q, s.cache, s.table, s.kv_lens, scale=float("nan"))
    assert e.value.status == 1
    flat = q.contiguous()
    with pytest.raises(nv.NVFP4Error, match="out overlaps q"):
        nv.kv_attention(flat, s.cache, s.table, s.kv_lens, out=flat)


def test_workspace():
    s = Sequences(15, [3000, 10], 1, 128, 32).append()
    q = queries(2, 2, 4, 128).cuda()
    want = nv.kv_attention(q, s.cache, s.table, s.kv_lens)
    need = nv.kv_attention_workspace_size(2, 2, 4, 1, 128, 32, s.table.shape[1], 0, True)
    assert need > 0
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN where nothing is written
    assert torch.equal(nv.kv_attention(q, s.cache, s.table, s.kv_lens, workspace=ws[:need]), want)
    assert (ws[need:] == 0xFF).all()
    with pytest.raises(nv.NVFP4Error) as e:
        nv.kv_attention(q, s.cache, s.table, s.kv_lens, workspace=ws[:need - 16])
    assert e.value.status == 4


def test_pages_past_4_gib():
    """Offsets of pages and of queries' rows past 32 bits."""
    page, heads_, d = 256, 8, 128
    pages = (5 << 30) // nv.kv_page_bytes(heads_, d, page)
    cache = nv.KVCache.empty(pages, page, heads_, d)
    rng = np.random.default_rng(0)
    k, v = heads(rng, 300, heads_, d), heads(rng, 300, heads_, d)
    ids = torch.tensor([pages - 1, pages - 2], dtype=torch.int32, device="cuda")
    i = torch.arange(300, device="cuda")
    slots = (ids[i // page] * page + i % page).int()
    nv.kv_append(cache, k.cuda(), v.cuda(), slots)
    one = np.ones(heads_, np.float32)
    want = okv.cached(k.float().numpy(), v.float().numpy(), one, one)
    gk, gv = nv.kv_read(cache, slots, torch.float32)
    assert _same(_np(gk), want[0]) and _same(_np(gv), want[1])
    q = queries(1, 1, 8, d)
    out = nv.kv_attention(q.cuda(), cache, ids[None], torch.tensor([300], dtype=torch.int32, device="cuda"))
    ref = okv.attention(q.float().numpy(), *want, d ** -0.5, okv.visible(300, 1))
    assert np.abs(out.double().cpu().numpy() - ref[0]).max() <= 2.0 ** -7 * np.abs(ref[0]).max()
    # the same pages copied into a small cache hold the same tokens
    small = nv.KVCache(cache.data[ids.long()].contiguous(), cache.k_scale, cache.v_scale, d, page)
    sk, _ = nv.kv_read(small, torch.arange(300, dtype=torch.int32, device="cuda"), torch.float32)
    assert torch.equal(sk, gk)


def test_decoding_step_by_step():
    """A prompt and then single tokens, as a decoder layer uses the operators together: each step's output is that of
    the whole sequence at once, up to the order of the sums."""
    d, hq, hkv, page, n = 128, 8, 2, 32, 75
    rng = np.random.default_rng(4)
    x = torch.cat((heads(rng, n, hq, d), heads(rng, n, hkv, d), heads(rng, n, hkv, d)), 1).cuda()
    rope = torch.from_numpy(rope_table(128, d)).cuda()
    table = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32, device="cuda")
    i = torch.arange(n, device="cuda")
    slots = (table[0, i // page] * page + i % page).int()
    pos = i.int()

    def step(cache, a, b):
        q, k, v = x[a:b].split((hq, hkv, hkv), 1)
        q = nv.kv_append(cache, k, v, slots[a:b], q=q, positions=pos[a:b], rope=rope)
        lens = torch.tensor([b], dtype=torch.int32, device="cuda")
        return nv.kv_attention(q, cache, table, lens, starts([b - a]))

    whole_cache, cache = (nv.KVCache.empty(4, page, hkv, d, k_scale=0.01, v_scale=0.01) for _ in range(2))
    whole = step(whole_cache, 0, n)
    parts = [step(cache, 0, 40)] + [step(cache, t, t + 1) for t in range(40, n)]
    gap = (torch.cat(parts).float() - whole.float()).abs().max()
    assert float(gap) <= 2.0 ** -7 * float(whole.float().abs().max())
    assert torch.equal(nv.kv_read(cache, slots)[0], nv.kv_read(whole_cache, slots)[0])


def test_captured_step_follows_lengths_and_slots():
    """A decoding step in a graph, replayed with other tokens, slots, lengths and pages: bit-identical to eager calls."""
    d, hq, hkv, page, b = 128, 8, 2, 32, 3
    x = torch.zeros(b, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda")
    rope = torch.from_numpy(rope_table(4096, d)).cuda()
    table = torch.zeros(b, 100, dtype=torch.int32, device="cuda")
    lens, slots, pos = (torch.zeros(b, dtype=torch.int32, device="cuda") for _ in range(3))
    base = Sequences(20, [3100, 40, 900], hkv, d, page, spare=20).append()
    ws = torch.empty(nv.kv_attention_workspace_size(b, b, hq, hkv, d, page, 100, 0, True), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(b, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(b, hq, device="cuda")
    q_out = torch.empty(b, hq, d, dtype=torch.bfloat16, device="cuda")

    def step():
        q, k, v = x.split((hq, hkv, hkv), 1)
        nv.kv_append(base.cache, k, v, slots, q=q, q_out=q_out, positions=pos, rope=rope)
        nv.kv_attention(q_out, base.cache, table, lens, out=out, lse=lse, workspace=ws)

    def fill(seed):
        rng = np.random.default_rng(seed)
        x.copy_(heads(rng, b, hq + 2 * hkv, d))
        new = torch.tensor([rng.integers(1, n) for n in base.lens], dtype=torch.int32)
        lens.copy_(new)
        pos.copy_(new - 1)
        table[:, : base.table.shape[1]].copy_(base.table)
        at = base.table.cpu()[torch.arange(b), ((new - 1) // page).long()]
        slots.copy_(at * page + (new - 1) % page)

    fill(0)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(1, 6):
        fill(seed)
        before = base.cache.data.clone()
        out.fill_(3.0), ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone(), base.cache.data.clone()
        base.cache.data.copy_(before)
        step()
        assert torch.equal(out, got[0]) and torch.equal(lse, got[1]) and torch.equal(base.cache.data, got[2])


def test_two_streams_at_once():
    s = [Sequences(30 + i, [2500, 700], 2, 128, 32).append() for i in range(2)]
    q = [queries(i, 2, 8, 128).cuda() for i in range(2)]
    want = [nv.kv_attention(q[i], s[i].cache, s[i].table, s[i].kv_lens) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(nv.kv_attention(q[i], s[i].cache, s[i].table, s[i].kv_lens))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])
