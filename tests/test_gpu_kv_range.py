"""Attention over the NVFP4 key/value cache at the ends of its numbers' range:
infinities and NaN in queries, rows of queries of very different sizes, head
scales next to fp32's least, factors past its largest."""

import numpy as np
import pytest
import torch

import bit_gemm_amd as nv
import oracle.kv as okv
from kv_cases import Sequences, check_attention, queries, starts
from test_gpu_kv import PATHS, _table_for

pytestmark = pytest.mark.gpu

EVERY_PATH = pytest.mark.parametrize("d,rows", PATHS)
INF, NAN = float("inf"), float("nan")


# ------------------------------------------------- infinities and NaN in queries


@EVERY_PATH
@pytest.mark.parametrize("scale", [None, -0.3, 0.0])
def test_queries_that_are_not_finite_give_nan(d, rows, scale):
    """A row of q that holds an infinity or a NaN is NaN in out and lse wherever it sees a token: each of its logits is
    NaN or an infinity, also where all of them are -inf.  Rows that see nothing are as without it, and so are all other
    rows within the bounds of any row: rows of one wave raise their bounds together, and the exponent of a logit is
    s f - m rounded once where none is raised and s f rounded before m is taken off where one is, so that a neighbour's
    NaN may change a row by such a rounding (2^-24 of the logit), which `bounds` counts."""
    lens, new = [70, 200, 5], [40, 150, 9]
    pages = _table_for(rows, lens, new, 4, 2, d, 32, 0)
    print("kv attention infinite queries", d, rows, scale, flush=True)
    s = Sequences(31, lens, 2, d, 32, table_pages=pages)
    for k in s.k:
        k[:, :, 3], k[:, :, 4] = 50.0, -50.0  # of one sign each in every token
        k[:, :, 16:32] = 0.0
    s.append()
    q = queries(32, sum(new), 4, d)
    bad = q.clone()
    at = {(1, 0): {3: -INF}, (5, 1): {3: INF}, (17, 2): {4: INF}, (39, 3): {7: NAN}, (40, 0): {20: INF}, (63, 1): {d - 1: -INF},
          (100, 2): {3: INF, 4: INF}, (101, 3): {3: -INF, 4: INF}, (189, 0): {3: -INF, 9: NAN}, (188, 0): {4: -INF},
          (190, 1): {3: -INF}, (193, 3): {5: NAN}, (194, 0): {3: -INF}, (198, 2): {4: INF}}  # 190 .. 193 see nothing
    poisoned = torch.zeros(sum(new), 4, dtype=torch.bool)
    for (t, h), elements in at.items():
        for i, x in elements.items():
            bad[t, h, i] = x
        poisoned[t, h] = not 190 <= t < 194
    args = s.cache, s.table, s.kv_lens, starts(new)
    scale = d ** -0.5 if scale is None else scale
    want, want_lse = nv.kv_attention(q.cuda(), *args, scale=scale, return_lse=True)
    out, lse = nv.kv_attention(bad.cuda(), *args, scale=scale, return_lse=True)
    assert torch.equal(torch.isnan(out).all(-1).cpu(), poisoned) and torch.equal(torch.isnan(lse).cpu(), poisoned)
    at = poisoned.cuda()
    check_attention(s, new, q, torch.where(at[..., None], want, out), torch.where(at, want_lse, lse), scale)
    assert (out[190:194] == 0).all() and torch.isneginf(lse[190:194]).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_queries_that_are_not_finite_over_a_split_context(d):
    s = Sequences(33, [5000, 3000], 1, d, 32)
    for k in s.k:
        k[:, :, 3] = 50.0
    s.append()
    q = queries(34, 2, 8, d)
    bad = q.clone()
    bad[0, 1, 3], bad[0, 2, 3], bad[1, 7, 9] = -INF, INF, NAN
    assert nv.kv_attention_workspace_size(2, 2, 8, 1, d, 32, s.table.shape[1], 0, True) > 0
    want, want_lse = nv.kv_attention(q.cuda(), s.cache, s.table, s.kv_lens, return_lse=True)
    out, lse = nv.kv_attention(bad.cuda(), s.cache, s.table, s.kv_lens, return_lse=True)
    at = torch.zeros(2, 8, dtype=torch.bool, device="cuda")
    at[0, 1] = at[0, 2] = at[1, 7] = True
    assert torch.equal(torch.isnan(out).all(-1), at) and torch.equal(torch.isnan(lse), at)
    check_attention(s, [1, 1], q, torch.where(at[..., None], want, out), torch.where(at, want_lse, lse), d ** -0.5)


# ------------------------------------------------------ queries of many sizes


@EVERY_PATH
@pytest.mark.parametrize("spread", [20, 32, 33, 37, 40, 60, 150])
def test_queries_of_very_different_sizes(d, rows, spread):
    """Elements 2^-spread of the row's largest decide the softmax where the keys are zero at the larger ones: nothing
    of a finite query may be lost to a number format shared by the row.  Rows of ordinary queries lie between."""
    lens, new = [150, 700], [40, 33]
    pages = _table_for(rows, lens, new, 3, 1, d, 32, 0)
    print("kv attention spread queries", d, rows, spread, flush=True)
    s = Sequences(35, lens, 1, d, 32, table_pages=pages)
    for k in s.k:
        k[:, :, 16:32] = 0.0
    s.append()
    q = queries(36, sum(new), 3, d)
    large = q[:, :, 16:32].clone()
    q[:, :, 16:32] = 0.0
    wide = torch.arange(sum(new)) % 4 != 1
    # the largest at 2^(spread / 2) and the rest at 2^(-spread / 2), which scale makes up for; other rows: at the rest's size
    down = 2.0 ** -(spread // 2)
    q = (q.float() * down).bfloat16()
    q[:, :, 16:32] = torch.where(wide[:, None, None], large.float() * 2.0 ** (spread - spread // 2), large.float() * down).bfloat16()
    scale = d ** -0.5 / down
    out, lse = nv.kv_attention(q.cuda(), s.cache, s.table, s.kv_lens, starts(new), scale=scale, return_lse=True)
    check_attention(s, new, q, out, lse, scale)


@EVERY_PATH
def test_one_row_of_very_different_sizes_among_ordinary_ones(d, rows):
    """One row in another wave (and most workgroups) than the rest: both kinds of operands in one call."""
    lens, new = [400, 900], [300, 130]
    pages = _table_for(rows, lens, new, 3, 1, d, 32, 0)
    print("kv attention one spread row", d, rows, flush=True)
    s = Sequences(39, lens, 1, d, 32, table_pages=pages)
    for k in s.k:
        k[:, :, 16:32] = 0.0
    s.append()
    q = queries(40, sum(new), 3, d)
    for t, h in ((71, 1), (250, 0), (429, 2)):
        q[t, h, 16:32] = (q[t, h, 16:32].float() * 2.0 ** 45).bfloat16()
    out, lse = nv.kv_attention(q.cuda(), s.cache, s.table, s.kv_lens, starts(new), return_lse=True)
    check_attention(s, new, q, out, lse, d ** -0.5)


def test_one_small_query_element_beside_a_large_one():
    """q = (2^24, 1.4453125 * 2^-12, 0, ..) and a key that is 0 in the first element and 2688 in the second: 0.948."""
    d = 128
    cache = nv.KVCache.empty(1, 32, 1, d)
    k = torch.zeros(2, 1, d, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 1] = 2688.0
    nv.kv_append(cache, k, torch.ones_like(k), torch.arange(2, dtype=torch.int32, device="cuda"))
    assert float(nv.kv_read(cache, torch.zeros(1, dtype=torch.int32, device="cuda"))[0][0, 0, 1]) == 2688.0
    q = torch.zeros(1, 1, d, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0], q[0, 0, 1] = 2.0 ** 24, 1.4453125 * 2.0 ** -12
    i32 = dict(dtype=torch.int32, device="cuda")
    _, lse = nv.kv_attention(q, cache, torch.zeros(1, 1, **i32), torch.tensor([2], **i32), scale=1.0, return_lse=True)
    want = np.log(1.0 + np.exp(2688.0 * 1.4453125 * 2.0 ** -12))
    assert abs(float(lse[0, 0]) - want) <= 2.0 ** -15  # as in kv_cases.bounds


# ------------------------------------------------------------ factors


@EVERY_PATH
@pytest.mark.parametrize("power", [-100, -119, -122])
def test_value_scales_next_to_the_least(d, rows, power):
    """Values and their head's scale times 2^power: the same codes, the output 2^power of what it was."""
    lens, new = [150, 2700], [40, 33]
    pages = _table_for(rows, lens, new, 3, 2, d, 32, 0) if rows != 16 else -(-max(lens) // 32)
    print("kv attention value scales", d, rows, power, flush=True)
    s = Sequences(37, lens, 3, d, 32, table_pages=pages)
    s.v = [(v.float().clamp(-30, 30).bfloat16()) for v in s.v]
    s.append()
    q = queries(38, sum(new), 3, d)
    want, want_lse = nv.kv_attention(q.cuda(), s.cache, s.table, s.kv_lens, starts(new), return_lse=True)
    cache = nv.KVCache(s.cache.data, s.cache.k_scale, s.cache.v_scale * 2.0 ** power, d, 32)
    out, lse = nv.kv_attention(q.cuda(), cache, s.table, s.kv_lens, starts(new), return_lse=True)
    assert torch.equal(lse, want_lse)
    # the scale times 2^power may be subnormal: the output then goes with what is left of it
    ratio = (cache.v_scale.double() / s.cache.v_scale.double())[None, :, None]
    exact = want.double() * ratio
    # each side rounded to bf16 once, the quotients of fp32 before; subnormal results to steps of 2^-133
    assert ((out.double() - exact).abs() <= 2.0 ** -7 * (1 + 2.0 ** -8) * exact.abs() + 2.0 ** -133).all()
    assert (out != 0).any()


def test_a_factor_past_fp32():
    """scale * k_scale / the row's power of two passes fp32's largest number: tokens whose logit is 0 share the row,
    those far below it are not seen."""
    for d, tokens in ((64, 1), (128, 1), (128, 40), (256, 1)):
        n = 100
        k = torch.zeros(n, 1, d, dtype=torch.bfloat16)
        k[:, 0, 5] = -6.0
        k[[7, 33], 0, 5] = 0.0
        v = torch.zeros(n, 1, d, dtype=torch.bfloat16)
        v[7], v[33] = 6.0, 3.0
        cache = nv.KVCache.empty(4, 32, 1, d)
        nv.kv_append(cache, k.cuda(), v.cuda(), torch.arange(n, dtype=torch.int32, device="cuda"))
        q = torch.zeros(tokens, 2, d, dtype=torch.bfloat16, device="cuda")
        q[:, :, 5] = 2.0 ** 100
        table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
        out, lse = nv.kv_attention(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), starts([tokens]),
                                   scale=1e20, return_lse=True)
        assert (out == 4.5).all(), d
        assert ((lse - np.log(2.0)).abs() <= 2.0 ** -20).all(), d


def test_finite_logits_under_a_factor_past_fp32():
    """As above, with finite logits: of elements 2^-30 of the row's largest, at which the keys are 0."""
    for d, tokens in ((64, 1), (128, 1), (128, 40), (256, 1)):
        k = torch.zeros(40, 1, d, dtype=torch.bfloat16)
        k[:, 0, 17] = 3.0
        k[9, 0, 17] = 6.0
        v = torch.zeros(40, 1, d, dtype=torch.bfloat16)
        v[9] = 5.0  # (the nearest codes: 4 and 6, times the block's scale 5 / 6 rounded to 0.8125)
        cache = nv.KVCache.empty(2, 32, 1, d)
        slots = torch.arange(40, dtype=torch.int32, device="cuda")
        nv.kv_append(cache, k.cuda(), v.cuda(), slots)
        held_k, held_v = nv.kv_read(cache, slots, torch.float32)
        q = torch.zeros(tokens, 2, d, dtype=torch.bfloat16, device="cuda")
        q[:, :, 5], q[:, :, 17] = 2.0 ** 100, 2.0 ** 70
        table = torch.arange(2, dtype=torch.int32, device="cuda")[None]
        out, lse = nv.kv_attention(q, cache, table, torch.tensor([40], dtype=torch.int32, device="cuda"), starts([tokens]),
                                   scale=2.0 ** 45, return_lse=True, causal=False)
        want = float(held_k[9, 0, 17]) * 2.0 ** 115
        # the logit's factors and the return to natural logarithms are each rounded in fp32 (2^-24), five times at most
        assert ((lse.double() - want).abs() <= 5 * 2.0 ** -24 * want).all(), d
        assert torch.equal(out, held_v[9].bfloat16().expand_as(out)), d
