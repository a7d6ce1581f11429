"""kv_attention in every form that a plan can give it, under every mask: windows
on whole and on split contexts, split contexts that every token sees, both forms
of the join, more sequences than a wave has lanes; and rows of tokens whose
offsets pass 32 bits."""

import numpy as np
import pytest
import torch

import bit_gemm_amd as nv
import oracle.kv as okv
from kv_cases import Sequences, bounds, check_attention, heads, queries, rope_table, starts
from kv_plan_cases import CALLS, check_plan

pytestmark = pytest.mark.gpu


def _check_some(s, new, q, out, lse, scale, causal, window, seed):
    """The first and last new tokens of each sequence and a few between, all heads, against the oracle."""
    rng = np.random.default_rng(seed)
    few = 8 if len(new) < 20 else 2
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    at = 0
    for b, (n, m) in enumerate(zip(s.lens, new)):
        pick = np.unique(np.concatenate((np.arange(m)[:2], np.arange(m)[-2:], rng.integers(0, max(m, 1), few if m else 0))))
        k, v = s.held(b)
        ref = okv.attention(q[at:at + m][pick].float().numpy(), k, v, scale, okv.visible(n, m, causal, window)[pick])
        tol_o, tol_l = bounds(*ref, max(n, 1), s.d)
        got_o, got_l = out[at:at + m][pick], lse[at:at + m][pick]
        empty = np.isneginf(ref[1])
        assert np.array_equal(np.isneginf(got_l), empty) and (got_o[empty] == 0).all(), b
        err_o = np.abs(got_o - ref[0])
        err_l = np.abs(np.where(empty, 0, got_l) - np.where(empty, 0, ref[1]))
        assert (err_o <= tol_o).all() and (err_l <= tol_l).all(), (b, (err_o / tol_o).max(), (err_l / tol_l).max())
        at += m
    assert np.isfinite(out).all() and not np.isnan(lse).any()


@pytest.mark.parametrize("c", CALLS, ids=str)
def test_attention_in_every_form(c):
    check_plan(c)
    print("kv attention", c, flush=True)
    s = Sequences(41, c.lens, c.hkv, c.d, c.page, table_pages=c.table_pages).append()
    q = queries(42, sum(c.new), c.hq, c.d)
    first = None if c.one_each else starts(c.new)

    def call():
        return nv.kv_attention(q.cuda(), s.cache, s.table, s.kv_lens, first, causal=c.causal, window=c.window, return_lse=True)

    out, lse = call()
    _check_some(s, c.new, q, out, lse, c.d ** -0.5, c.causal, c.window, 43)
    again = call()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hq,hkv,window", [([31, 0, 300, 64], 8, 2, 0), ([3000, 70], 8, 1, 0), ([900, 33], 34, 2, 100)])
def test_single_tokens_named_by_their_rows(d, lens, hq, hkv, window):
    """q_starts of one token each: the call without them, up to the order of its sums."""
    s = Sequences(44, lens, hkv, d, 32).append()
    q = queries(45, len(lens), hq, d)
    for first in (None, starts([1] * len(lens))):
        out, lse = nv.kv_attention(q.cuda(), s.cache, s.table, s.kv_lens, first, window=window, return_lse=True)
        check_attention(s, [1] * len(lens), q, out, lse, d ** -0.5, True, window)


def test_rows_of_tokens_past_32_bits():
    """Tokens 2^30 elements and more apart: q, k, v and the rotated q as columns of one matrix of 4.3 GB, whose last
    row's offset passes 2^31 elements and 2^32 bytes."""
    n, hq, hkv, d = 3, 4, 2, 128
    width = 2 * hq + 2 * hkv  # q, k, v, q_out
    stride = (1 << 30) + 64
    flat = torch.empty((n - 1) * stride + width * d, dtype=torch.bfloat16, device="cuda")
    far = flat.as_strided((n, width, d), (stride, d, 1))
    assert (n - 1) * stride > 2 ** 31
    near = heads(np.random.default_rng(1), n, width, d).cuda()
    far.copy_(near)
    near, far = ([*x.split((hq, hkv, hkv, hq), 1)] for x in (near, far))
    rope = torch.from_numpy(rope_table(8, d)).cuda()
    slots = torch.tensor([5, 40, 70], dtype=torch.int32, device="cuda")
    lens = torch.tensor([96], dtype=torch.int32, device="cuda")
    table = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    results = []
    for q, k, v, q_out in (near, far):
        cache = nv.KVCache.empty(3, 32, hkv, d, k_scale=0.01, v_scale=0.01)
        cache.data.zero_()
        nv.kv_append(cache, k, v, slots, q=q, q_out=q_out, positions=slots.remainder(8), rope=rope)
        out, lse = nv.kv_attention(q_out, cache, table, lens, starts([n]), return_lse=True)
        results.append((q_out.clone(), cache.data.clone(), out, lse))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert not torch.equal(results[0][0], near[0].contiguous())
