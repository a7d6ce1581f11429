"""Inputs and error bounds shared by the tests of the key/value cache."""

import numpy as np
import torch

import bit_gemm_amd as nv
import oracle.kv as okv

UBF16 = 2.0 ** -8  # half a step of bf16, relative
UF16 = 2.0 ** -11  # of fp16
U32 = 2.0 ** -24


def rope_table(positions, rot, base=10000.0):
    """float32 [positions, rot]: cosines, then sines."""
    angle = np.arange(positions)[:, None] * base ** (-np.arange(0, rot, 2) / max(rot, 1))
    return np.concatenate((np.cos(angle), np.sin(angle)), 1).astype(np.float32)


def bf16(x):
    """float32 numpy -> bf16 tensor on the host."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16()


def heads(rng, tokens, n, d):
    """Keys or values with channels of different sizes, as bf16 on the host."""
    return bf16(rng.standard_normal((tokens, n, d)) * np.exp(rng.standard_normal((n, d))))


class Sequences:
    """Contexts of the given lengths in scattered pages of one cache."""

    def __init__(self, seed, lens, heads_, d, page, spare=2, fill=None, table_pages=None):
        rng = np.random.default_rng(seed)
        self.lens, self.d, self.page = list(lens), d, page
        per = [-(-n // page) for n in lens]
        total = sum(per) + spare
        ids = rng.permutation(total)[: sum(per)].astype(np.int32)
        ks = (rng.uniform(4, 40, heads_) / 2688).astype(np.float32)
        vs = (rng.uniform(4, 40, heads_) / 2688).astype(np.float32)
        self.cache = nv.KVCache.empty(total, page, heads_, d, "cuda", torch.from_numpy(ks).cuda(), torch.from_numpy(vs).cuda())
        self.cache.data.fill_(0xFF if fill is None else fill)  # NaN scales, or as asked, where nothing is written
        width = max(per + [1]) if table_pages is None else table_pages
        table = np.full((len(lens), width), -7, np.int32)
        self.k, self.v, slots = [], [], []
        at = 0
        for b, n in enumerate(lens):
            table[b, : per[b]] = ids[at : at + per[b]]
            i = np.arange(n)
            slots.append(table[b, i // page].astype(np.int64) * page + i % page)
            at += per[b]
            self.k.append(heads(rng, n, heads_, d))
            self.v.append(heads(rng, n, heads_, d))
        self.slots = torch.from_numpy(np.concatenate(slots + [np.zeros(0, np.int64)]).astype(np.int32)).cuda()
        self.table = torch.from_numpy(table).cuda()
        self.kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.scales = ks, vs

    def append(self):
        k, v = torch.cat(self.k), torch.cat(self.v)
        nv.kv_append(self.cache, k.cuda(), v.cuda(), self.slots)
        return self

    def held(self, b):
        """What the cache holds for sequence b, by the oracle."""
        return okv.cached(self.k[b].float().numpy(), self.v[b].float().numpy(), *self.scales)


def queries(seed, tokens, q_heads, d, size=1.0):
    rng = np.random.default_rng(seed)
    return bf16(size * rng.standard_normal((tokens, q_heads, d)) * np.exp(0.5 * rng.standard_normal((q_heads, d))))


def starts(new):
    return torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")


def bounds(out, lse, weight, size, n, d):
    """How far out and lse may be off (float64 arrays as oracle.kv.attention returns them).

    A logit's products are exact; their sum in any order in fp32 and the factors' roundings are off by at most
    (d + 8) u of the sum of magnitudes `size`, the argument of the exponential (at most 160 in magnitude where p is
    not negligible) and the exponential itself by 2^-16 (160 u and 2^-22, with room).  That relative error of every p
    counts twice in the quotient; p's rounding to fp16 is 2^-11, or 2^-32 of the row's largest p for each of n tokens;
    sums of n terms add n u; the output is rounded to bf16 once.
    """
    logit = (d + 8) * U32 * size + 2.0 ** -16
    rel = 2 * logit + UF16 + 2 * (n + 16) * U32
    largest = np.maximum(weight, np.abs(out))
    floor = n * 2.0 ** -32 * largest.max(-1, keepdims=True) if out.size else 0.0
    return (rel[..., None] * weight + UBF16 * (np.abs(out) + rel[..., None] * weight) + floor + 2.0 ** -126,
            logit + (n + 16) * U32 + 8 * U32 * np.abs(np.where(np.isfinite(lse), lse, 0)))


def check_attention(seqs, new, q, out, lse, scale, causal=True, window=0):
    """out, lse (tensors) of the sequences' last `new` tokens against the oracle."""
    at = 0
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, (n, m) in enumerate(zip(seqs.lens, new)):
        k, v = seqs.held(b)
        seen = okv.visible(n, m, causal, window)
        ref = okv.attention(q[at : at + m].float().numpy(), k, v, scale, seen)
        tol_o, tol_l = bounds(*ref, max(n, 1), seqs.d)
        got_o, got_l = out[at : at + m], lse[at : at + m]
        empty = np.isneginf(ref[1])
        assert np.array_equal(np.isneginf(got_l), empty), b
        assert (got_o[empty] == 0).all(), b
        err_o, err_l = np.abs(got_o - ref[0]), np.abs(np.where(empty, 0, got_l) - np.where(empty, 0, ref[1]))
        assert (err_o <= tol_o).all(), (b, float((err_o / tol_o).max()))
        assert (err_l <= tol_l).all(), (b, float((err_l / tol_l).max()))
        at += m
