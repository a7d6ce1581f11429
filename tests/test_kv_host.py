"""Refusals of the key/value cache's operators: by the library on the host,
before any HIP call, and by the Python binding before the library is reached."""

import os

import pytest
import torch

import bit_gemm_amd as nv

AT = {n: (1 << 30) * (i + 1) for i, n in enumerate(["k", "v", "q", "qo", "pos", "rope", "slots", "cache", "ks", "vs", "out",
                                                   "lse", "table", "lens", "starts", "ws"])}  # never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nv.LIB_PATH):
        from bit_gemm_amd import build
        build.build()
    return nv.lib()


def test_page_bytes(L):
    f = L.nvfp4_kv_page_bytes
    assert f(8, 128, 64) == 8 * 64 * (128 + 16) and f(1, 64, 32) == 32 * 72 and f(3, 256, 1024) == 3 * 1024 * 288
    for bad in ((0, 128, 64), (-1, 128, 64), (8, 96, 64), (8, 0, 64), (8, 128, 16), (8, 128, 48), (8, 128, 0),
                (8, 128, 1 << 17), (65537, 128, 64)):
        assert f(*bad) == 0, bad


def _append(L, **o):
    a = dict(k=AT["k"], kst=1024, v=AT["v"], vst=1024, q=AT["q"], qst=4096, qo=AT["qo"], qost=4096, qh=32, pos=AT["pos"],
             rope=AT["rope"], maxp=100, rot=128, il=0, slots=AT["slots"], t=5, cache=AT["cache"], pages=10, page=64, h=8,
             d=128, ks=AT["ks"], vs=AT["vs"])
    a.update(o)
    return L.nvfp4_kv_append(*a.values(), None)


def test_append(L):
    def f(**o):
        return _append(L, **o)

    assert f(d=96) == 2 and f(page=48) == 2 and f(page=16) == 2 and f(rot=16) == 2 and f(rot=160) == 2 and f(rot=-32) == 2
    assert "rope_dim" in L.nvfp4_last_error().decode()
    assert f(pages=1 << 26) == 2 and f(t=(1 << 27) + 1) == 2 and f(t=1 << 26) == 2  # slots, tokens, work-items
    assert f(t=-1) == 1 and f(pages=-1) == 1 and f(h=0) == 1 and f(k=None) == 1 and f(v=None) == 1 and f(slots=None) == 1
    assert f(q=None) == 1 and f(qo=None) == 1 and f(qh=0) == 1 and f(pos=None) == 1 and f(rope=None) == 1 and f(maxp=-1) == 1 and f(maxp=0) == 1
    assert f(cache=None) == 1 and f(ks=None) == 1 and f(vs=None) == 1
    assert f(kst=1016) == 1 and f(vst=0) == 1 and f(qst=-4096) == 1 and f(qost=4088) == 1 and f(kst=1 << 41) == 1
    assert f(kst=1028) == 3 and f(k=AT["k"] + 8) == 3 and f(qo=AT["qo"] + 2) == 3 and f(slots=AT["slots"] + 2) == 3
    assert f(rope=AT["rope"] + 4) == 3 and f(pos=AT["pos"] + 1) == 3 and f(cache=AT["cache"] + 8) == 3 and f(ks=AT["ks"] + 1) == 3
    assert f(t=0, k=None, v=None, q=None, qo=None, slots=None, pos=None, rope=None) == 0
    assert f(t=0, cache=None, pages=0) == 0


def test_append_refuses_overlaps(L):
    """Outputs that share memory with what other threads read; columns of one matrix do not."""
    cache_bytes = 10 * nv.kv_page_bytes(8, 128, 64)
    for name, size in (("k", 5 * 2048), ("v", 5 * 2048), ("q", 5 * 8192), ("slots", 20), ("pos", 20), ("rope", 51200), ("ks", 32)):
        for at in (AT[name] - cache_bytes + 16, AT[name], AT[name] + (size - 1) // 16 * 16):
            assert _append(L, cache=at) == 1, (name, at)
            assert "cache overlaps" in L.nvfp4_last_error().decode()
    for name in ("k", "v", "slots", "pos", "rope", "vs", "cache"):
        assert _append(L, qo=AT[name]) == 1, name
    assert _append(L, qo=AT["q"] + 16) == 1 and _append(L, qo=AT["q"], qost=4104) == 1
    # q, k and v as columns of one matrix of 48 heads; q_out over k's columns, over q's and v's
    row = 48 * 128
    fused = dict(k=AT["q"] + 2 * 4096, v=AT["q"] + 2 * 5120, kst=row, vst=row, qst=row, qost=row)
    assert _append(L, **fused, qo=AT["q"] + 16) == 1 and _append(L, **fused, qo=AT["q"] + 2 * row) == 1
    assert _append(L, **fused, qo=AT["q"] + 2 * 4096) == 1
    ok = 5 if torch.cuda.is_available() else 4  # past every check
    if not torch.cuda.is_available():
        assert _append(L, **fused, qo=AT["q"]) > ok and _append(L) > ok
        # q_out as 32 further columns of the same matrix
        wide = dict(fused, kst=row + 4096, vst=row + 4096, qst=row + 4096, qost=row + 4096)
        assert _append(L, **wide, qo=AT["q"] + 2 * row) > ok


def test_strides_past_any_memory(L):
    """Refused before spans of rows are computed, which would pass 64 bits."""
    for name in ("kst", "vst", "qst", "qost"):
        assert _append(L, **{name: (1 << 34) + 8}) == 1 and "2^34" in L.nvfp4_last_error().decode(), name


def test_read(L):
    def f(**o):
        a = dict(cache=AT["cache"], pages=10, page=64, h=8, d=128, ks=AT["ks"], vs=AT["vs"], slots=AT["slots"], t=5,
                 k=AT["k"], v=AT["v"], dt=0)
        a.update(o)
        return L.nvfp4_kv_read(*a.values(), None)

    assert f(dt=2) == 1 and f(k=None) == 1 and f(v=None) == 1 and f(slots=None) == 1 and f(t=-1) == 1 and f(h=-2) == 1
    assert f(d=32) == 2 and f(page=31) == 2 and f(t=1 << 26) == 2
    assert f(k=AT["k"] + 4) == 3 and f(slots=AT["slots"] + 3) == 3
    assert f(k=AT["v"]) == 1 and f(v=AT["cache"] + 64) == 1 and f(k=AT["slots"] - 10224) == 1
    assert f(t=0, k=None, v=None, slots=None) == 0


def test_attention(L):
    def f(**o):
        a = dict(q=AT["q"], qst=4096, cache=AT["cache"], pages=10, page=64, h=8, d=128, ks=AT["ks"], vs=AT["vs"],
                 table=AT["table"], tp=4, lens=AT["lens"], starts=AT["starts"], b=3, t=5, qh=32, scale=0.1, causal=1,
                 window=0, out=AT["out"], lse=AT["lse"], ws=AT["ws"], wsb=1 << 29)
        a.update(o)
        return L.nvfp4_kv_attention(*a.values(), None)

    assert f(qh=33) == 1 and f(qh=0) == 1 and f(b=-1) == 1 and f(b=65537) == 1 and f(t=-1) == 1
    assert f(scale=float("nan")) == 1 and f(scale=float("inf")) == 1 and f(window=-1) == 1 and f(window=4, causal=0) == 1
    assert f(tp=-1) == 1 and f(tp=1 << 26) == 1 and f(starts=None) == 1 and f(q=None) == 1 and f(out=None) == 1
    assert f(lens=None) == 1 and f(table=None) == 1 and f(cache=None) == 1 and f(pages=0, cache=None) == 1
    assert f(d=80) == 2 and f(page=33) == 2 and f(t=1 << 26) == 2
    assert f(qst=4088) == 1 and f(qst=4100) == 3 and f(q=AT["q"] + 8) == 3 and f(out=AT["out"] + 8) == 3
    assert f(lse=AT["lse"] + 2) == 3 and f(lens=AT["lens"] + 1) == 3 and f(table=AT["table"] + 2) == 3
    for name in ("q", "cache", "table", "lens", "starts", "ks", "vs", "lse", "ws"):
        assert f(out=AT[name], tp=64) == 1, name
    assert f(ws=AT["q"], tp=64) == 1 and f(lse=AT["lens"]) == 1
    assert f(b=0) == 0 and f(t=0, b=0, q=None, out=None, lens=None, table=None) == 0
    size = L.nvfp4_kv_attention_workspace_size
    need = size(3, 5, 32, 8, 128, 64, 64, 0, 0)
    assert need > 0 and f(tp=64, wsb=need - 1) == 4 and f(tp=64, ws=None) == 1 and f(tp=64, ws=AT["ws"] + 8) == 3
    for bad in ((0, 5, 32, 8, 128, 64, 64, 0, 0), (3, 5, 33, 8, 128, 64, 64, 0, 0), (3, 5, 32, 8, 96, 64, 64, 0, 0),
                (3, 5, 32, 8, 128, 64, 64, 0, 1), (3, 5, 32, 8, 128, 64, 0, 0, 0), (3, 0, 32, 8, 128, 64, 64, 0, 0),
                (3, 5, 32, 8, 128, 64, 64, -1, 0)):
        assert size(*bad) == 0, bad


def test_attention_refuses_more_work_items_than_a_launch_holds(L):
    """More workgroups of 256 threads than 2^24, of 512 (the tiles) than 2^23: below them memory is what bounds a call."""
    h, b = 256, 1 << 15  # 2^23 pairs of a sequence and a head, 128 rows and more of each pair
    t = (1 << 30) // h
    assert L.nvfp4_kv_attention_path(b, t, h, h, 128, 64, 4, 0, 0) == 256
    assert L.nvfp4_kv_attention(AT["q"], h * 128, 1 << 41, 10, 64, h, 128, AT["ks"], AT["vs"], AT["table"], 4, AT["lens"],
                                AT["starts"], b, t, h, 0.1, 1, 0, 1 << 42, None, None, 0, None) == 2
    assert "in one call" in L.nvfp4_last_error().decode()


def test_binding_refuses():
    cache = nv.KVCache.empty(4, 64, 2, 64, "cpu")
    t = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="KVCache"):
        nv.kv_append(cache.data, t, t, i)
    for call in (lambda: nv.kv_append(cache, t, t, i), lambda: nv.kv_read(cache, i),
                 lambda: nv.kv_attention(t, cache, i[:, None], i)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="no cache"):
        nv.KVCache.empty(4, 48, 2, 64, "cpu")
    with pytest.raises(ValueError, match="no cache"):
        nv.kv_read(nv.KVCache(cache.data, cache.k_scale, cache.v_scale, 80, 64), i)
    with pytest.raises(ValueError, match="cache.data"):
        nv.kv_read(nv.KVCache(cache.data[0], cache.k_scale, cache.v_scale, 64, 64), i)
    with pytest.raises(ValueError, match="k_scale"):
        nv.kv_read(nv.KVCache(cache.data, None, cache.v_scale, 64, 64), i)
    with pytest.raises(ValueError, match="v_scale"):
        nv.kv_read(nv.KVCache(cache.data, cache.k_scale, cache.v_scale[:1], 64, 64), i)
    with pytest.raises(ValueError, match="shape"):
        nv.kv_read(nv.KVCache(cache.data[:, 16:].contiguous(), cache.k_scale, cache.v_scale, 64, 64), i)


def test_attention_paths(L):
    """The sizes that choose each kernel, by the work at hand."""
    def path(t, hq, h, d, pages=64, b=1, window=0, one=0):
        return L.nvfp4_kv_attention_path(b, t, hq, h, d, 64, pages, window, one)

    assert path(1, 32, 8, 128, 1 << 20, one=1) == 16 and path(64, 64, 8, 128, 1 << 20, 64, one=1) == 16
    assert path(1000, 32, 8, 128, 16) == 16 and path(2000, 32, 8, 128, 32) == 32 and path(4096, 32, 8, 128) == 256
    assert path(4096, 32, 8, 128, window=100) == 16  # a short window is little work
    assert path(300, 5, 5, 64, 5) == 16 and path(4096, 32, 8, 64) == 32 and path(1 << 20, 32, 8, 64, 1 << 20) == 32
    assert path(1000, 16, 4, 256, 16) == 16 and path(4096, 16, 4, 256) == 128
    assert path(0, 32, 8, 128) == -1 and path(5, 33, 8, 128) == -1 and path(5, 32, 8, 128, one=1) == -1
    size = L.nvfp4_kv_attention_workspace_size
    assert size(1, 1, 32, 8, 128, 64, 16, 0, 1) == 0  # 1024 tokens: not split
    assert size(1, 1, 32, 8, 128, 64, 32, 0, 1) > 0 and size(1, 1, 32, 8, 128, 64, 32, 500, 1) == 0
    assert size(64, 64, 32, 8, 128, 64, 32, 0, 1) == 0  # 2048 tokens of many: not split
    assert size(64, 64, 32, 8, 128, 64, 64, 0, 1) > 0 and size(1, 4096, 32, 8, 128, 64, 64, 0, 0) == 0
