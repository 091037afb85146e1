"""CPU pins of the attention cache's plain forms, and the entry points' refusals (nothing is launched)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import cache_ref as ref
import oracle

E_OK, E_NULL, E_SHAPE, E_ALIGN, E_DTYPE, E_WS = 0, -1, -2, -3, -4, -5
NULL = ctypes.c_void_p(0)


def P(addr):
    return ctypes.c_void_p(addr)


Q, K, V, W, S = P(0x10000), P(0x20000), P(0x30000), P(0x40000), P(0x50000)
CACHE = [P(0x100000), P(0x200000), P(0x300000), P(0x400000)]


@pytest.fixture(scope="module")
def lib():
    import gemm_e2m1_lut_amd as g
    return g.load_library()


# ------------------------------------------------------------ plain forms --

def test_encode_matches_the_oracle():
    """bf16 rows: the codes and scales of mxfp4_quantize."""
    r = np.random.default_rng(1)
    bits = (r.standard_normal((64, 128)) * np.exp2(r.integers(-20, 20, (64, 1)))).astype(np.float32).view(np.uint32) >> 16
    bits = bits.astype(np.uint16)
    x = (bits.astype(np.uint32) << 16).view(np.float32)
    codes, scales = ref.encode(x)
    want = oracle.mxfp4_quantize(bits)
    assert np.array_equal(codes, want[0]) and np.array_equal(scales, want[1])


def test_encode_ties_and_ends():
    x = np.zeros((1, 32))
    x[0, :10] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7, -0.75]
    codes, scales = ref.encode(x)
    assert scales.tolist() == [[127]]
    n = np.stack([codes & 15, codes >> 4], -1).reshape(-1)[:10]
    assert n.tolist() == [6, 0, 2, 2, 4, 4, 6, 6, 7, 10]
    assert ref.encode(np.full((1, 32), 2.0**-140))[1].tolist() == [[0]]
    assert ref.encode(np.full((1, 32), 3e38))[1].tolist() == [[252]]
    for bad in (np.nan, np.inf, -np.inf):
        x[0, 3] = bad
        codes, scales = ref.encode(x)
        assert scales.tolist() == [[255]] and not codes.any()
        assert np.isnan(ref.decode(codes, scales)).all()


def test_attention_form_against_a_softmax():
    """Against torch's softmax in 64 bits, and what the masks leave."""
    r = np.random.default_rng(2)
    q, k, v = r.standard_normal((5, 4, 64)), r.standard_normal((9, 2, 64)), r.standard_normal((9, 2, 64))
    out, bound = ref.attention(q, k, v, 0.3, True, 3)
    for h in range(4):
        s = torch.from_numpy(q[:, h] @ k[:, h // 2].T) * 0.3
        for i in range(5):
            p = 4 + i
            lo = p - 2
            w = torch.softmax(s[i, lo:p + 1], 0).numpy() @ v[lo:p + 1, h // 2]
            assert np.allclose(out[i, h], w, rtol=1e-12)
    assert (bound > 0).all() and (bound < 0.25).all()
    assert not ref.attention(q, k[:0], v[:0], 0.3, True, 0)[0].any()
    out, _ = ref.attention(q, k[:3], v[:3], 0.3, True, 0)   # the first two queries come before the first key
    assert not out[:2].any() and out[2:].any()
    s, _ = ref.attention(q, k, v, 0.3, False, 0, sinks=np.full(4, -1e9))
    assert np.allclose(s, ref.attention(q, k, v, 0.3, False, 0)[0])


# --------------------------------------------------------------- refusals --

def write(lib, k=K, v=V, dtype=1, ks=1024, vs=1024, slots=S, cache=None, tokens=4, heads=8, dim=128, pages=4, page=16,
          err=NULL):
    return lib.mxfp4_cache_write(k, v, dtype, ks, vs, slots, *(cache or CACHE), tokens, heads, dim, pages, page, err, NULL)


def rope(lib, qkv=Q, dtype=1, stride=6144, wq=NULL, wk=NULL, eps=1e-6, table=W, max_pos=100, rot=128, inter=0, pos=K,
         slots=S, out=V, cache=None, tokens=4, heads=32, kv=8, dim=128, pages=4, page=16, err=NULL):
    return lib.norm_rope_mxfp4_cache_write(qkv, dtype, stride, wq, wk, eps, table, max_pos, rot, inter, pos, slots, out,
                                           *(cache or CACHE), tokens, heads, kv, dim, pages, page, err, NULL)


def read(lib, cache=None, slots=S, k=K, v=V, tokens=4, heads=8, dim=128, pages=4, page=16, err=NULL):
    return lib.mxfp4_cache_read(*(cache or CACHE), slots, k, v, tokens, heads, dim, pages, page, err, NULL)


def attend(lib, q=Q, stride=4096, cache=None, table=W, lens=K, offsets=V, sinks=NULL, scale=0.1, causal=1, window=0,
           out=S, ws=P(0x1000000), ws_bytes=None, tokens=4, seqs=2, heads=32, kv=8, dim=128, pages=4, page=16, width=3,
           err=NULL):
    if ws_bytes is None:
        ws_bytes = 1 << 40
    return lib.mxfp4_attention(q, stride, *(cache or CACHE), table, lens, offsets, sinks, scale, causal, window, out, ws,
                               ws_bytes, tokens, seqs, heads, kv, dim, pages, page, width, err, NULL)


BAD_CACHE_SHAPES = [dict(dim=96), dict(dim=0), dict(dim=256), dict(page=8), dict(page=24), dict(page=0), dict(page=2**17),
                    dict(pages=-1), dict(pages=2**31), dict(tokens=-1), dict(tokens=2**26 + 1)]


@pytest.mark.parametrize("bad", BAD_CACHE_SHAPES, ids=str)
@pytest.mark.parametrize("call", [write, rope, read, attend], ids=lambda f: f.__name__)
def test_cache_shapes_refused(lib, call, bad):
    assert call(lib, **bad) == E_SHAPE


@pytest.mark.parametrize("call", [write, rope, read, attend], ids=lambda f: f.__name__)
def test_cache_pointers_refused(lib, call):
    for i in range(4):
        cache = list(CACHE)
        cache[i] = NULL
        assert call(lib, cache=cache) == E_NULL
        cache[i] = P(0x100008)
        assert call(lib, cache=cache) == E_ALIGN
    assert call(lib, err=P(0x2)) == E_ALIGN


def test_write_refusals(lib):
    assert write(lib, dtype=2) == E_DTYPE
    assert write(lib, tokens=0, k=NULL, v=NULL, slots=NULL) == E_OK
    assert write(lib, heads=0) == E_SHAPE and write(lib, heads=4097) == E_SHAPE
    for bad in (1023, 1016, 1028, -1024, 2**60):
        assert write(lib, ks=bad) == E_SHAPE and write(lib, vs=bad) == E_SHAPE
    assert write(lib, ks=1028, k=NULL, dtype=0) == E_NULL    # 16 bytes of fp32
    for name in ("k", "v", "slots"):
        assert write(lib, **{name: NULL}) == E_NULL
        assert write(lib, **{name: P(0x20004)}) == E_ALIGN


def test_rope_refusals(lib):
    assert rope(lib, dtype=-1) == E_DTYPE
    assert rope(lib, tokens=0, qkv=NULL) == E_OK
    for bad in (dict(heads=-1), dict(heads=4097), dict(kv=0), dict(rot=8), dict(rot=-16), dict(rot=144), dict(max_pos=-1),
                dict(max_pos=2**31), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(stride=6136)):
        assert rope(lib, **bad) == E_SHAPE, bad
    for name in ("qkv", "slots", "out", "table", "pos"):
        assert rope(lib, **{name: NULL}) == E_NULL, name
    for name in ("qkv", "wq", "wk", "table", "out"):
        assert rope(lib, **{name: P(0x20008)}) == E_ALIGN, name
    assert rope(lib, pos=P(0x20004)) == E_ALIGN and rope(lib, slots=P(0x20004)) == E_ALIGN


def test_read_refusals(lib):
    assert read(lib, tokens=0, slots=NULL, k=NULL) == E_OK
    assert read(lib, heads=0) == E_SHAPE
    for name in ("slots", "k", "v"):
        assert read(lib, **{name: NULL}) == E_NULL
        assert read(lib, **{name: P(0x20004)}) == E_ALIGN


def test_attention_refusals(lib):
    assert attend(lib, tokens=0, q=NULL) == E_OK
    assert attend(lib, seqs=0, table=NULL) == E_OK
    for bad in (dict(heads=30), dict(heads=4), dict(kv=0), dict(heads=8192, kv=8), dict(seqs=-1), dict(width=-1),
                dict(window=-1), dict(window=5, causal=0), dict(scale=-0.1), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(scale=2.0**127), dict(tokens=2**26, stride=2**13), dict(width=2**27), dict(stride=4095), dict(stride=4088), dict(stride=4100)):
        assert attend(lib, **bad) == E_SHAPE, bad
    for name in ("q", "table", "lens", "offsets", "out"):
        assert attend(lib, **{name: NULL}) == E_NULL, name
    assert attend(lib, q=P(0x10008)) == E_ALIGN and attend(lib, out=P(0x10008)) == E_ALIGN
    for name in ("table", "lens", "offsets", "sinks"):
        assert attend(lib, **{name: P(0x20002)}) == E_ALIGN, name


def test_attention_workspace(lib):
    size = lib.mxfp4_attention_workspace_size
    no = ctypes.c_size_t(-1).value
    assert size(0, 3, 8, 8, 64) == 0 and size(3, 0, 8, 8, 64) == 0
    assert size(1, 1, 9, 8, 64) == no and size(1, 1, 8, 8, 32) == no and size(-1, 1, 8, 8, 64) == no
    assert size(2**22, 2**22, 64, 64, 64) < 1 << 32 and size(2**22 + 1, 1, 64, 64, 64) == no
    assert size(2**16, 2**16, 4096, 1, 128) < 1 << 32 and size(2**16 + 1, 2**16, 4096, 1, 128) == no
    need = size(4, 2, 32, 8, 128)
    assert need < 1 << 32
    if need:
        assert attend(lib, ws_bytes=need - 1) == E_WS
        assert attend(lib, ws=NULL) == E_WS
        assert attend(lib, ws=P(0x1000010)) == E_ALIGN


@pytest.mark.parametrize("group", [1, 2, 3, 16, 17, 32, 33, 64, 65, 100, 4096])
@pytest.mark.parametrize("queries", [1, 1.001, 2, 2.001, 3, 5, 64, 1e6])
def test_attention_launches_fit(lib, group, queries):
    """The most rows a call may have: its grid has fewer than 2^32 threads, the units of the cut form have a size."""
    form = lib.e2m1_mxfp4_attention_form
    form.argtypes = [ctypes.c_int64] * 6
    for kv in (1, 8, 64):
        heads = group * kv
        if heads > 4096:
            continue
        tokens = 2**28 // heads
        seqs = max(1, int(tokens / queries))
        for dim in (64, 128):
            for length in (1, 100, 2**30):
                f = form(tokens, seqs, heads, kv, dim, length)
                kind, nq = f // 100 % 10, f // 10 % 10
                bound = (tokens * group // (16 * nq) + min(seqs, tokens)) * kv
                if kind == 0:
                    tiles = tokens * group // (64 * nq) + min(seqs, tokens)
                    each = max(1, 256 // kv)
                    assert -(-tiles // each) * each * kv * 256 < 2**32
                elif kind == 1:
                    assert bound * 512 < 2**32
                else:
                    assert bound <= 2**29


def test_attention_workspace_holds_every_form(lib):
    """The size does not know how far a table reaches, the form does: it has to do for all of them."""
    form = lib.e2m1_mxfp4_attention_form
    form.argtypes = [ctypes.c_int64] * 6
    seen = set()
    for heads, kv in ((8, 8), (8, 2), (32, 8), (64, 8), (16, 1), (17, 1), (4096, 1)):
        for seqs in (1, 2, 3, 8, 16, 40, 64, 65, 100, 256, 257, 1000, 5000):
            for queries in (1, 2, 4, 5, 8, 12, 16, 30, 64, 300, 2000):
                for tokens in (seqs * queries, seqs * queries - seqs // 2):
                    if tokens * heads > 2**28:
                        continue
                    for dim in (64, 128):
                        size = lib.mxfp4_attention_workspace_size(tokens, seqs, heads, kv, dim)
                        for length in (1, 16, 32, 64, 100, 200, 500, 1000, 1600, 2000, 3000, 5000, 9000, 40000, 2**20, 2**30):
                            f = form(tokens, seqs, heads, kv, dim, length)
                            kind, nq, waves = f // 100 % 10, f // 10 % 10, f % 10
                            seen.add(f)
                            if kind == 2:
                                workers = 8 // waves * 256
                                segments = (tokens * (heads // kv) // (16 * nq) + min(seqs, tokens)) * kv
                                need = 32 * min(segments, workers) + workers * 2 * 16 * nq * (dim + 2) * 4
                                assert size >= need, (tokens, seqs, heads, kv, dim, length, f, size, need)
    assert {10, 20, 30, 111, 114, 118, 211, 1211, 214, 2214, 224, 1224, 2224} <= seen


def test_binding_checks_its_tensors():
    import gemm_e2m1_lut_amd as g
    t = torch.zeros
    cache = tuple(t(2, 2, 16, n, dtype=torch.uint8) for n in (32, 2, 32, 2))
    with pytest.raises(ValueError):
        g.mxfp4_cache_read(cache, t(3, dtype=torch.int64))                 # on the CPU
    with pytest.raises(ValueError):
        g.mxfp4_cache_read(cache[:3], t(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        g.mxfp4_cache_write(t(1, 2, 64), t(1, 2, 64), t(1, dtype=torch.int64), cache)
    with pytest.raises(ValueError):
        g.norm_rope_mxfp4_cache_write(t(1, 384), None, None, t(1, dtype=torch.int64), cache)
    with pytest.raises(ValueError):
        g.mxfp4_attention(t(1, 2, 64, dtype=torch.bfloat16), cache, t(1, 1, dtype=torch.int32), t(1, dtype=torch.int32),
                          t(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        g.mxfp4_attention_workspace_size(1, 1, 9, 8, 64)
