"""GPU parity of the attention cache's writers and reader against 64-bit plain forms.

Plain writes and reads are exact (codes, scales and values bit for bit). After a
norm and a rotation a value is an fp32 number within DELTA of the formula's, so a
query is within that and half a step of bf16, and a key's code is the code of some
value within it.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import cache_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def new_cache(pages, heads, page, dim, fill=0):
    return tuple(torch.full((pages, heads, page, n), fill, dtype=torch.uint8, device=DEV)
                 for n in (dim // 2, dim // 32, dim // 2, dim // 32))


def rows(r, shape, dtype):
    """Normal rows of many sizes with some zeros, some exact ties (small whole numbers) and a block of zeros."""
    x = r.standard_normal(shape) * np.exp2(r.integers(-30, 30, (*shape[:-1], 1)))
    whole = r.random(shape[:-1]) < 0.3
    x[whole] = np.round(r.standard_normal(shape)[whole] * 8) / 4
    x[r.random(shape) < 0.02] = 0.0
    x.reshape(-1, 32)[::7] = 0.0
    x.reshape(-1, 32)[3::11] *= -0.0
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype])


def at_slots(cache, slots, page):
    """The cache's bytes [tokens, heads, n] at non-negative slots, on the host."""
    out = []
    for t in cache:
        t = t.cpu()
        out.append(t[slots // page, :, slots % page].numpy())
    return out


def untouched(cache, slots, page, fill):
    """Whether every byte outside `slots` still is `fill`."""
    for t in cache:
        t = t.cpu().clone().transpose(1, 2).reshape(-1, t.shape[1], t.shape[3])
        t[slots] = fill
        if not bool((t == fill).all()):
            return False
    return True


SIZES = [(1, 1, 64, 16), (1, 8, 128, 16), (3, 2, 128, 32), (17, 5, 64, 64), (130, 8, 128, 16), (1025, 3, 64, 128),
         (700, 8, 128, 64)]


@pytest.mark.parametrize("tokens,heads,dim,page", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_and_read(gpu, tokens, heads, dim, page, dtype):
    say(f"cache write/read: {tokens} x {heads} x {dim}, page {page}, {dtype}")
    r = np.random.default_rng(tokens + dim)
    k, v = rows(r, (tokens, heads, dim), dtype), rows(r, (tokens, heads, dim), dtype)
    pages = -(-tokens // page) + 2
    slots = torch.from_numpy(r.permutation(pages * page)[:tokens].copy())
    pad = r.random(tokens) < 0.1
    pad[0] = False
    marked = slots.clone()
    marked[torch.from_numpy(pad)] = -1
    cache = new_cache(pages, heads, page, dim, 0x5A)
    assert gpu.mxfp4_cache_write(k.to(DEV), v.to(DEV), marked.to(DEV), cache) is cache
    kept = slots[~torch.from_numpy(pad)]
    got = at_slots(cache, kept, page)
    want_k, want_v = ref.encode(k.float().numpy()[~pad]), ref.encode(v.float().numpy()[~pad])
    for a, b, name in zip(got, (*want_k, *want_v), ("k codes", "k scales", "v codes", "v scales")):
        assert np.array_equal(a, b), name
    assert untouched(cache, kept, page, 0x5A)
    ko, vo = gpu.mxfp4_cache_read(cache, marked.to(DEV))
    for o, w in ((ko, want_k), (vo, want_v)):
        full = np.zeros((tokens, heads, dim))
        full[~pad] = ref.decode(*w)
        assert np.array_equal(o.float().cpu().numpy(), full)
        assert not torch.signbit(o[o == 0]).any()      # both zero codes read as +0


def test_write_from_a_fused_row(gpu):
    """Slices of a fused product as k and v; a repeated read; slots as int64 views."""
    say("cache write: strided rows")
    r = np.random.default_rng(5)
    x = rows(r, (19, 12 * 64), "bf16").to(DEV)
    k, v = x[:, 4 * 64:8 * 64].view(19, 4, 64), x[:, 8 * 64:].view(19, 4, 64)
    assert not k.is_contiguous()
    cache = new_cache(3, 4, 16, 64)
    slots = torch.arange(5, 24, device=DEV)
    gpu.mxfp4_cache_write(k, v, slots, cache)
    back = gpu.mxfp4_cache_read(cache, torch.cat([slots, slots.flip(0), slots[:1].expand(3)]))
    for t, b in ((k, back[0]), (v, back[1])):
        want = ref.decode(*ref.encode(t.float().cpu().numpy()))
        want = np.concatenate([want, want[::-1], want[:1], want[:1], want[:1]])
        assert np.array_equal(b.float().cpu().numpy(), want)
    with pytest.raises(ValueError):
        gpu.mxfp4_cache_write(k.transpose(1, 2).contiguous().transpose(1, 2), v, slots, cache)
    with pytest.raises(ValueError):
        gpu.mxfp4_cache_write(k[:1].expand(19, 4, 64), v, slots, cache)     # tokens on top of each other
    with pytest.raises(TypeError):
        gpu.mxfp4_cache_write(k, v.float(), slots, cache)
    with pytest.raises(ValueError):
        gpu.mxfp4_cache_write(k, v, slots[:18], cache)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_blocks_that_are_not_finite(gpu, dtype):
    say(f"cache: NaN and infinities, {dtype}")
    r = np.random.default_rng(6)
    k, v = rows(r, (40, 2, 128), dtype), rows(r, (40, 2, 128), dtype)
    for i, bad in enumerate((np.nan, np.inf, -np.inf)):
        k[i, 0, 37 + i] = bad
        v[10 + i, 1, 127] = bad
    big = 3.3e38
    k[20, 0, 0], k[21, 0, 0] = big, -big
    k[22] = 0.0
    k[22, 0, 5] = 1e-40       # below the smallest normal number
    cache = new_cache(4, 2, 16, 128)
    slots = torch.arange(7, 47, device=DEV)
    gpu.mxfp4_cache_write(k.to(DEV), v.to(DEV), slots, cache)
    got = at_slots(cache, slots.cpu(), 16)
    want = (*ref.encode(k.float().numpy()), *ref.encode(v.float().numpy()))
    assert all(np.array_equal(a, b) for a, b in zip(got, want))
    ko, vo = (t.float().cpu().numpy() for t in gpu.mxfp4_cache_read(cache, slots))
    assert np.array_equal(ko, ref.decode(*want[:2]), equal_nan=True)
    assert np.array_equal(vo, ref.decode(*want[2:]), equal_nan=True)
    assert np.isnan(ko[0, 0, 32:64]).all() and np.isfinite(ko[0, 0, :32]).all() and np.isfinite(ko[0, 1]).all()


def test_slots_outside_the_cache(gpu):
    """Nothing is written, zeros are read, the flag is set for slots past the end only and never cleared."""
    say("cache: slots outside")
    r = np.random.default_rng(7)
    k = rows(r, (6, 2, 64), "bf16").to(DEV)
    cache = new_cache(2, 2, 16, 64, 0x11)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    slots = torch.tensor([-1, -2**62, 3, -5, 31, -1], device=DEV)
    gpu.mxfp4_cache_write(k, k, slots, cache, err_flag=flag)
    assert flag.item() == 0 and untouched(cache, torch.tensor([3, 31]), 16, 0x11)
    slots = torch.tensor([32, 2**62, 3, -5, 2**40, -1], device=DEV)
    gpu.mxfp4_cache_write(k, k, slots, cache, err_flag=flag)
    assert flag.item() == 1 and untouched(cache, torch.tensor([3, 31]), 16, 0x11)
    flag.zero_()
    a, _ = gpu.mxfp4_cache_read(cache, slots, err_flag=flag)
    assert flag.item() == 1 and not a[[0, 1, 3, 4, 5]].any() and a[2].any()
    gpu.mxfp4_cache_read(cache, slots)          # without a flag
    flag.zero_()
    gpu.mxfp4_cache_read(cache, slots[2:4], err_flag=flag)
    assert flag.item() == 0
    empty = tuple(t[:0] for t in cache)
    assert not gpu.mxfp4_cache_read(empty, slots[2:4])[0].any()
    gpu.mxfp4_cache_write(k, k, slots, empty)
    gpu.mxfp4_cache_write(k[:0], k[:0], slots[:0], cache)


def angles(max_pos, rot, seed):
    r = np.random.default_rng(seed)
    a = r.uniform(-np.pi, np.pi, (max_pos, rot // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def check_rope(gpu, tokens, heads, kv, dim, rot, page, dtype, normed, interleaved, seed, scale=None):
    r = np.random.default_rng(seed)
    x = rows(r, (tokens, heads + 2 * kv, dim), dtype)
    if scale is not None:
        x = (x.float() * scale).to(DT[dtype])
    wq, wk = ((torch.from_numpy(1 + 0.2 * r.standard_normal(dim)).to(DT[dtype]) if normed else None) for _ in range(2))
    eps = 1e-5
    table = angles(50, rot, seed) if rot else None
    pos = torch.from_numpy(r.integers(0, 50, tokens))
    pages = -(-tokens // page) + 1
    slots = torch.from_numpy(r.permutation(pages * page)[:tokens].copy())
    cache = new_cache(pages, kv, page, dim, 0x33)
    on = lambda t: None if t is None else t.to(DEV)   # noqa: E731
    q = gpu.norm_rope_mxfp4_cache_write(on(x.view(tokens, -1)), on(torch.from_numpy(table)) if rot else None,
                                        on(pos) if rot else None, on(slots), cache, q_weight=on(wq), k_weight=on(wk),
                                        eps=eps, interleaved=interleaved)
    assert q.dtype == torch.bfloat16 and q.shape == (tokens, heads, dim)
    xv = x.float().numpy().astype(np.float64)
    cos, sin = np.split(table[pos.numpy()], 2, axis=1) if rot else (np.zeros((tokens, 0)),) * 2
    made = []
    for part, w in ((xv[:, :heads], wq), (xv[:, heads:heads + kv], wk)):
        y, size = ref.rotate(ref.norm(part, None if w is None else w.float().numpy(), eps), cos, sin, interleaved)
        # a sum of d squares in a tree (8 in a row, then 4 levels), 1/D, + eps, root, reciprocal (2 steps each), two
        # products, then a product and an fma of the rotation: 12 + 1 + 1 + 2 + 2 + 2 + 2 roundings
        made.append((y, 24 * ref.U_F32 * size))
    y, delta = made[0]
    got = q.float().cpu().numpy().astype(np.float64)
    assert (np.abs(got - y) <= ref.U_BF16 * (np.abs(y) + delta) + delta + 2.0**-134).all()
    codes, scales, vcodes, vscales = at_slots(cache, slots, page)
    want_v = ref.encode(xv[:, heads + kv:])
    assert np.array_equal(vcodes, want_v[0]) and np.array_equal(vscales, want_v[1])
    y, delta = made[1]
    amax = np.abs(y).reshape(tokens, kv, -1, 32).max(-1)
    wide = delta.reshape(tokens, kv, -1, 32).max(-1) + 2.0**-149
    assert ((scales >= ref.exponent(np.maximum(amax - wide, 0))) & (scales <= ref.exponent(amax + wide))).all()
    unit = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, -1)
    got = ref.decode(codes, scales)
    lo, hi = y - delta - 2.0**-149, y + delta + 2.0**-149
    side = lambda z: np.sign(z) * ref.MAGS[ref.nearest(np.abs(z) / unit)] * unit   # noqa: E731
    assert ((got >= side(lo)) & (got <= side(hi))).all()
    assert untouched(cache, slots, page, 0x33)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,heads,kv,dim,rot,page,normed", [
    (1, 32, 8, 128, 128, 16, True), (1, 1, 1, 64, 64, 16, False), (15, 6, 2, 64, 32, 32, True), (16, 3, 3, 128, 64, 16, True),
    (17, 5, 1, 128, 16, 64, False), (33, 0, 2, 64, 48, 16, True), (600, 8, 2, 64, 64, 16, False), (2050, 32, 8, 128, 128, 64, True),
    (40, 8, 8, 128, 96, 16, False), (9, 4, 2, 128, 0, 16, True), (9, 4, 2, 64, 0, 16, False)])
def test_norm_rope(gpu, tokens, heads, kv, dim, rot, page, normed, dtype, interleaved):
    say(f"norm rope write: {tokens} x ({heads} + 2 x {kv}) x {dim}, rot {rot}, {dtype}, norm {normed}, {interleaved}")
    check_rope(gpu, tokens, heads, kv, dim, rot, page, dtype, normed, interleaved, tokens + dim + rot)


@pytest.mark.parametrize("scale", [2.0**-100, 2.0**62, 2.0**90])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_very_large_and_small_rows(gpu, dtype, scale):
    """Squares past the fp32 range on either side."""
    say(f"norm rope write: rows times {scale:.3g}, {dtype}")
    check_rope(gpu, 50, 4, 2, 128, 128, 16, dtype, True, False, 3, scale)
    check_rope(gpu, 50, 4, 2, 64, 64, 16, dtype, True, False, 4, scale)


def test_norm_of_zeros_and_one_weight(gpu):
    """A head of zeros stays zeros with eps 0; a norm for the queries only."""
    say("norm rope write: zeros")
    x = torch.zeros(2, 4 * 64, device=DEV)
    x[1, :64] = 3.0
    x[:, 128:192] = 2.0
    w = torch.full((64,), 2.0, device=DEV)
    cache = new_cache(1, 1, 16, 64)
    q = gpu.norm_rope_mxfp4_cache_write(x, None, None, torch.arange(2, device=DEV), cache, q_weight=w, eps=0.0)
    assert not q[0].any() and not q[1, 1].any() and (q[1, 0] == 2).all()
    k, v = gpu.mxfp4_cache_read(cache, torch.arange(2, device=DEV))
    assert (k == 2).all() and not v.any()
    q = gpu.norm_rope_mxfp4_cache_write(x, None, None, torch.arange(2, device=DEV), cache, k_weight=w, eps=0.0)
    k, v = gpu.mxfp4_cache_read(cache, torch.arange(2, device=DEV))
    assert (q[1, 0] == 3).all() and (k == 2).all() and not v.any()


def test_positions_outside_the_table(gpu):
    say("norm rope write: positions outside")
    r = np.random.default_rng(8)
    x = rows(r, (6, 4 * 64), "bf16").to(DEV)
    table = torch.from_numpy(angles(10, 64, 1)).to(DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    cache = new_cache(1, 1, 16, 64, 0x22)
    slots = torch.tensor([0, -1, 2, -1, 4, 5], device=DEV)
    q = gpu.norm_rope_mxfp4_cache_write(x, table, torch.tensor([0, 10, 9, -3, 5, 1], device=DEV), slots, cache, err_flag=flag)
    assert flag.item() == 0 and not q[[1, 3]].any() and all(q[i].any() for i in (0, 2, 4, 5))
    assert untouched(cache, torch.tensor([0, 2, 4, 5]), 16, 0x22)
    cache = new_cache(1, 1, 16, 64, 0x22)
    q = gpu.norm_rope_mxfp4_cache_write(x, table, torch.tensor([0, 1, 2**40, 3, -1, 10], device=DEV), slots, cache, err_flag=flag)
    assert flag.item() == 1 and not q[[2, 4, 5]].any() and q[1].any() and q[3].any()
    assert untouched(cache, torch.tensor([0]), 16, 0x22)


@pytest.mark.parametrize("interleaved", [False, True])
def test_no_positions_at_all(gpu, interleaved):
    """An angle table of no rows is not read: every position is outside it."""
    say("norm rope write: an empty table")
    r = np.random.default_rng(10)
    x = rows(r, (5, 4 * 64), "bf16").to(DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    cache = new_cache(1, 1, 16, 64, 0x22)
    slots = torch.full((5,), -1, dtype=torch.int64, device=DEV)
    pos = torch.zeros(5, dtype=torch.int64, device=DEV)
    call = lambda: gpu.norm_rope_mxfp4_cache_write(x, torch.empty(0, 64, device=DEV), pos, slots, cache,   # noqa: E731
                                                   interleaved=interleaved, err_flag=flag)
    assert not call().any() and flag.item() == 0
    slots[3] = 7
    assert not call().any() and flag.item() == 1
    assert untouched(cache, torch.tensor([], dtype=torch.int64), 16, 0x22)


def test_streams_graphs_and_rows(gpu):
    """Strided rows, another stream, a graph replayed with poisoned outputs: the eager bits each time."""
    say("norm rope write: graph")
    r = np.random.default_rng(9)
    wide = rows(r, (70, 24 * 128), "bf16").to(DEV)
    x = wide[:, 512:512 + 16 * 128]
    table = torch.from_numpy(angles(90, 128, 1)).to(DEV)
    pos, slots = torch.arange(5, 75, device=DEV), torch.arange(69, -1, -1, device=DEV)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    cache = new_cache(5, 2, 16, 128)
    out = torch.empty(70, 12, 128, dtype=torch.bfloat16, device=DEV)
    back = tuple(torch.empty(70, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def step(stream=None):
        gpu.norm_rope_mxfp4_cache_write(x, table, pos, slots, cache, q_weight=w, k_weight=w, out=out, stream=stream)
        gpu.mxfp4_cache_read(cache, slots, out=back, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (*cache, out, *back)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(4):
        for t in (*cache, out, *back):
            t.view(torch.uint8).fill_(0)
        torch.cuda.synchronize()
        graph.replay() if rep % 2 == 0 else step(side if rep == 1 else side.cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip((*cache, out, *back), want)), rep


@pytest.mark.slow
def test_cache_past_32_bits(gpu):
    """A cache of more than 2^32 code bytes: its first and last slots, and those around 2^31 and 2^32."""
    say("cache: past 32 bits")
    heads, dim, page = 8, 128, 64
    per = heads * page * dim // 2
    pages = (1 << 32) // per + 3
    cache = tuple(torch.empty(pages, heads, page, n, dtype=torch.uint8, device=DEV) for n in (64, 4, 64, 4))
    half = (1 << 31) // per * page
    slots = torch.tensor([0, half - 1, half, half + page, 2 * half - 1, 2 * half, pages * page - 1], device=DEV)
    r = np.random.default_rng(10)
    k, v = rows(r, (7, heads, dim), "f32"), rows(r, (7, heads, dim), "f32")
    gpu.mxfp4_cache_write(k.to(DEV), v.to(DEV), slots, cache)
    for o, t in zip(gpu.mxfp4_cache_read(cache, slots), (k, v)):
        assert np.array_equal(o.float().cpu().numpy(), ref.decode(*ref.encode(t.numpy())))
