"""GPU tests of the int8 operators against their plain 64-bit forms (int8_ref.py).

Codes have to be equal: they are defined on the exact quotient. Scales are one
64-bit value rounded to fp32: off by at most 2^-24 of it, and a few 2^-52 of
the 64-bit steps before (the norm's sum of k squares: k 2^-53). int8_gemm takes
the exact sum through at most four fp32 roundings (sum, two scales, bias),
each 2^-24 of a value no larger than |product| + |y|, then rounds to the output
type (half a step: 2^-24 fp32, 2^-8 bf16).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import int8_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GUARD = 64   # elements kept untouched before and after every output


def guarded(n: int, dtype: torch.dtype):
    """(view of n elements, whole buffer): the elements around the view hold a pattern."""
    buf = torch.empty(n + 2 * GUARD, dtype=dtype, device=DEV)
    buf.view(torch.uint8).fill_(0x5A)
    return buf[GUARD:GUARD + n], buf


def untouched(buf: torch.Tensor) -> bool:
    b = buf.view(torch.uint8)
    e = GUARD * buf.element_size()
    return bool((b[:e] == 0x5A).all()) and bool((b[-e:] == 0x5A).all())


def on_gpu(a: np.ndarray, dtype: str) -> tuple[torch.Tensor, np.ndarray]:
    """(device tensor of the type, its values as fp32)."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DT[dtype])
    return t.to(DEV), t.float().numpy()


def codes_out(rows: int, k: int):
    q, qbuf = guarded(rows * k, torch.int8)
    s, sbuf = guarded(rows, torch.float32)
    return (q.view(rows, k), s), (qbuf, sbuf)


def same_scale(got: torch.Tensor, want: np.ndarray, k: int) -> None:
    got = got.cpu().numpy().astype(np.float64)
    with np.errstate(over="ignore"):
        want32 = want.astype(np.float32).astype(np.float64)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    inf = np.isinf(want32) & ~nan
    assert np.array_equal(got[inf], want32[inf])
    ok = ~nan & ~inf
    bound = np.abs(want[ok]) * (2.0**-24 + (k + 16) * 2.0**-53) + 2.0**-150
    assert (np.abs(got[ok] - want[ok]) <= bound).all()


def same_codes(got: torch.Tensor, want: np.ndarray) -> None:
    got = got.cpu().numpy()
    wrong = np.argwhere(got != want)
    assert wrong.size == 0, (len(wrong), wrong[:5].tolist(), got[tuple(wrong[0])], want[tuple(wrong[0])])


def normal_rows(rows: int, k: int, seed: int) -> np.ndarray:
    r = np.random.default_rng(seed)
    return r.standard_normal((rows, k)) * 2.0 ** r.integers(-20, 20, (rows, 1))


# Every row layout: one wave a row, one workgroup of each size with one, two and four units a thread (the last six
# shapes are large enough for more units a thread), the form that reads a row twice; ragged widths in each.
SHAPES = [(1, 16), (3, 48), (1030, 496), (1025, 1008), (1027, 2032), (1024, 2048), (5, 2064), (2, 4096), (9, 2880),
          (3, 4112), (2, 8192), (1100, 4096), (2, 14336), (1, 16384), (2, 16400), (3, 40000), (1, 131072), (6301, 1008), (3100, 2032), (1700, 4080), (800, 8176), (450, 14336),
          (385, 16384)]


def check_quantize(g, a: np.ndarray, dtype: str):
    rows, k = a.shape
    say(f"int8_quantize: rows={rows} k={k} {dtype}")
    x, xv = on_gpu(a, dtype)
    out, bufs = codes_out(rows, k)
    got = g.int8_quantize(x, out=out)
    torch.cuda.synchronize()
    q, s = ref.quantize(xv)
    same_codes(got[0], q)
    same_scale(got[1], s, 0)
    assert all(untouched(b) for b in bufs)


@pytest.mark.parametrize("rows,k", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_shapes(gpu, rows, k, dtype):
    check_quantize(gpu, normal_rows(rows, k, rows + k), dtype)


def border_rows() -> np.ndarray:
    """fp32 rows with elements at and next to every border, for maxima that make exact ties (254 2^e) and others,
    over the whole range of fp32."""
    out = []
    for top in [254.0 * 2.0**e for e in (-140, -60, -7, 0, 30, 110)] + [127.0, 1.0, 3.140625, 2.0**-149, 2.0**-130,
                                                                        1.7e-38, 3.4e38, 1e30, 8e-31, 1.2e30]:
        top = np.float32(top)
        h = ((np.arange(-127, 127) + 0.5) / 127.0 * np.float64(top)).astype(np.float32)
        row = np.concatenate([h, np.nextafter(h, np.float32(0)), np.nextafter(h, np.float32(np.inf)),
                              np.nextafter(h, -np.float32(np.inf)), [top, -top, 0.0, -0.0, 2.0**-149, -2.0**-149]])
        row = np.clip(row, -top, top)
        out.append(np.concatenate([row, np.zeros(-len(row) % 16)]))
    return np.array(out, np.float32)


def test_quantize_borders_f32(gpu):
    check_quantize(gpu, border_rows(), "f32")


@pytest.mark.parametrize("top", [254.0, 127.0, 1.0, 190.0, 2.0**-126, 2.0**126])
def test_quantize_every_bf16_pattern(gpu, top):
    """Every finite bf16 pattern up to `top`, 64 in a row beside it."""
    p = (np.arange(1 << 16, dtype=np.uint32) << 16).view(np.float32)
    p = p[np.isfinite(p) & (np.abs(p) <= top)]
    p = np.concatenate([p, np.zeros(-len(p) % 64, np.float32)]).reshape(-1, 64)
    edge = np.zeros((len(p), 16), np.float32)
    edge[:, 3] = top
    check_quantize(gpu, np.concatenate([p, edge], axis=1), "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [32, 4096, 20000])
def test_quantize_special_rows(gpu, dtype, k):
    a = np.random.default_rng(k).standard_normal((7, k))
    a[0] = 0.0
    a[1, k - 1] = np.nan
    a[2, 0] = np.inf
    a[3, k // 2] = -np.inf
    a[4] = -0.0
    a[5] = 0.0
    a[5, k - 1] = -2.0**-133   # one subnormal
    check_quantize(gpu, a, dtype)


# ------------------------------------------------------------------- norm --

def check_norm(g, a, w, eps, dtype, res=None, in_place=False):
    rows, k = a.shape
    say(f"rmsnorm_int8_quantize: rows={rows} k={k} {dtype} residual={res is not None} in_place={in_place}")
    x, xv = on_gpu(a, dtype)
    wt, wv = on_gpu(w, dtype)
    r, rv, hbuf, h = None, None, None, None
    if res is not None:
        r, rv = on_gpu(res, dtype)
        h, hbuf = guarded(rows * k, DT[dtype])
        h = h.view(rows, k)
        if in_place:
            h.copy_(r)
            r = h
    out, bufs = codes_out(rows, k)
    got = g.rmsnorm_int8_quantize(x, wt, eps, residual=r, residual_out=h, out=out)
    torch.cuda.synchronize()
    q, s, hv = ref.rmsnorm(xv, wv, eps, rv)
    same_codes(got[0], q)
    same_scale(got[1], s, k)
    assert all(untouched(b) for b in bufs)
    if res is None:
        assert len(got) == 2
    else:
        assert got[2].data_ptr() == h.data_ptr() and untouched(hbuf)
        want = torch.from_numpy(hv).to(DT[dtype])
        assert torch.equal(torch.nan_to_num(got[2].cpu(), nan=12345.0), torch.nan_to_num(want, nan=12345.0))


@pytest.mark.parametrize("rows,k", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", ["plain", "residual", "in_place"])
def test_norm_shapes(gpu, rows, k, dtype, mode):
    r = np.random.default_rng(rows * 3 + k)
    w = 1.0 + 0.3 * r.standard_normal(k)
    res = None if mode == "plain" else normal_rows(rows, k, k + 7)
    check_norm(gpu, normal_rows(rows, k, rows + 5 * k), w, 1e-5, dtype, res, mode == "in_place")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1.0])
def test_norm_range(gpu, dtype, eps):
    """Squares past the fp32 range on both sides, zero and non-finite rows, weights of zero and of both signs."""
    r = np.random.default_rng(9)
    k = 4096
    a = r.standard_normal((12, k)) * np.array([1e25, 1e36, 1e-25, 1e-36, 1, 1, 1, 1, 1, 1e-3, 1e3, 1e-42])[:, None]
    a[4] = 0.0
    a[5, 17] = np.nan
    a[6, 4095] = np.inf
    a[7, :] = 0.0
    a[7, 5] = 1e-20
    w = r.standard_normal(k)
    w[5::64] = 0.0
    check_norm(gpu, a, w, eps, dtype)
    res = r.standard_normal((12, k)) * np.abs(a).max(axis=1, keepdims=True).clip(0, 1e36)
    res[np.isnan(res)] = 1.0
    check_norm(gpu, a, w, eps, dtype, res, True)


def test_norm_weight_hides_the_largest(gpu):
    """Weights of zero: rows whose products all vanish have scale 0, whatever h is."""
    w = np.zeros(64)
    check_norm(gpu, normal_rows(3, 64, 1), w, 1e-5, "bf16")
    check_norm(gpu, normal_rows(3, 64, 1), w, 1e-5, "f32", normal_rows(3, 64, 2))


# -------------------------------------------------------------------- act --

def check_act(g, a, dtype):
    rows, k = a.shape[0], a.shape[1] // 2
    say(f"silu_mul_int8_quantize: rows={rows} inter={k} {dtype}")
    x, xv = on_gpu(a, dtype)
    out, bufs = codes_out(rows, k)
    got = g.silu_mul_int8_quantize(x, out=out)
    torch.cuda.synchronize()
    q, s = ref.silu_mul(xv)
    same_codes(got[0], q)
    same_scale(got[1], s, 0)
    assert all(untouched(b) for b in bufs)


@pytest.mark.parametrize("rows,k", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_act_shapes(gpu, rows, k, dtype):
    r = np.random.default_rng(rows + k)
    a = np.concatenate([r.standard_normal((rows, k)) * 2.0 ** r.integers(-4, 4, (rows, 1)),
                        normal_rows(rows, k, rows * 7 + k)], axis=1)
    check_act(gpu, a, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_act_range(gpu, dtype):
    """Gates from -1000 to 1000 with values that bring their products back into range, rows of tiny and of large
    products, equal maxima, zero and non-finite rows."""
    r = np.random.default_rng(3)
    k = 1024
    g = np.stack([r.uniform(-110, 110, k), r.uniform(-100, -60, k), r.uniform(-1000, 1000, k),
                  r.standard_normal(k), r.standard_normal(k) * 1e-20, np.full(k, 3.0), np.zeros(k),
                  r.standard_normal(k), r.standard_normal(k), r.standard_normal(k), r.standard_normal(k) * 1e18,
                  r.uniform(-87.5, -86, k)])
    u = np.stack([r.standard_normal(k), r.standard_normal(k) * 1e37, r.standard_normal(k),
                  r.standard_normal(k) * 1e-18, r.standard_normal(k) * 1e-10, r.choice([-2.0, 2.0], k), r.standard_normal(k),
                  r.standard_normal(k), r.standard_normal(k), r.standard_normal(k), r.standard_normal(k) * 1e18,
                  r.standard_normal(k) * 1e36])
    u[5, :7] = [1.0, 0.5, 1.9921875, -1.0, 0.25, 0.0, 2.0]
    g[7, 3] = np.nan
    u[8, 1000] = np.inf
    g[9, 5] = -np.inf
    check_act(gpu, np.concatenate([g, u], axis=1), dtype)


def test_act_every_bf16_gate(gpu):
    """Every finite bf16 gate of magnitude up to 128, 256 to a row, with up = +-1 beside a largest element."""
    p = (np.arange(1 << 16, dtype=np.uint32) << 16).view(np.float32)
    p = p[np.isfinite(p) & (np.abs(p) <= 128)]
    p = np.sort(p)
    p = np.concatenate([p, np.zeros(-len(p) % 256, np.float32)]).reshape(-1, 256)
    u = np.random.default_rng(4).choice([-1.0, 1.0, 1.5], p.shape)
    check_act(gpu, np.concatenate([p, u], axis=1), "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [512, 4096])
def test_act_moderate_gates(gpu, dtype, k):
    """Units of eight whose gates all lie within 44, units with one beyond, subnormal gates, and `up` near both ends."""
    r = np.random.default_rng(k)
    g = np.stack([r.uniform(-44, 44, k), r.uniform(-44.5, 44.5, k), r.uniform(-44, -43, k), r.uniform(-4, 4, k),
                  r.standard_normal(k) * 1e-39, r.uniform(40, 44, k), r.uniform(-46, -43, k), r.standard_normal(k)])
    u = np.stack([r.standard_normal(k), r.standard_normal(k) * 1e30, r.standard_normal(k) * 1e37,
                  r.standard_normal(k) * 1e-30, r.standard_normal(k) * 1e36, r.standard_normal(k) * 1e36,
                  r.standard_normal(k) * 1e10, r.standard_normal(k) * 1e-16])
    check_act(gpu, np.concatenate([g, u], axis=1), dtype)


def spread_products(r, g: np.ndarray, size: float) -> np.ndarray:
    """up for gates g whose products silu(g) up are spread evenly over -size .. size, so that a row meets every code."""
    return r.uniform(-1, 1, g.shape) * size * (1.0 + np.exp(-g)) / g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lo,hi,size", [(-64, -44, 1.0), (-90, -86, 1e-3), (-110, -44, 1e-12), (-44, -1, 1.0),
                                        (44, 300, 1e3)])
def test_act_spread_products(gpu, dtype, lo, hi, size):
    """Gates far from zero in rows whose products reach every code: 1.3 million codes and 320 row maxima a case."""
    r = np.random.default_rng(int(hi - lo))
    g = r.uniform(lo, hi, (320, 4096))
    check_act(gpu, np.concatenate([g, spread_products(r, g, size)], axis=1), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_act_spread_products_in_mixed_units(gpu, dtype):
    """One gate beyond 44 in every unit of eight, the others' moderate: the evaluation for wide gates on those too."""
    r = np.random.default_rng(8)
    g = r.uniform(-44, 44, (320, 4096))
    g[:, ::8] = r.uniform(-60, -44.5, g[:, ::8].shape)
    check_act(gpu, np.concatenate([g, spread_products(r, g, 1.0)], axis=1), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_act_largest_up(gpu, dtype):
    """`up` at its type's largest value beside very negative gates, those whose -g log2 e lies next to a whole number
    (above it or below) among them: products far inside the fp32 range. Every gate with the largest `up`, a row each."""
    n = np.arange(64, 150, dtype=np.float64)
    at = (n / np.log2(np.e)).astype(np.float32)
    g = -np.concatenate([at + d * np.spacing(at) for d in range(-3, 4)]).astype(np.float64)
    rows = np.tile(g[:, None], (1, 16))
    u = np.full(rows.shape, float(torch.finfo(DT[dtype]).max)) * np.where(np.arange(16) % 3, 1.0, 2.0**-8)
    check_act(gpu, np.concatenate([rows, u * np.random.default_rng(1).choice([-1.0, 1.0], u.shape)], axis=1), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("first", [3.0, 50.0, -50.0])
def test_act_products_near_the_fp32_limit(gpu, dtype, first):
    """Products of 2^127 to 2^128 are finite numbers whatever the other gates of their unit of eight are; a larger one
    counts as infinite."""
    r = np.random.default_rng(5)
    g = r.uniform(1, 2, (6, 64))
    g[:, ::8] = first
    u = r.uniform(-1, 1, (6, 64)) * 1e30
    for row, (gate, up) in enumerate([(4.0, 6e37), (2.0, 1.9e38), (1.5, -2.5e38), (1.25, 3.3e38), (40.0, 8e36)]):
        g[row, 13], u[row, 13] = gate, up
        u[row, 20:] *= 1e6
    check_act(gpu, np.concatenate([g, u], axis=1), dtype)
    for gate, up in ((4.0, 1e38), (2.0, -2e38), (40.0, 9e36)):   # 1.15, 1.04, 1.06 times 2^128
        g[0, 13], u[0, 13] = gate, up
        x, xv = on_gpu(np.concatenate([g, u], axis=1), dtype)
        q, s = gpu.silu_mul_int8_quantize(x)
        wq, ws = ref.silu_mul(xv)
        wq[0], ws[0] = 0, np.nan
        same_codes(q, wq)
        same_scale(s, ws, 0)


# ------------------------------------------------------------------- gemm --

def random_codes(r, rows: int, k: int) -> np.ndarray:
    return r.integers(-128, 128, (rows, k), dtype=np.int8)


def check_gemm(g, x, w, dtype: str, bias=False, seed=0, offset=0):
    """`offset`: elements by which y starts past a 16-byte border."""
    m, k = x.shape
    n = w.shape[0]
    say(f"int8_gemm: m={m} n={n} k={k} {dtype} bias={bias} offset={offset}")
    r = np.random.default_rng(seed)
    xs = (r.uniform(0.1, 2.0, m) * 2.0 ** r.integers(-10, 4, m)).astype(np.float32)
    ws = (r.uniform(0.1, 2.0, n) * 2.0 ** r.integers(-10, 4, n)).astype(np.float32)
    b = (r.standard_normal(n) * 10).astype(np.float32) if bias else None
    flat, buf = guarded(m * n + offset, DT[dtype])
    y = flat[offset:].view(m, n)
    dev = lambda a: torch.from_numpy(a).to(DEV)   # noqa: E731
    got = g.int8_gemm(dev(x), dev(xs), dev(w), dev(ws), bias=None if b is None else dev(b), out=y)
    torch.cuda.synchronize()
    assert got.data_ptr() == y.data_ptr() and untouched(buf)
    got = got.float().cpu().numpy().astype(np.float64)
    want, part = ref.gemm(x, xs, w, ws, b)
    half = torch.finfo(DT[dtype]).eps / 2
    bound = (half + 2.0**-24) * (np.abs(want) + 4 * 2.0**-24 * part) + 3 * 2.0**-24 * part + 1e-37
    assert np.isfinite(got).all()
    off = np.abs(got - want)
    assert (off <= bound).all(), (np.argwhere(off > bound)[:5].tolist(), float((off / bound).max()))


GEMM_SHAPES = [
    (1, 1, 16), (1, 16, 64), (1, 17, 48), (2, 33, 128), (3, 100, 144), (16, 64, 256), (15, 1000, 1008),
    (1, 14336, 4096), (16, 4096, 1024), (7, 130, 16384), (1, 40, 131056), (16, 2880, 2880),
    (17, 31, 80), (31, 97, 528), (33, 64, 512), (64, 256, 1024), (65, 129, 2896), (100, 48, 4112), (128, 128, 128),
    (130, 1003, 1040), (255, 257, 272), (256, 256, 384), (257, 511, 640), (300, 2881, 1536), (513, 770, 2880),
    (1000, 300, 16), (700, 1030, 4096), (4099, 65, 96), (20, 8200, 160),
    # the larger tiles, with rows of y that are aligned and rows that are not; the last two: more of the largest
    # tiles than compute units, the last round's halved
    (700, 2052, 1040), (515, 2881, 2896), (1020, 4092, 1040), (1020, 4091, 528), (1025, 4100, 1040), (1500, 4097, 1040),
    (2047, 8188, 400), (2047, 8191, 400), (4100, 4097, 1040), (4100, 4100, 1040),
    # the same tiles over rows of whole 128-byte lines
    (515, 2881, 1024), (700, 2052, 1152), (1020, 4092, 512), (1020, 4091, 1024), (1025, 4100, 1024), (1500, 4097, 512),
    (2047, 8188, 512), (4100, 4097, 512),
]


@pytest.mark.parametrize("m,n,k", GEMM_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gemm_shapes(gpu, m, n, k, dtype):
    r = np.random.default_rng(m * 7 + n * 3 + k)
    check_gemm(gpu, random_codes(r, m, k), random_codes(r, n, k), dtype, bias=(m + n) % 2 == 1, seed=k)


@pytest.mark.parametrize("m", list(range(1, 36)) + [48, 63, 64, 65, 95, 96, 97, 127, 129])
def test_gemm_every_small_batch(gpu, m):
    r = np.random.default_rng(m)
    check_gemm(gpu, random_codes(r, m, 208), random_codes(r, 83, 208), "f32", bias=True, seed=m)


@pytest.mark.parametrize("m,n", [(3, 37), (70, 67), (300, 264)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [1, 2, 4])
def test_gemm_output_anywhere(gpu, m, n, dtype, offset):
    """y aligned to its elements only."""
    r = np.random.default_rng(m)
    check_gemm(gpu, random_codes(r, m, 160), random_codes(r, n, 160), dtype, bias=True, offset=offset)


@pytest.mark.parametrize("m,n,k", [(1, 50, 256), (40, 200, 512), (300, 2881, 256), (515, 2880, 384), (1020, 4092, 128),
                                   (1025, 4100, 256)])
@pytest.mark.parametrize("at_x,at_w", [(0, 16), (48, 0), (112, 64), (64, 112)])
def test_gemm_operands_inside_lines(gpu, m, n, k, at_x, at_w):
    """x and w that start inside a 128-byte line, between codes that must not count."""
    r = np.random.default_rng(m + at_x + at_w)

    def placed(rows, at):
        buf = torch.full((rows * k + 256,), 127, dtype=torch.int8, device=DEV)
        assert buf.data_ptr() % 128 == 0
        codes = random_codes(r, rows, k)
        t = buf[at:at + rows * k].view(rows, k)
        t.copy_(torch.from_numpy(codes))
        return t, codes.astype(np.int64)

    (x, cx), (w, cw) = placed(m, at_x), placed(n, at_w)
    y = gpu.int8_gemm(x, torch.ones(m, device=DEV), w, torch.ones(n, device=DEV), out_dtype=torch.float32)
    # sums below 2^14 k <= 2^23 are fp32 numbers
    assert np.array_equal(y.cpu().numpy().astype(np.int64), (cx.astype(np.float64) @ cw.T.astype(np.float64)))


@pytest.mark.parametrize("m", [1, 20, 130, 600])
@pytest.mark.parametrize("a,b", [(-128, -128), (-128, 127), (127, 127)])
def test_gemm_largest_sums(gpu, m, a, b):
    """The longest rows accepted, every product at its largest: sums just below 2^31."""
    k = gpu.INT8_MAX_K
    check_gemm(gpu, np.full((m, k), a, np.int8), np.full((20, k), b, np.int8), "f32")


@pytest.mark.parametrize("m,n", [(1, 64), (40, 64), (300, 300)])
def test_gemm_each_column_counts_once(gpu, m, n):
    """x with a single nonzero column per row, w with a distinct pattern per column: any lost, doubled or misplaced
    column of either operand shows."""
    k = 1040
    x = np.zeros((m, k), np.int8)
    x[np.arange(m), (np.arange(m) * 37 + 11) % k] = 1
    w = ((np.arange(n)[:, None] * 31 + np.arange(k)[None, :] * 7) % 255 - 127).astype(np.int8)
    check_gemm(gpu, x, w, "f32")


@pytest.mark.parametrize("n,k", [(300, 1040), (301, 1024), (2881, 400), (4096, 512)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bias", [False, True])
def test_gemm_rows_do_not_depend_on_the_batch(gpu, n, k, dtype, bias):
    """Every form gives the formula's bits: fl32(sum) x_scale, then one fma with w_scale and the bias."""
    r = np.random.default_rng(n)
    x, w = random_codes(r, 1300, k), random_codes(r, n, k)
    xs, ws = r.uniform(-1, 1, 1300).astype(np.float32), r.uniform(-1, 1, n).astype(np.float32)
    b = (r.standard_normal(n) * 100).astype(np.float32) if bias else None
    dev = lambda a: torch.from_numpy(a).to(DEV)   # noqa: E731
    dx, dxs, dw, dws, db = dev(x), dev(xs), dev(w), dev(ws), None if b is None else dev(b)
    whole = gpu.int8_gemm(dx, dxs, dw, dws, bias=db, out_dtype=DT[dtype])
    for lo, hi in ((0, 1), (3, 20), (7, 40), (100, 200), (17, 500), (250, 1299)):
        part = gpu.int8_gemm(dx[lo:hi], dxs[lo:hi].clone(), dw, dws, bias=db, out_dtype=DT[dtype])
        assert torch.equal(part.view(torch.int16 if dtype == "bf16" else torch.int32),
                           whole[lo:hi].view(torch.int16 if dtype == "bf16" else torch.int32)), (lo, hi)
    if dtype == "f32":
        # the fma in 64 bits: its product is exact there, and its sum off by 2^-53 of the larger term before the
        # rounding to 32 bits, which so differs only where that sum lies next to a halfway value
        sums = (x[:64].astype(np.float64) @ w.T.astype(np.float64)).astype(np.float32)
        want = (sums * xs[:64, None]).astype(np.float64) * ws + (0.0 if b is None else b)
        got = whole[:64].cpu().numpy()
        near = np.abs(want.astype(np.float32) - got)
        assert np.all(near <= np.spacing(np.abs(got))) and np.mean(near != 0) < 1e-5


@pytest.mark.parametrize("m", [1, 20, 130])
@pytest.mark.parametrize("low", [0x0000, 0x7FFF, 0x8000, 0x8001])
def test_gemm_rounds_to_the_nearest_bf16(gpu, m, low):
    """Products of zero leave the bias (every upper half, subnormal, infinite and NaN ones too) for the rounding."""
    bits = torch.arange(1 << 16, device="cuda", dtype=torch.int64) << 16 | low
    bias = torch.where(bits < 1 << 31, bits, bits - (1 << 32)).to(torch.int32).view(torch.float32)
    n = bias.numel()
    y = gpu.int8_gemm(torch.zeros(m, 16, dtype=torch.int8, device="cuda"), torch.ones(m, device="cuda"),
                      torch.zeros(n, 16, dtype=torch.int8, device="cuda"), torch.ones(n, device="cuda"), bias=bias)
    want = (bias.cpu() + 0.0).to(torch.bfloat16)
    got = y.cpu()
    nan = torch.isnan(want)
    assert bool((torch.isnan(got) == nan).all())
    assert bool((got.view(torch.int16)[:, ~nan] == want.view(torch.int16)[~nan]).all())


def test_gemm_no_columns(gpu):
    say("int8_gemm: k = 0")
    x, w = torch.empty(3, 0, dtype=torch.int8, device=DEV), torch.empty(5, 0, dtype=torch.int8, device=DEV)
    s3, s5, b = torch.ones(3, device=DEV), torch.ones(5, device=DEV), torch.arange(5.0, device=DEV)
    assert torch.equal(gpu.int8_gemm(x, s3, w, s5, out_dtype=torch.float32).cpu(), torch.zeros(3, 5))
    assert torch.equal(gpu.int8_gemm(x, s3, w, s5, bias=b, out_dtype=torch.float32).cpu(), torch.arange(5.0).expand(3, 5))
    q, s = gpu.int8_quantize(torch.empty(3, 0, device=DEV))
    assert q.shape == (3, 0) and torch.equal(s.cpu(), torch.zeros(3))


def test_empty(gpu):
    say("int8: empty extents")
    q, s = gpu.int8_quantize(torch.empty(0, 64, device=DEV))
    assert q.shape == (0, 64) and s.shape == (0,)
    q, s, h = gpu.rmsnorm_int8_quantize(torch.empty(0, 64, device=DEV), torch.ones(64, device=DEV), 1e-5,
                                        residual=torch.empty(0, 64, device=DEV))
    assert h.shape == (0, 64)
    q, s = gpu.silu_mul_int8_quantize(torch.empty(0, 64, device=DEV))
    assert q.shape == (0, 32)
    i = torch.empty(4, 64, dtype=torch.int8, device=DEV)
    assert gpu.int8_gemm(i[:0], torch.empty(0, device=DEV), i, torch.ones(4, device=DEV)).shape == (0, 4)
    assert gpu.int8_gemm(i, torch.ones(4, device=DEV), i[:0], torch.empty(0, device=DEV)).shape == (4, 0)


def test_gemm_nonfinite_scales(gpu):
    """A token quantized from a NaN has the scale NaN: its outputs are NaN, the others' are untouched by it."""
    say("int8_gemm: NaN scale")
    r = np.random.default_rng(6)
    for m in (3, 200):
        x, w = torch.from_numpy(random_codes(r, m, 64)).to(DEV), torch.from_numpy(random_codes(r, 40, 64)).to(DEV)
        xs = torch.ones(m, device=DEV)
        xs[1] = float("nan")
        y = gpu.int8_gemm(x, xs, w, torch.ones(40, device=DEV)).float().cpu()
        assert torch.isnan(y[1]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[2:]).all()


def test_refusals(gpu):
    say("int8: refusals on the GPU")
    x = torch.zeros(4, 64, device=DEV)
    i = torch.zeros(4, 64, dtype=torch.int8, device=DEV)
    s = torch.zeros(4, device=DEV)
    w = torch.ones(64, device=DEV)
    with pytest.raises(gpu.E2M1Error):
        gpu.int8_quantize(torch.zeros(4, 40, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        gpu.int8_quantize(torch.zeros(64, 32, device=DEV).t())
    with pytest.raises(TypeError):
        gpu.int8_quantize(x.half())
    with pytest.raises(ValueError, match="shape"):
        gpu.int8_quantize(x, out=(i[:2], s))
    with pytest.raises(TypeError):
        gpu.rmsnorm_int8_quantize(x, w.bfloat16(), 1e-5)
    with pytest.raises(ValueError, match="shape"):
        gpu.rmsnorm_int8_quantize(x, w[:32], 1e-5)
    with pytest.raises(ValueError, match="residual"):
        gpu.rmsnorm_int8_quantize(x, w, 1e-5, residual_out=x)
    with pytest.raises(gpu.E2M1Error):
        gpu.rmsnorm_int8_quantize(x, w, -1.0)
    with pytest.raises(ValueError, match="one width"):
        gpu.silu_mul_int8_quantize(torch.zeros(4, 33, device=DEV))
    with pytest.raises(ValueError, match="shape"):
        gpu.int8_gemm(i, s, i[:, :32].contiguous(), s)
    with pytest.raises(ValueError, match="shape"):
        gpu.int8_gemm(i, s[:3], i, s)
    with pytest.raises(TypeError):
        gpu.int8_gemm(i, s, i, s, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="contiguous"):
        gpu.int8_gemm(i, s, i.t().contiguous().t(), s)


# --------------------------------------------------------------- together --

def mlp(g, x, res, norm_w, w13, s13, w2, s2, outs=None, stream=None):
    """A gated MLP in 8 bits: residual and norm, gate and up in one product, silu(gate) * up, down."""
    o = outs or {}
    q, s, h = g.rmsnorm_int8_quantize(x, norm_w, 1e-5, residual=res, residual_out=o.get("h"), out=o.get("qn"), stream=stream)
    gu = g.int8_gemm(q, s, w13, s13, out=o.get("gu"), stream=stream)
    qa, sa = g.silu_mul_int8_quantize(gu, out=o.get("qa"), stream=stream)
    y = g.int8_gemm(qa, sa, w2, s2, out=o.get("y"), stream=stream)
    return q, s, h, gu, qa, sa, y


def mlp_inputs(gpu, tokens, hidden, inter, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *shape: torch.randn(*shape, device=DEV, generator=gen)   # noqa: E731
    w13, s13 = gpu.int8_quantize((rnd(2 * inter, hidden) * 0.05).bfloat16())
    w2, s2 = gpu.int8_quantize((rnd(hidden, inter) * 0.05).bfloat16())
    return rnd(tokens, hidden).bfloat16(), rnd(tokens, hidden).bfloat16(), (1 + 0.1 * rnd(hidden)).bfloat16(), w13, s13, w2, s2


@pytest.mark.parametrize("tokens", [1, 5, 40, 300])
def test_mlp_stage_by_stage(gpu, tokens):
    """Each stage against the plain form of what it was given."""
    say(f"int8 MLP: tokens={tokens}")
    x, res, nw, w13, s13, w2, s2 = mlp_inputs(gpu, tokens, 1024, 1424, tokens)
    q, s, h, gu, qa, sa, y = mlp(gpu, x, res, nw, w13, s13, w2, s2)
    torch.cuda.synchronize()
    f = lambda t: t.float().cpu().numpy()   # noqa: E731
    i = lambda t: t.cpu().numpy()           # noqa: E731
    wq, wsc, wh = ref.rmsnorm(f(x), f(nw), 1e-5, f(res))
    same_codes(q, wq)
    same_scale(s, wsc, 1024)
    assert torch.equal(h.cpu(), torch.from_numpy(wh).bfloat16())
    want, part = ref.gemm(i(q), i(s), i(w13), i(s13))
    assert (np.abs(f(gu) - want) <= (2.0**-8 + 2.0**-22) * part + 1e-37).all()
    wq, wsc = ref.silu_mul(f(gu))
    same_codes(qa, wq)
    same_scale(sa, wsc, 0)
    want, part = ref.gemm(i(qa), i(sa), i(w2), i(s2))
    assert (np.abs(f(y) - want) <= (2.0**-8 + 2.0**-22) * part + 1e-37).all()
    # and the whole against the unquantized layer: int8 rounding is a percent or so of the output's size, not more
    norm = wh.astype(np.float64) / np.sqrt((wh.astype(np.float64) ** 2).mean(1, keepdims=True) + 1e-5) * f(nw)
    gate, up = np.split(norm @ (i(w13) * i(s13)[:, None].astype(np.float64)).T, 2, axis=1)
    full = (gate / (1 + np.exp(-gate)) * up) @ (i(w2) * i(s2)[:, None].astype(np.float64)).T
    assert np.linalg.norm(f(y) - full) <= 0.05 * np.linalg.norm(full)


def test_mlp_graph_replays(gpu):
    """The layer captured into two graphs, replayed in turn with eager work between, against the eager results."""
    say("int8 MLP: graph")
    graphs, outs, eager, args = [], [], [], []
    for tokens, seed in ((3, 1), (150, 2)):
        a = mlp_inputs(gpu, tokens, 512, 768, seed)
        o = {"h": torch.empty(tokens, 512, dtype=torch.bfloat16, device=DEV),
             "qn": (torch.empty(tokens, 512, dtype=torch.int8, device=DEV), torch.empty(tokens, device=DEV)),
             "gu": torch.empty(tokens, 1536, dtype=torch.bfloat16, device=DEV),
             "qa": (torch.empty(tokens, 768, dtype=torch.int8, device=DEV), torch.empty(tokens, device=DEV)),
             "y": torch.empty(tokens, 512, dtype=torch.bfloat16, device=DEV)}
        eager.append([t.clone() for t in mlp(gpu, *a, outs=o)])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mlp(gpu, *a, outs=o)
        graphs.append(graph)
        outs.append(o)
        args.append(a)
    for rep in range(4):
        for o in outs:
            for t in (o["h"], *o["qn"], o["gu"], *o["qa"], o["y"]):
                t.view(torch.uint8).fill_(0xA5)
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for o, want in zip(outs, eager):
            got = [o["qn"][0], o["qn"][1], o["h"], o["gu"], *o["qa"], o["y"]]
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want)), rep
        mlp(gpu, *args[rep % 2], outs=outs[rep % 2])   # eager work between replays


def test_mlp_on_other_streams(gpu):
    """Two streams at once, outputs allocated by the calls, as a torch stream and as a raw handle."""
    say("int8 MLP: streams")
    a, b = mlp_inputs(gpu, 4, 512, 768, 3), mlp_inputs(gpu, 260, 512, 768, 4)
    want = [[t.clone() for t in mlp(gpu, *v)] for v in (a, b)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = [mlp(gpu, *a, stream=s1), mlp(gpu, *b, stream=s2.cuda_stream)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(g, w))


@pytest.mark.slow
def test_rows_past_32_bits(gpu):
    """More than 2^31 elements in every array: the last rows of each operator against the plain form."""
    rows, k = 65537, 32768
    say(f"int8: rows={rows} k={k}")
    x = torch.empty(rows, k, dtype=torch.bfloat16, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(5)
    for r in range(0, rows, 4096):
        x[r:r + 4096] = torch.randn(min(4096, rows - r), k, device=DEV, generator=gen)
    sel = [0, 1, 32767, 32768, rows - 2, rows - 1]
    q, s = gpu.int8_quantize(x)
    xv = x[sel].float().cpu().numpy()
    wq, ws = ref.quantize(xv)
    same_codes(q[sel], wq)
    same_scale(s[sel], ws, 0)
    nw = torch.ones(k, dtype=torch.bfloat16, device=DEV)
    q, s, h = gpu.rmsnorm_int8_quantize(x, nw, 1e-5, residual=x, out=(q, s))
    wq, ws, wh = ref.rmsnorm(xv, nw.float().cpu().numpy(), 1e-5, xv)
    same_codes(q[sel], wq)
    same_scale(s[sel], ws, k)
    assert torch.equal(h[sel].cpu(), torch.from_numpy(wh).bfloat16())
    del h
    qa, sa = gpu.silu_mul_int8_quantize(x)
    wq, ws = ref.silu_mul(xv)
    same_codes(qa[sel], wq)
    same_scale(sa[sel], ws, 0)
    del qa
    # a product with a tall left operand, and with a tall right one (the transposed problem)
    few = torch.from_numpy(np.random.default_rng(1).integers(-128, 128, (24, k), dtype=np.int8)).to(DEV)
    fs = torch.full((24,), 0.01, device=DEV)
    y = gpu.int8_gemm(q, s, few, fs, out_dtype=torch.float32)
    want, part = ref.gemm(q[sel].cpu().numpy(), s[sel].cpu().numpy(), few.cpu().numpy(), fs.cpu().numpy())
    assert (np.abs(y[sel].cpu().numpy() - want) <= 2.0**-22 * part + 1e-37).all()
    yt = gpu.int8_gemm(few, fs, q, s, out_dtype=torch.float32)
    assert (np.abs(yt[:, sel].cpu().numpy().T - want) <= 2.0**-22 * part + 1e-37).all()


@pytest.mark.slow
def test_output_past_32_bits(gpu):
    """y with more than 2^31 elements: every one of the last rows and a sample of the others."""
    m, n, k = 70001, 32000, 16
    say(f"int8_gemm: m={m} n={n} k={k}")
    r = np.random.default_rng(2)
    x, w = random_codes(r, m, k), random_codes(r, n, k)
    xs, ws = r.uniform(0.5, 1, m).astype(np.float32), r.uniform(0.5, 1, n).astype(np.float32)
    dev = lambda a: torch.from_numpy(a).to(DEV)   # noqa: E731
    y = gpu.int8_gemm(dev(x), dev(xs), dev(w), dev(ws))
    sel = np.array([0, 1, 255, 256, 33000, 67107, 67108, 67109, 69999, 70000])
    want, part = ref.gemm(x[sel], xs[sel], w, ws)
    got = y[torch.from_numpy(sel).to(DEV)].float().cpu().numpy()
    assert (np.abs(got - want) <= (2.0**-8 + 2.0**-22) * part + 1e-37).all()
