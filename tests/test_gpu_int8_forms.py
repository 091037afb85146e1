"""int8_gemm in each of its forms: every tile shape of both tables and the halved last round.

The library chooses a form by the product's sizes and by whether rows start on 128-byte lines. The lists below name
one product for each, and test_int8_ref.py holds them to the library's choice, so that a change of that choice cannot
leave a form untested. Sums of less than 2^24 are fp32 numbers, so with scales of one the fp32 output is the sum;
larger ones round once.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import int8_ref as ref
from gpu_util import DEV, say
from test_gpu_int8 import DT, guarded, random_codes, untouched

pytestmark = pytest.mark.gpu

LARGEST_HALVED = 8   # after the table's eight shapes

# form, m, n, k, bytes by which x and w start past a 128-byte line. k % 128 == 0 and neither displaced: the table for
# whole lines. n is a multiple of four (of eight in some), so only y's address decides how its rows are stored.
WHOLE_LINES = [
    (0, 13, 308, 1024), (1, 17, 2052, 256), (2, 19, 4100, 256), (3, 39, 8196, 256), (4, 65, 8196, 256),
    (5, 130, 12292, 256), (6, 4099, 1004, 256), (7, 2305, 5124, 256), (8, 3001, 6148, 1024),
]
INSIDE_LINES = [
    (0, 13, 308, 1040, 0, 0), (1, 17, 2052, 272, 0, 0), (2, 23, 4100, 272, 0, 0), (3, 39, 8196, 272, 0, 0),
    (4, 65, 8196, 272, 0, 0), (5, 130, 8200, 272, 0, 0), (6, 259, 12292, 272, 0, 0), (7, 2049, 4100, 272, 0, 0),
    (8, 2049, 8196, 272, 0, 0),
    # rows of whole lines' length, displaced
    (0, 13, 308, 1024, 16, 112), (1, 17, 2052, 256, 48, 0), (2, 23, 4100, 256, 0, 80), (7, 2049, 4100, 256, 112, 16),
    (8, 2049, 8196, 256, 64, 48),
]
# the longest rows that either table can have
LONGEST = [
    (0, 3, 36, 131056), (1, 259, 300, 131056), (2, 259, 516, 131056), (3, 515, 516, 131056), (4, 1025, 1004, 131056),
    (5, 2049, 1004, 131056), (7, 3001, 4100, 131056), (8, 4099, 5124, 131056),
    (0, 3, 36, 130944), (1, 259, 300, 130944), (2, 259, 516, 130944), (3, 515, 516, 130944), (4, 1025, 1004, 130944),
    (5, 2049, 1004, 130944), (6, 2049, 2052, 130944), (7, 3001, 2884, 130944), (8, 4099, 4100, 130944),
]


def placed(codes: np.ndarray, at: int) -> torch.Tensor:
    """The codes on the GPU, `at` bytes past a 128-byte line, between others that must not count."""
    rows, k = codes.shape
    buf = torch.full((rows * k + 256,), 127, dtype=torch.int8, device=DEV)
    assert buf.data_ptr() % 128 == 0
    t = buf[at:at + rows * k].view(rows, k)
    t.copy_(torch.from_numpy(codes))
    return t


def bits(t: torch.Tensor) -> torch.Tensor:
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("form,m,n,k,at_x,at_w", [(*c, 0, 0) for c in WHOLE_LINES] + INSIDE_LINES)
def test_each_form(gpu, form, m, n, k, at_x, at_w):
    """Exact sums; scaled outputs in both types at every alignment of y; rows with the bits that a small batch has."""
    say(f"int8_gemm: form {form} m={m} n={n} k={k} at {at_x}, {at_w}")
    r = np.random.default_rng(m + n + k + at_x)
    cx, cw = random_codes(r, m, k), random_codes(r, n, k)
    x, w = placed(cx, at_x), placed(cw, at_w)
    y = gpu.int8_gemm(x, torch.ones(m, device=DEV), w, torch.ones(n, device=DEV), out_dtype=torch.float32)
    xs, ws = r.uniform(0.1, 2.0, m).astype(np.float32), r.uniform(0.1, 2.0, n).astype(np.float32)
    b = (r.standard_normal(n) * 100).astype(np.float32)
    sums = cx.astype(np.float64) @ cw.T.astype(np.float64)
    assert np.array_equal(y.cpu().numpy(), sums.astype(np.float32))
    part = np.abs(sums) * xs.astype(np.float64)[:, None] * ws
    want = torch.from_numpy(sums * xs.astype(np.float64)[:, None] * ws + b.astype(np.float64)).to(DEV)
    part = torch.from_numpy(part).to(DEV)
    dev = lambda a: torch.from_numpy(a).to(DEV)   # noqa: E731
    dxs, dws, db = dev(xs), dev(ws), dev(b)
    few = [(0, 1), (2, 13), (m - 11, m)]
    for dtype in ("bf16", "f32"):
        small = [gpu.int8_gemm(x[lo:hi].clone(), dxs[lo:hi].clone(), w, dws, bias=db, out_dtype=DT[dtype]) for lo, hi in few]
        half = torch.finfo(DT[dtype]).eps / 2
        # the sum and its product with x_scale round to fp32: 2^-24 of the product each (and 2^-48); the fma's 2^-24 and
        # the output type's half step are of the value with those errors
        off = (2 * 2.0**-24 + 2.0**-48) * part
        bound = off + (2.0**-24 + half + 2.0**-24 * half) * (want.abs() + off)
        for offset in (0, 1, 2, 4):   # elements past a 16-byte border
            flat, buf = guarded(m * n + offset, DT[dtype])
            y = flat[offset:].view(m, n)
            gpu.int8_gemm(x, dxs, w, dws, bias=db, out=y)
            assert untouched(buf), (dtype, offset)
            assert bool(((y.double() - want).abs() <= bound).all()), (dtype, offset)
            for (lo, hi), s in zip(few, small):
                assert torch.equal(bits(y[lo:hi]), bits(s)), (dtype, offset, lo, hi)


@pytest.mark.parametrize("form,m,n,k", LONGEST)
def test_longest_rows(gpu, form, m, n, k):
    """Sums next to +-2^31 in every output, and random codes in some."""
    say(f"int8_gemm: form {form} m={m} n={n} k={k}")
    ones_m, ones_n = torch.ones(m, device=DEV), torch.ones(n, device=DEV)
    for a, b in ((-128, -128), (-128, 127)):
        x = torch.full((m, k), a, dtype=torch.int8, device=DEV)
        w = torch.full((n, k), b, dtype=torch.int8, device=DEV)
        y = gpu.int8_gemm(x, ones_m, w, ones_n, out_dtype=torch.float32)
        assert bool((y == float(np.float32(a * b * k))).all()), (a, b)
    gen = torch.Generator(device=DEV).manual_seed(m)
    x = torch.randint(-128, 128, (m, k), dtype=torch.int8, device=DEV, generator=gen)
    w = torch.randint(-128, 128, (n, k), dtype=torch.int8, device=DEV, generator=gen)
    y = gpu.int8_gemm(x, ones_m, w, ones_n, out_dtype=torch.float32)
    rows, cols = sorted({0, m // 2, m - 1}), sorted({0, 1, n // 2, n - 2, n - 1})
    want, _ = ref.gemm(x[rows].cpu().numpy(), np.ones(len(rows)), w[cols].cpu().numpy(), np.ones(len(cols)))
    assert np.array_equal(y[rows][:, cols].cpu().numpy(), want.astype(np.float32))
