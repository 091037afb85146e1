"""CPU checks of the int8 operators: their plain forms against exact arithmetic, and every refusal.

No call here reaches a kernel launch (each is rejected by validation or is an
empty problem).
"""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import int8_ref as ref
from test_abi import A, B, C, D, E2M1_OK, E_ALIGN, E_DTYPE, E_NULL, E_SHAPE, NULL, P

F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    import gemm_e2m1_lut_amd as g
    return g.load_library()


def test_codes_against_exact_fractions():
    r = np.random.default_rng(1)
    for top in (1.0, 254.0, 127.0, 3.140625, 2.0**-140, 3e38):
        top = float(np.float32(top))
        p = (r.uniform(-1, 1, 300) * top).astype(np.float32)
        halves = (np.arange(-127, 127) + 0.5) / 127.0 * top      # at and next to every border
        h32 = halves.astype(np.float32)
        p = np.concatenate([p, h32, np.nextafter(h32, np.float32(0)), np.nextafter(h32, np.float32(np.inf)),
                            np.float32([top, -top])])
        p = np.clip(p, -top, top).astype(np.float32)
        q, t = ref.codes(p[None, :])
        assert t[0] == top
        assert [ref.code_fraction(float(v), top) for v in p] == q[0].tolist()


def test_codes_of_special_rows():
    p = np.array([[0.0, -0.0, 0.0], [1.0, np.nan, 2.0], [np.inf, 1.0, 2.0], [-3.0, 1.5, 0.0]])
    q, t = ref.codes(p)
    assert q.tolist() == [[0, 0, 0], [0, 0, 0], [0, 0, 0], [-127, 64, 0]]   # 63.5 goes to the even 64
    assert t[0] == 0 and np.isnan(t[1:3]).all() and t[3] == 3


def test_norm_scale_restores_the_norm():
    r = np.random.default_rng(2)
    x, w = r.standard_normal((4, 64)).astype(np.float32), r.standard_normal(64).astype(np.float32)
    q, s, h = ref.rmsnorm(x, w, 1e-5)
    y = x * w / np.sqrt((x.astype(np.float64) ** 2).mean(1, keepdims=True) + 1e-5)
    assert (np.abs(q * s[:, None] - y) <= 0.501 * s[:, None]).all()
    assert np.array_equal(h, x)


# ------------------------------------------------------------- validation --

@pytest.mark.parametrize("name", ["int8_quantize", "silu_mul_int8_quantize"])
def test_row_quantizer_validation(lib, name):
    f = getattr(lib, name)
    assert f(A, 7, B, C, 4, 64, NULL) == E_DTYPE
    assert f(A, F32, B, C, 4, 72, NULL) == E_SHAPE           # k % 16
    assert f(A, F32, B, C, -1, 64, NULL) == E_SHAPE
    assert f(A, F32, B, C, 4, -16, NULL) == E_SHAPE
    assert f(A, F32, B, C, 1, 2**31, NULL) == E_SHAPE
    assert f(A, F32, B, C, 2**60, 64, NULL) == E_SHAPE
    assert f(NULL, BF16, NULL, NULL, 0, 64, NULL) == E2M1_OK
    assert f(NULL, BF16, NULL, NULL, 3, 0, NULL) == E_NULL    # k = 0 still writes the scales
    assert f(NULL, BF16, NULL, P(0x30002), 3, 0, NULL) == E_ALIGN
    assert f(NULL, BF16, B, C, 4, 64, NULL) == E_NULL
    assert f(A, BF16, NULL, C, 4, 64, NULL) == E_NULL
    assert f(A, BF16, B, NULL, 4, 64, NULL) == E_NULL
    assert f(P(0x10008), BF16, B, C, 4, 64, NULL) == E_ALIGN
    assert f(A, BF16, P(0x20008), C, 4, 64, NULL) == E_ALIGN
    assert f(A, BF16, B, P(0x30002), 4, 64, NULL) == E_ALIGN


def test_silu_width_limit(lib):
    assert lib.silu_mul_int8_quantize(A, F32, B, C, 1, 2**30, NULL) == E_SHAPE


def test_rmsnorm_validation(lib):
    f = lib.rmsnorm_int8_quantize

    def call(x=A, res=B, w=C, dtype=BF16, eps=1e-5, out=D, q=P(0x50000), s=P(0x60000), rows=4, k=64):
        return f(x, res, w, dtype, ctypes.c_float(eps), out, q, s, rows, k, NULL)

    assert call(dtype=2) == E_DTYPE
    assert call(k=40) == E_SHAPE
    assert call(rows=-1) == E_SHAPE
    assert call(eps=-1e-6) == E_SHAPE
    assert call(eps=float("nan")) == E_SHAPE
    assert call(eps=float("inf")) == E_SHAPE
    assert call(rows=0, x=NULL, res=NULL, w=NULL, out=NULL, q=NULL, s=NULL) == E2M1_OK
    assert call(res=NULL) == E_NULL            # residual_out without a residual
    assert call(out=NULL) == E_NULL            # and the other way round
    for arg in ("x", "w", "q", "s"):
        assert call(**{arg: NULL}) == E_NULL
    for arg in ("x", "res", "w", "out", "q"):
        assert call(**{arg: P(0x90008)}) == E_ALIGN
    assert call(s=P(0x90002)) == E_ALIGN


def test_int8_gemm_validation(lib):
    f = lib.int8_gemm

    def call(x=A, xs=B, w=C, ws=D, bias=NULL, y=P(0x50000), dtype=BF16, m=4, n=8, k=64):
        return f(x, xs, w, ws, bias, y, dtype, m, n, k, NULL)

    assert call(dtype=3) == E_DTYPE
    assert call(k=72) == E_SHAPE
    assert call(k=131072) == E_SHAPE           # sums could pass 2^31
    assert call(m=-1) == E_SHAPE
    assert call(n=2**31) == E_SHAPE
    assert call(m=2**31) == E_SHAPE
    assert call(m=2**30, n=2**30) == E_SHAPE   # more outputs than any memory holds
    assert call(m=0, x=NULL, xs=NULL, y=NULL) == E2M1_OK
    assert call(n=0, w=NULL, ws=NULL, y=NULL) == E2M1_OK
    for arg in ("x", "xs", "w", "ws", "y"):
        assert call(**{arg: NULL}) == E_NULL
    assert call(x=P(0x10004)) == E_ALIGN
    assert call(w=P(0x30008)) == E_ALIGN
    assert call(y=P(0x50001)) == E_ALIGN
    assert call(y=P(0x50002), dtype=F32) == E_ALIGN
    assert call(xs=P(0x20002)) == E_ALIGN
    assert call(ws=P(0x20002)) == E_ALIGN
    assert call(bias=P(0x20002)) == E_ALIGN


def test_binding_refuses():
    import gemm_e2m1_lut_amd as g
    x = torch.zeros(4, 64)
    i = torch.zeros(4, 64, dtype=torch.int8)
    s = torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        g.int8_quantize(x)
    with pytest.raises(ValueError, match="rows, k"):
        g.int8_quantize(torch.zeros(64))
    with pytest.raises(ValueError, match="GPU"):
        g.rmsnorm_int8_quantize(x, torch.zeros(64), 1e-5)
    with pytest.raises(ValueError, match="GPU"):
        g.silu_mul_int8_quantize(x)
    with pytest.raises(ValueError, match="GPU"):
        g.int8_gemm(i, s, i, s)
    with pytest.raises(ValueError, match="2-dimensional"):
        g.int8_gemm(i[0], s, i, s)


def test_gpu_tests_reach_every_form_of_the_product(lib):
    """The form that the library takes on 256 compute units for each product of test_gpu_int8_forms.py."""
    import test_gpu_int8_forms as t
    variant = lib.e2m1_int8_gemm_variant
    variant.argtypes, variant.restype = [ctypes.c_int64] * 3 + [ctypes.c_int] * 2, ctypes.c_int
    reached = {True: set(), False: set()}
    for form, m, n, k, *at in t.WHOLE_LINES + t.INSIDE_LINES:
        whole = k % 128 == 0 and not any(at)
        assert variant(m, n, k, whole, 256) == form, (m, n, k, at)
        reached[whole].add(form)
        assert n % 4 == 0
    assert reached[True] == reached[False] == set(range(t.LARGEST_HALVED + 1))
    for form, m, n, k in t.LONGEST:
        assert variant(m, n, k, k % 128 == 0, 256) == form, (m, n, k)
