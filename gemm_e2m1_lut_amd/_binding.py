"""ctypes binding of libe2m1lut.so (declared in include/e2m1lut.h).

Argument marshalling only: each function checks the torch tensors it is
given (device, dtype, shape, contiguity), allocates the output with torch when
none is passed, and calls the C entry point of the same name with raw device
pointers and the current HIP stream. Every step of the computation runs in the
library's kernels. A missing library raises at load time; there is no
fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libe2m1lut.so")

ABI_VERSION = 2
DTYPE_F32 = 0
DTYPE_BF16 = 1
GEMV_MAX_BATCH = 16
TERNARY_MAX_BATCH = 16

_lib = None


class E2M1Error(RuntimeError):
    """A library call returned a negative status."""

    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn} failed with status {status}: {message}")
        self.status = status


def library_path() -> str:
    return LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load the in-tree libe2m1lut.so (build it with `python -m gemm_e2m1_lut_amd.build`)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m gemm_e2m1_lut_amd.build` "
                          "(or __graft_entry__.build())")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    sigs = {
        "e2m1_abi_version": (ctypes.c_int, []),
        "e2m1_strerror": (ctypes.c_char_p, [ctypes.c_int]),
        "dequant_decode": (ctypes.c_int, [vp, vp, vp, i64, i64, vp]),
        "dequant_gemv": (ctypes.c_int, [vp, vp, vp, vp, i32, i64, i64, i64, vp]),
        "dequant_gemm": (ctypes.c_int, [vp, vp, vp, vp, i32, i64, i64, i64, vp]),
        "dequant_gemv_grouped": (ctypes.c_int, [i32, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp),
                                                ctypes.POINTER(vp), ctypes.POINTER(i64), ctypes.POINTER(i64),
                                                i32, vp]),
        "nm_spmm": (ctypes.c_int, [vp, vp, vp, vp, i32, i64, i64, i64, i32, i32, vp]),
        "mxfp4_quantize": (ctypes.c_int, [vp, vp, vp, i64, i64, vp]),
        "nvfp4_quantize": (ctypes.c_int, [vp, vp, vp, vp, i64, i64, vp]),
        "int8_quantize": (ctypes.c_int, [vp, i32, vp, vp, i64, i64, vp]),
        "rmsnorm_int8_quantize": (ctypes.c_int, [vp, vp, vp, i32, ctypes.c_float, vp, vp, vp, i64, i64, vp]),
        "silu_mul_int8_quantize": (ctypes.c_int, [vp, i32, vp, vp, i64, i64, vp]),
        "int8_gemm": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, i32, i64, i64, i64, vp]),
        "mxfp4_cache_write": (ctypes.c_int, [vp, vp, i32, i64, i64, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, vp, vp]),
        "norm_rope_mxfp4_cache_write": (ctypes.c_int, [vp, i32, i64, vp, vp, ctypes.c_float, vp, i64, i64, i32, vp, vp,
                                                       vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, vp, vp]),
        "mxfp4_cache_read": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, vp, vp]),
        "mxfp4_attention_workspace_size": (sz, [i64, i64, i64, i64, i64]),
        "mxfp4_attention": (ctypes.c_int, [vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, i32, i64, vp, vp, sz,
                                           i64, i64, i64, i64, i64, i64, i64, i64, vp, vp]),
        "ternary_gemv": (ctypes.c_int, [vp, vp, vp, vp, i64, i64, vp]),
        "ternary_gemm_workspace_size": (sz, [i64, i64, i64]),
        "ternary_gemm": (ctypes.c_int, [vp, vp, vp, vp, vp, sz, i64, i64, i64, vp]),
        "ternary_wl_gemv": (ctypes.c_int, [ctypes.POINTER(vp), vp, vp, vp, vp, vp, i64, i64, vp]),
        "nvfp4_embedding_gather": (ctypes.c_int, [vp, vp, vp, vp, vp, i64, i64, i64, vp, vp]),
        "mxfp4_moe_workspace_size": (sz, [i64, i64, i64, i64, i64]),
        "mxfp4_moe_gemm": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i64, i64, i64, i64,
                                          i64, vp]),
        "mxfp4_moe_gemm_noalloc": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64,
                                                  vp]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    version = lib.e2m1_abi_version()
    if version != ABI_VERSION:
        raise ImportError(f"{LIB_PATH} has ABI version {version}, binding expects {ABI_VERSION}")
    _lib = lib
    return lib


def abi_version() -> int:
    return int(load_library().e2m1_abi_version())


def strerror(status: int) -> str:
    return load_library().e2m1_strerror(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise E2M1Error(fn, status, strerror(status))


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return ctypes.c_void_p(handle)


def _ptr(t: torch.Tensor | None) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t: torch.Tensor, name: str, dtypes, shape=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


_U8 = (torch.uint8,)
_SCALE8 = (torch.uint8, torch.float8_e4m3fn)


# ----------------------------------------------------------------- decode --

def dequant_decode(packed: torch.Tensor, scales: torch.Tensor, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """MXFP4 packed uint8 [rows, k/2] + E8M0 uint8 [rows, k/32] -> bf16 [rows, k]."""
    _need(packed, "packed", _U8)
    rows, half = packed.shape
    k = 2 * half
    _need(scales, "scales", _U8, (rows, k // 32))
    if out is None:
        out = torch.empty((rows, k), dtype=torch.bfloat16, device=packed.device)
    _need(out, "out", (torch.bfloat16, torch.int16), (rows, k))
    _check("dequant_decode", load_library().dequant_decode(_ptr(packed), _ptr(scales), _ptr(out),
                                                            rows, k, _stream(stream)))
    return out


# ------------------------------------------------------------------- GEMV --

def dequant_gemv(packed: torch.Tensor, scales: torch.Tensor, x: torch.Tensor,
                 out_dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """y[b, n] = sum_k W[n, k] x[b, k]: W MXFP4 [n, k/2] + [n, k/32], x bf16 [batch, k] (or [k])."""
    _need(packed, "packed", _U8)
    n, half = packed.shape
    k = 2 * half
    _need(scales, "scales", _U8, (n, k // 32))
    squeeze = x.dim() == 1
    xb = x.unsqueeze(0) if squeeze else x
    _need(xb, "x", (torch.bfloat16,))
    batch = xb.shape[0]
    if xb.shape[1] != k:
        raise ValueError(f"x has {xb.shape[1]} columns, W has {k}")
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    if out is None:
        out = torch.empty((batch, n), dtype=out_dtype, device=packed.device)
    _need(out, "out", (out_dtype,), (batch, n))
    code = DTYPE_F32 if out_dtype == torch.float32 else DTYPE_BF16
    _check("dequant_gemv", load_library().dequant_gemv(_ptr(packed), _ptr(scales), _ptr(xb), _ptr(out),
                                                        code, batch, n, k, _stream(stream)))
    return out[0] if squeeze else out


def dequant_gemv_grouped(mats, out_dtype: torch.dtype = torch.float32, outs=None, stream=None) -> list:
    """[y_g = W_g x_g for (packed_g, scales_g, x_g) in mats]: independent batch-1 products in shared launches.
    x_g is bf16 [k_g] (or [1, k_g]); y_g comes back with x_g's leading shape."""
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    mats = list(mats)
    if outs is not None and len(outs) != len(mats):
        raise ValueError(f"{len(outs)} outputs for {len(mats)} matrices")
    res, xs, ns, ks = [], [], [], []
    for g, (packed, scales, x) in enumerate(mats):
        _need(packed, "packed", _U8)
        n, half = packed.shape
        k = 2 * half
        _need(scales, "scales", _U8, (n, k // 32))
        squeeze = x.dim() == 1
        xb = x.unsqueeze(0) if squeeze else x
        _need(xb, "x", (torch.bfloat16,), (1, k))
        out = torch.empty((1, n), dtype=out_dtype, device=packed.device) if outs is None else outs[g]
        _need(out, "out", (out_dtype,), (1, n) if out.dim() == 2 else (n,))
        res.append(out[0] if (squeeze and out.dim() == 2) else out)
        xs.append(xb)
        ns.append(n)
        ks.append(k)
    cnt = len(mats)
    arr = ctypes.c_void_p * max(cnt, 1)
    a64 = ctypes.c_int64 * max(cnt, 1)
    code = DTYPE_F32 if out_dtype == torch.float32 else DTYPE_BF16
    _check("dequant_gemv_grouped", load_library().dequant_gemv_grouped(
        cnt, arr(*[m[0].data_ptr() for m in mats]), arr(*[m[1].data_ptr() for m in mats]),
        arr(*[x.data_ptr() for x in xs]), arr(*[o.data_ptr() for o in res]), a64(*ns), a64(*ks), code,
        _stream(stream)))
    return res


def dequant_gemm(packed: torch.Tensor, scales: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None,
                 out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """MXFP4 W [n, k/2] + E8M0 [n, k/32], bf16 x [m, k] -> y [m, n] (fp32 accumulate), any m."""
    _need(packed, "packed", _U8)
    n, half = packed.shape
    k = 2 * half
    _need(scales, "scales", _U8, (n, k // 32))
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a [m, k] tensor")
    m = x.shape[0]
    _need(x, "x", (torch.bfloat16, torch.int16), (m, k))
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=packed.device)
    _need(out, "out", (torch.float32, torch.bfloat16), (m, n))
    code = DTYPE_F32 if out.dtype == torch.float32 else DTYPE_BF16
    _check("dequant_gemm", load_library().dequant_gemm(_ptr(packed), _ptr(scales), _ptr(x), _ptr(out), code,
                                                        m, n, k, _stream(stream)))
    return out


def nm_spmm(values: torch.Tensor, meta: torch.Tensor, x: torch.Tensor, n_keep: int, m_group: int,
            out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """N:M sparse W (values bf16 [rows, (k/M) N], packed positions int32/uint32 [rows, words]) times
    bf16 x [batch, k] -> y [batch, rows]."""
    _need(values, "values", (torch.bfloat16, torch.int16))
    _need(meta, "meta", (torch.int32, torch.uint32))
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a [batch, k] tensor")
    batch, k = x.shape
    _need(x, "x", (torch.bfloat16, torch.int16))
    rows = values.shape[0]
    if m_group < 1 or k % m_group != 0 or values.shape[1] != (k // m_group) * n_keep:
        raise ValueError("values must hold (k / m_group) * n_keep entries per row")
    bits = 1 if m_group <= 2 else (m_group - 1).bit_length()
    words = -(-values.shape[1] // (32 // bits))
    _need(meta, "meta", (torch.int32, torch.uint32), (rows, words))
    if out is None:
        out = torch.empty((batch, rows), dtype=out_dtype, device=values.device)
    _need(out, "out", (torch.float32, torch.bfloat16), (batch, rows))
    code = DTYPE_F32 if out.dtype == torch.float32 else DTYPE_BF16
    _check("nm_spmm", load_library().nm_spmm(_ptr(values), _ptr(meta), _ptr(x), _ptr(out), code, batch, rows, k,
                                              n_keep, m_group, _stream(stream)))
    return out


# -------------------------------------------------------------- quantize --

def _bf16_rows(x: torch.Tensor, name: str):
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"{name} must be a [rows, k] tensor")
    _need(x, name, (torch.bfloat16, torch.int16, torch.uint16))
    return x.shape


def mxfp4_quantize(x: torch.Tensor, out: tuple[torch.Tensor, torch.Tensor] | None = None,
                   stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """bf16 [rows, k] -> (codes uint8 [rows, k/2], E8M0 uint8 [rows, k/32])."""
    rows, k = _bf16_rows(x, "x")
    if out is None:
        out = (torch.empty((rows, k // 2), dtype=torch.uint8, device=x.device),
               torch.empty((rows, k // 32), dtype=torch.uint8, device=x.device))
    _need(out[0], "out[0]", _U8, (rows, k // 2))
    _need(out[1], "out[1]", _U8, (rows, k // 32))
    _check("mxfp4_quantize", load_library().mxfp4_quantize(_ptr(x), _ptr(out[0]), _ptr(out[1]), rows, k,
                                                            _stream(stream)))
    return out


def nvfp4_quantize(x: torch.Tensor, global_scale: torch.Tensor,
                   out: tuple[torch.Tensor, torch.Tensor] | None = None,
                   stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """bf16 [rows, k], fp32 global scale [1] -> (codes uint8 [rows, k/2], E4M3 bytes uint8 [rows, k/16])."""
    rows, k = _bf16_rows(x, "x")
    _need(global_scale, "global_scale", (torch.float32,))
    if global_scale.numel() != 1:
        raise ValueError("global_scale must hold one value")
    if out is None:
        out = (torch.empty((rows, k // 2), dtype=torch.uint8, device=x.device),
               torch.empty((rows, k // 16), dtype=torch.uint8, device=x.device))
    _need(out[0], "out[0]", _U8, (rows, k // 2))
    _need(out[1], "out[1]", _SCALE8, (rows, k // 16))
    _check("nvfp4_quantize", load_library().nvfp4_quantize(_ptr(x), _ptr(global_scale), _ptr(out[0]),
                                                            _ptr(out[1]), rows, k, _stream(stream)))
    return out


# ------------------------------------------------------------------- int8 --
# Called for every layer of every token, so one test accepts a good tensor and
# only a bad one goes through the checks that say what is wrong.

_FLOAT_CODE = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
INT8_MAX_K = 131056


def _need_on(t, name: str, dtype: torch.dtype, shape: tuple, device: int) -> int:
    """_need, and on GPU `device`; the tensor's address."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device
            and t.is_contiguous()):
        _need(t, name, (dtype,), shape)
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    return t.data_ptr()


def _float_rows(x, name: str) -> tuple:
    """(rows, columns, dtype code, GPU) of a [rows, k] fp32 or bf16 tensor."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"{name} must be a [rows, k] tensor")
    code = _FLOAT_CODE.get(x.dtype)
    if code is None or not x.is_cuda or not x.is_contiguous():
        _need(x, name, tuple(_FLOAT_CODE))
    rows, k = x.shape
    return rows, k, code, x.get_device()


def _handle_on(stream, device: int) -> int:
    """The handle of the stream a call on GPU `device` runs on."""
    if stream is None:
        # what torch.cuda.current_stream(device).cuda_stream gives, in 0.1 us instead of 1.9
        return torch._C._cuda_getCurrentRawStream(device)
    if not hasattr(stream, "cuda_stream"):
        return int(stream)
    if stream.device.index != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{device}")
    return stream.cuda_stream


def _new(shape: tuple, dtype: torch.dtype, device: int, stream) -> torch.Tensor:
    """An output; for a stream of the caller's it is allocated for that stream, so that its memory is not still in
    use by work queued on another one."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _call_on(device: int, name: str, *args) -> None:
    fn = getattr(_lib or load_library(), name)
    if torch._C._cuda_getDevice() == device:   # torch.cuda.current_device(), without its check for a first call
        status = fn(*args)
    else:   # the launch goes to the tensors' device, whichever is current
        with torch.cuda.device(device):
            status = fn(*args)
    if status != 0:
        _check(name, status)


def _codes_out(out, rows: int, k: int, device: int, stream):
    if out is None:
        out = (_new((rows, k), torch.int8, device, stream), _new((rows,), torch.float32, device, stream))
    q, scale = out
    return (out, _need_on(q, "out[0]", torch.int8, (rows, k), device),
            _need_on(scale, "out[1]", torch.float32, (rows,), device))


def int8_quantize(x: torch.Tensor, out: tuple[torch.Tensor, torch.Tensor] | None = None,
                  stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """bf16 or fp32 [rows, k] -> (codes int8 [rows, k], scale fp32 [rows]); x is about codes * scale."""
    rows, k, code, device = _float_rows(x, "x")
    handle = _handle_on(stream, device)
    out, qp, sp = _codes_out(out, rows, k, device, stream)
    _call_on(device, "int8_quantize", x.data_ptr(), code, qp, sp, rows, k, handle)
    return out


def rmsnorm_int8_quantize(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: torch.Tensor | None = None,
                          residual_out: torch.Tensor | None = None,
                          out: tuple[torch.Tensor, torch.Tensor] | None = None, stream=None) -> tuple:
    """Codes and scales of rmsnorm(x + residual) * weight: x, residual [rows, k] and weight [k], all bf16 or all fp32.

    Returns (codes int8 [rows, k], scale fp32 [rows]), and with a residual also residual_out = x + residual in the
    input type (allocated when not given; it may be residual itself)."""
    rows, k, code, device = _float_rows(x, "x")
    wp = _need_on(weight, "weight", x.dtype, (k,), device)
    handle = _handle_on(stream, device)
    rp = hp = None
    if residual is not None:
        rp = _need_on(residual, "residual", x.dtype, (rows, k), device)
        if residual_out is None:
            residual_out = _new((rows, k), x.dtype, device, stream)
        hp = _need_on(residual_out, "residual_out", x.dtype, (rows, k), device)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    out, qp, sp = _codes_out(out, rows, k, device, stream)
    _call_on(device, "rmsnorm_int8_quantize", x.data_ptr(), rp, wp, code, eps, hp, qp, sp, rows, k, handle)
    return out if residual is None else (*out, residual_out)


def silu_mul_int8_quantize(gate_up: torch.Tensor, out: tuple[torch.Tensor, torch.Tensor] | None = None,
                           stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """bf16 or fp32 [rows, 2 inter], gate then up -> int8 [rows, inter] and fp32 [rows] of silu(gate) * up."""
    rows, both, code, device = _float_rows(gate_up, "gate_up")
    if both % 2 != 0:
        raise ValueError(f"gate_up has {both} columns, expected gate and up of one width")
    inter = both // 2
    handle = _handle_on(stream, device)
    out, qp, sp = _codes_out(out, rows, inter, device, stream)
    _call_on(device, "silu_mul_int8_quantize", gate_up.data_ptr(), code, qp, sp, rows, inter, handle)
    return out


def int8_gemm(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
              bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
              out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """y[m, n] = (x . w^T) * x_scale[m] * w_scale[n] + bias[n]: x int8 [m, k], w int8 [n, k], scales and bias fp32,
    exact int32 sums, y fp32 or bf16 (the type of `out` where it is given)."""
    for t, name in ((x, "x"), (w, "w")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{name} must be a 2-dimensional tensor")
    m, k = x.shape
    n = w.shape[0]
    if not w.is_cuda:
        raise ValueError(f"w must be on a GPU, got {w.device}")
    device = w.get_device()
    xp = _need_on(x, "x", torch.int8, (m, k), device)
    wp = _need_on(w, "w", torch.int8, (n, k), device)
    xsp = _need_on(x_scale, "x_scale", torch.float32, (m,), device)
    wsp = _need_on(w_scale, "w_scale", torch.float32, (n,), device)
    bp = None if bias is None else _need_on(bias, "bias", torch.float32, (n,), device)
    if out is not None:
        out_dtype = out.dtype
    code = _FLOAT_CODE.get(out_dtype)
    if code is None:
        raise TypeError("the output must be torch.float32 or torch.bfloat16")
    handle = _handle_on(stream, device)
    if out is None:
        out = _new((m, n), out_dtype, device, stream)
    yp = _need_on(out, "out", out_dtype, (m, n), device)
    _call_on(device, "int8_gemm", xp, xsp, wp, wsp, bp, yp, code, m, n, k, handle)
    return out


# -------------------------------------------------------- attention cache --

def _cache_of(cache) -> tuple:
    """(addresses, pages, kv heads, page size, head dim, GPU) of (k_codes, k_scales, v_codes, v_scales)."""
    try:
        k, ks, v, vs = cache
        pages, heads, page, half = shape = k.shape
    except (TypeError, ValueError, AttributeError):
        raise ValueError("cache must hold four tensors (k_codes, k_scales, v_codes, v_scales), codes [pages, kv_heads, "
                         "page_size, head_dim / 2]") from None
    scales = (pages, heads, page, half // 16)
    device = k.get_device()
    u8 = torch.uint8
    if not (device >= 0 and k.dtype is u8 and ks.dtype is u8 and v.dtype is u8 and vs.dtype is u8 and v.shape == shape
            and ks.shape == scales and vs.shape == scales and k.is_contiguous() and ks.is_contiguous()
            and v.is_contiguous() and vs.is_contiguous() and ks.get_device() == device and v.get_device() == device
            and vs.get_device() == device):
        for i, want in ((0, shape), (1, scales), (2, shape), (3, scales)):
            _need(cache[i], f"cache[{i}]", _U8, want)
        raise ValueError("the cache's tensors are on different GPUs")
    return (k.data_ptr(), ks.data_ptr(), v.data_ptr(), vs.data_ptr()), pages, heads, page, 2 * half, device


def _token_rows(t, name: str, dtypes, shape: tuple, device: int) -> int:
    """Checks a tensor of `shape` whose tokens (the first extent) may be further apart than their rows; that distance."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.shape != shape or t.get_device() != device:
        raise ValueError(f"{name} is {tuple(t.shape)} on {t.device}, expected {shape} on cuda:{device}")
    row = 1
    for n in shape[1:]:
        row *= n
    if t.is_contiguous():
        return row
    if len(shape) == 3 and t.stride()[1:] == (shape[2], 1) or len(shape) == 2 and t.stride(1) == 1:
        if shape[0] < 2:
            return row
        if t.stride(0) >= row:
            return t.stride(0)
    raise ValueError(f"{name}: a token's values must be contiguous and the tokens apart, got strides {t.stride()}")


def _err_ptr(err_flag, device: int):
    return None if err_flag is None else _need_on(err_flag, "err_flag", torch.int32, (1,), device)


_FLOATS = (torch.float32, torch.bfloat16)


def mxfp4_cache_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache, err_flag: torch.Tensor | None = None,
                      stream=None):
    """Keys and values, bf16 or fp32 [tokens, kv_heads, head_dim] (slices along the tokens are fine), quantized into
    `cache` at int64 slots [tokens] (negative: left out). Returns the cache.

    cache: (k_codes, k_scales, v_codes, v_scales), uint8 [pages, kv_heads, page_size, head_dim / 2] and [..,
    head_dim / 32]."""
    ptrs, pages, heads, page, dim, device = _cache_of(cache)
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be a [tokens, kv_heads, head_dim] tensor")
    tokens = k.shape[0]
    ks = _token_rows(k, "k", _FLOATS, (tokens, heads, dim), device)
    vs = _token_rows(v, "v", (k.dtype,), (tokens, heads, dim), device)
    sp = _need_on(slots, "slots", torch.int64, (tokens,), device)
    _call_on(device, "mxfp4_cache_write", k.data_ptr(), v.data_ptr(), _FLOAT_CODE[k.dtype], ks, vs, sp, *ptrs, tokens,
             heads, dim, pages, page, _err_ptr(err_flag, device), _handle_on(stream, device))
    return cache


def norm_rope_mxfp4_cache_write(qkv: torch.Tensor, cos_sin: torch.Tensor | None, positions: torch.Tensor | None,
                                slots: torch.Tensor, cache, q_weight: torch.Tensor | None = None,
                                k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                                out: torch.Tensor | None = None, err_flag: torch.Tensor | None = None,
                                stream=None) -> torch.Tensor:
    """Rows of a fused product, bf16 or fp32 [tokens, (heads + 2 kv_heads) * head_dim], q | k | v: each query and key
    head normed (where its weight [head_dim] is given) and rotated, keys and values quantized into `cache` at `slots`.
    Returns the queries, bf16 [tokens, heads, head_dim].

    cos_sin: fp32 [max_pos, rot_dim], cosines then sines; positions int64 [tokens]; both None: no rotation."""
    ptrs, pages, kv_heads, page, dim, device = _cache_of(cache)
    if not isinstance(qkv, torch.Tensor) or qkv.dim() != 2:
        raise ValueError("qkv must be a [tokens, (heads + 2 kv_heads) * head_dim] tensor")
    tokens, width = qkv.shape
    heads = width // dim - 2 * kv_heads if dim else -1
    if heads < 0 or width != (heads + 2 * kv_heads) * dim:
        raise ValueError(f"qkv has {width} columns, expected those of some query heads and {kv_heads} key and value "
                         f"heads of {dim}")
    stride = _token_rows(qkv, "qkv", _FLOATS, (tokens, width), device)
    sp = _need_on(slots, "slots", torch.int64, (tokens,), device)
    wq = None if q_weight is None else _need_on(q_weight, "q_weight", qkv.dtype, (dim,), device)
    wk = None if k_weight is None else _need_on(k_weight, "k_weight", qkv.dtype, (dim,), device)
    if (cos_sin is None) != (positions is None):
        raise ValueError("cos_sin and positions go together")
    cp = pp = None
    max_pos = rot = 0
    if cos_sin is not None:
        if not isinstance(cos_sin, torch.Tensor) or cos_sin.dim() != 2:
            raise ValueError("cos_sin must be a [max_pos, rot_dim] tensor")
        max_pos, rot = cos_sin.shape
        cp = _need_on(cos_sin, "cos_sin", torch.float32, (max_pos, rot), device)
        pp = _need_on(positions, "positions", torch.int64, (tokens,), device)
    handle = _handle_on(stream, device)
    if out is None:
        out = _new((tokens, heads, dim), torch.bfloat16, device, stream)
    op = _need_on(out, "out", torch.bfloat16, (tokens, heads, dim), device)
    _call_on(device, "norm_rope_mxfp4_cache_write", qkv.data_ptr(), _FLOAT_CODE[qkv.dtype], stride, wq, wk, eps, cp,
             max_pos, rot, int(interleaved), pp, sp, op, *ptrs, tokens, heads, kv_heads, dim, pages, page,
             _err_ptr(err_flag, device), handle)
    return out


def mxfp4_cache_read(cache, slots: torch.Tensor, out: tuple[torch.Tensor, torch.Tensor] | None = None,
                     err_flag: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The cache's tokens at int64 slots [tokens] -> (k, v), bf16 [tokens, kv_heads, head_dim]; zeros for a negative
    slot."""
    ptrs, pages, heads, page, dim, device = _cache_of(cache)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a [tokens] tensor")
    tokens = slots.shape[0]
    sp = _need_on(slots, "slots", torch.int64, (tokens,), device)
    handle = _handle_on(stream, device)
    if out is None:
        out = tuple(_new((tokens, heads, dim), torch.bfloat16, device, stream) for _ in range(2))
    k, v = out
    kp = _need_on(k, "out[0]", torch.bfloat16, (tokens, heads, dim), device)
    vp = _need_on(v, "out[1]", torch.bfloat16, (tokens, heads, dim), device)
    _call_on(device, "mxfp4_cache_read", *ptrs, sp, kp, vp, tokens, heads, dim, pages, page, _err_ptr(err_flag, device),
             handle)
    return out


def mxfp4_attention_workspace_size(tokens: int, seqs: int, heads: int, kv_heads: int, head_dim: int) -> int:
    """Bytes mxfp4_attention needs on the current device."""
    size = (_lib or load_library()).mxfp4_attention_workspace_size(tokens, seqs, heads, kv_heads, head_dim)
    if size == _NO_SIZE:
        raise ValueError("invalid attention extents")
    return size


_NO_SIZE = ctypes.c_size_t(-1).value


def mxfp4_attention(q: torch.Tensor, cache, page_table: torch.Tensor, kv_lens: torch.Tensor, q_offsets: torch.Tensor,
                    scale: float | None = None, causal: bool = True, window: int = 0,
                    sinks: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, err_flag: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Attention of packed query rows q, bf16 [tokens, heads, head_dim], over the paged cache -> bf16 of that shape.

    Sequence s: query rows q_offsets[s] .. q_offsets[s + 1] - 1 (int32 [seqs + 1]), the last of its kv_lens[s] (int32
    [seqs]) cached tokens, which are on the pages page_table[s] (int32 [seqs, width]). scale: head_dim ** -0.5 when not
    given; window: keys a query sees, its own included (0: all before it); sinks: fp32 [heads], a logit that takes part
    in the softmax and has no value. `workspace` (uint8, mxfp4_attention_workspace_size bytes) is allocated when not
    given."""
    ptrs, pages, kv_heads, page, dim, device = _cache_of(cache)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a [tokens, heads, head_dim] tensor")
    tokens, heads = q.shape[:2]
    stride = _token_rows(q, "q", (torch.bfloat16,), (tokens, heads, dim), device)
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be a [seqs, width] tensor")
    seqs, width = page_table.shape
    tp = _need_on(page_table, "page_table", torch.int32, (seqs, width), device)
    lp = _need_on(kv_lens, "kv_lens", torch.int32, (seqs,), device)
    fp = _need_on(q_offsets, "q_offsets", torch.int32, (seqs + 1,), device)
    np_ = None if sinks is None else _need_on(sinks, "sinks", torch.float32, (heads,), device)
    handle = _handle_on(stream, device)
    if out is None:
        out = _new((tokens, heads, dim), torch.bfloat16, device, stream)
    op = _need_on(out, "out", torch.bfloat16, (tokens, heads, dim), device)
    if workspace is None:
        with torch.cuda.device(device):
            need = mxfp4_attention_workspace_size(tokens, seqs, heads, kv_heads, dim)
        workspace = _new((need,), torch.uint8, device, stream)
    elif not (isinstance(workspace, torch.Tensor) and workspace.dtype is torch.uint8 and workspace.get_device() == device
              and workspace.is_contiguous()):
        _need(workspace, "workspace", _U8)
        raise ValueError(f"workspace is on {workspace.device}, expected cuda:{device}")
    _call_on(device, "mxfp4_attention", q.data_ptr(), stride, *ptrs, tp, lp, fp, np_,
             dim ** -0.5 if scale is None else scale, int(causal), window, op, workspace.data_ptr(), workspace.numel(),
             tokens, seqs, heads, kv_heads, dim, pages, page, width, _err_ptr(err_flag, device), handle)
    return out


# ---------------------------------------------------------------- ternary --

def ternary_gemv(packed: torch.Tensor, row_scale: torch.Tensor, x: torch.Tensor,
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Ternary W packed int32/uint32 [n, k/16] (16 weights per word), fp32 scale [n], fp32 x [k]."""
    _need(packed, "packed", (torch.int32, torch.uint32))
    n, words = packed.shape
    k = 16 * words
    _need(row_scale, "row_scale", (torch.float32,), (n,))
    _need(x, "x", (torch.float32,), (k,))
    if out is None:
        out = torch.empty((n,), dtype=torch.float32, device=packed.device)
    _need(out, "out", (torch.float32,), (n,))
    _check("ternary_gemv", load_library().ternary_gemv(_ptr(packed), _ptr(row_scale), _ptr(x), _ptr(out),
                                                        n, k, _stream(stream)))
    return out


def ternary_gemm_workspace_size(batch: int, n: int, k: int) -> int:
    size = load_library().ternary_gemm_workspace_size(batch, n, k)
    if size == ctypes.c_size_t(-1).value:
        raise ValueError("invalid ternary GEMM extents")
    return int(size)


def ternary_gemm(packed: torch.Tensor, row_scale: torch.Tensor, x: torch.Tensor,
                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """Ternary W packed int32/uint32 [n, k/16], fp32 scale [n], fp32 x [batch, k] -> y [batch, n].
    `workspace` (uint8, at least ternary_gemm_workspace_size bytes) is allocated when not given."""
    _need(packed, "packed", (torch.int32, torch.uint32))
    n, words = packed.shape
    k = 16 * words
    _need(row_scale, "row_scale", (torch.float32,), (n,))
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a [batch, k] tensor")
    batch = x.shape[0]
    _need(x, "x", (torch.float32,), (batch, k))
    if out is None:
        out = torch.empty((batch, n), dtype=torch.float32, device=packed.device)
    _need(out, "out", (torch.float32,), (batch, n))
    need = ternary_gemm_workspace_size(batch, n, k)
    if workspace is None and need > 0:
        workspace = torch.empty((need,), dtype=torch.uint8, device=packed.device)
    if workspace is not None:
        _need(workspace, "workspace", _U8)
    _check("ternary_gemm", load_library().ternary_gemm(
        _ptr(packed), _ptr(row_scale), _ptr(x), _ptr(out), _ptr(workspace),
        0 if workspace is None else workspace.numel(), batch, n, k, _stream(stream)))
    return out


def ternary_wl_gemv(packed, scale: torch.Tensor, x_re: torch.Tensor, x_im: torch.Tensor,
                    out: tuple[torch.Tensor, torch.Tensor] | None = None,
                    stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Widely-linear complex ternary layer y = U x + W conj(x).

    packed: the four ternary matrices U_re, U_im, W_re, W_im, each int32/uint32
    [n, k/16] (a sequence of four tensors, or one [4, n, k/16] tensor);
    scale: fp32 [4, n] in the same order; x_re, x_im: fp32 [k].
    Returns (y_re, y_im), fp32 [n] each."""
    mats = list(packed.unbind(0)) if isinstance(packed, torch.Tensor) else list(packed)
    if len(mats) != 4:
        raise ValueError("packed must hold four matrices (U_re, U_im, W_re, W_im)")
    for i, m in enumerate(mats):
        _need(m, f"packed[{i}]", (torch.int32, torch.uint32))
    n, words = mats[0].shape
    for i, m in enumerate(mats):
        if tuple(m.shape) != (n, words):
            raise ValueError(f"packed[{i}] has shape {tuple(m.shape)}, expected {(n, words)}")
    k = 16 * words
    _need(scale, "scale", (torch.float32,), (4, n))
    _need(x_re, "x_re", (torch.float32,), (k,))
    _need(x_im, "x_im", (torch.float32,), (k,))
    if out is None:
        out = (torch.empty((n,), dtype=torch.float32, device=x_re.device),
               torch.empty((n,), dtype=torch.float32, device=x_re.device))
    _need(out[0], "out[0]", (torch.float32,), (n,))
    _need(out[1], "out[1]", (torch.float32,), (n,))
    ptrs = (ctypes.c_void_p * 4)(*[m.data_ptr() for m in mats])
    _check("ternary_wl_gemv", load_library().ternary_wl_gemv(ptrs, _ptr(scale), _ptr(x_re), _ptr(x_im),
                                                              _ptr(out[0]), _ptr(out[1]), n, k,
                                                              _stream(stream)))
    return out


# ----------------------------------------------------------------- gather --

def nvfp4_embedding_gather(table: torch.Tensor, block_scale: torch.Tensor, global_scale: torch.Tensor,
                           ids: torch.Tensor, out: torch.Tensor | None = None,
                           err_flag: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """NVFP4 table uint8 [vocab, hidden/2], E4M3 block scale [vocab, hidden/16], fp32 global
    scale [1] (device), int64 ids of any shape -> bf16 [*ids.shape, hidden]."""
    _need(table, "table", _U8)
    vocab, half = table.shape
    hidden = 2 * half
    _need(block_scale, "block_scale", _SCALE8, (vocab, hidden // 16))
    _need(global_scale, "global_scale", (torch.float32,), (1,))
    _need(ids, "ids", (torch.int64,))
    ntok = ids.numel()
    if out is None:
        out = torch.empty((*ids.shape, hidden), dtype=torch.bfloat16, device=table.device)
    _need(out, "out", (torch.bfloat16, torch.int16), (*ids.shape, hidden))
    if err_flag is not None:
        _need(err_flag, "err_flag", (torch.int32,), (1,))
    _check("nvfp4_embedding_gather",
           load_library().nvfp4_embedding_gather(_ptr(table), _ptr(block_scale), _ptr(global_scale),
                                                 _ptr(ids), _ptr(out), vocab, hidden, ntok,
                                                 _ptr(err_flag), _stream(stream)))
    return out


# -------------------------------------------------------------------- MoE --

def mxfp4_moe_workspace_size(tokens: int, hidden: int, inter: int, experts: int, topk: int) -> int:
    size = load_library().mxfp4_moe_workspace_size(tokens, hidden, inter, experts, topk)
    if size == ctypes.c_size_t(-1).value:
        raise ValueError("invalid MoE extents")
    return int(size)


def mxfp4_moe_gemm(x: torch.Tensor, w13: torch.Tensor, w13_scale: torch.Tensor, w2: torch.Tensor,
                   w2_scale: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """MXFP4 MoE layer: x bf16 [T, H]; w13 [E, 2I, H/2] + [E, 2I, H/32]; w2 [E, H, I/2] +
    [E, H, I/32]; topk_ids int32 [T, K]; topk_weights fp32 [T, K] -> bf16 [T, H]."""
    _need(x, "x", (torch.bfloat16,))
    tokens, hidden = x.shape
    _need(w13, "w13", _U8)
    experts, two_inter, _ = w13.shape
    inter = two_inter // 2
    _need(w13, "w13", _U8, (experts, 2 * inter, hidden // 2))
    _need(w13_scale, "w13_scale", _U8, (experts, 2 * inter, hidden // 32))
    _need(w2, "w2", _U8, (experts, hidden, inter // 2))
    _need(w2_scale, "w2_scale", _U8, (experts, hidden, inter // 32))
    _need(topk_ids, "topk_ids", (torch.int32,))
    topk = topk_ids.shape[1]
    _need(topk_ids, "topk_ids", (torch.int32,), (tokens, topk))
    _need(topk_weights, "topk_weights", (torch.float32,), (tokens, topk))
    if out is None:
        out = torch.empty((tokens, hidden), dtype=torch.bfloat16, device=x.device)
    _need(out, "out", (torch.bfloat16,), (tokens, hidden))
    need = mxfp4_moe_workspace_size(tokens, hidden, inter, experts, topk)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=x.device)
    _need(workspace, "workspace", _U8)
    _check("mxfp4_moe_gemm",
           load_library().mxfp4_moe_gemm(_ptr(x), _ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale),
                                         _ptr(topk_ids), _ptr(topk_weights), _ptr(out), _ptr(workspace),
                                         workspace.numel(), tokens, hidden, inter, experts, topk,
                                         _stream(stream)))
    return out


# Per-GPU workspace of mxfp4_moe_gemm_noalloc inside the library (E2M1_MOE_NOALLOC_WORKSPACE_BYTES).
MOE_NOALLOC_WORKSPACE_BYTES = 32 << 20


def mxfp4_moe_gemm_noalloc(x: torch.Tensor, w13: torch.Tensor, w13_scale: torch.Tensor, w2: torch.Tensor,
                           w2_scale: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                           out: torch.Tensor, stream=None) -> torch.Tensor:
    """mxfp4_moe_gemm with the library's own fixed per-GPU workspace: nothing is allocated,
    so `out` must be given. Calls that overlap on one GPU race (they share that workspace)."""
    _need(x, "x", (torch.bfloat16,))
    tokens, hidden = x.shape
    _need(w13, "w13", _U8)
    experts, two_inter, _ = w13.shape
    inter = two_inter // 2
    _need(w13, "w13", _U8, (experts, 2 * inter, hidden // 2))
    _need(w13_scale, "w13_scale", _U8, (experts, 2 * inter, hidden // 32))
    _need(w2, "w2", _U8, (experts, hidden, inter // 2))
    _need(w2_scale, "w2_scale", _U8, (experts, hidden, inter // 32))
    _need(topk_ids, "topk_ids", (torch.int32,))
    topk = topk_ids.shape[1]
    _need(topk_ids, "topk_ids", (torch.int32,), (tokens, topk))
    _need(topk_weights, "topk_weights", (torch.float32,), (tokens, topk))
    _need(out, "out", (torch.bfloat16,), (tokens, hidden))
    _check("mxfp4_moe_gemm_noalloc",
           load_library().mxfp4_moe_gemm_noalloc(_ptr(x), _ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale),
                                                 _ptr(topk_ids), _ptr(topk_weights), _ptr(out), tokens, hidden,
                                                 inter, experts, topk, _stream(stream)))
    return out
