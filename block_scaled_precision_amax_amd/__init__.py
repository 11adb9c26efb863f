"""Python binding of libfp8q.so: amax-scaled FP8 quantization and the
block-scaled FP8 GEMM for AMD Instinct MI355X (gfx950).

Argument marshalling only.  Each function has the name and the argument
order of its C entry point in include/fp8q.h; pointer arguments take torch
tensors (their data_ptr() is passed) or raw integer addresses, the element
dtype argument of the C call is read from the input tensor, and ``stream``
defaults to torch's current stream on the tensor's device.  Every step of
the computation runs in the library's HIP kernels; there is no fallback.
A non-OK status raises Fp8qError with the library's message.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfp8q.so")

OK, EINVAL, ESHAPE, EALIGN, EHIP, ENOTIMPL = range(6)
F32, BF16 = 0, 1
E4M3FN, E5M2 = 0, 1
GRAN_TENSOR, GRAN_1x128, GRAN_128x128 = 0, 1, 2
ACT_SILU, ACT_GELU, ACT_NONE, ACT_RELU, ACT_GELU_ERF = range(5)
MAX_FINITE = {E4M3FN: 448.0, E5M2: 57344.0}

# every exported symbol declared in include/fp8q.h
SYMBOLS = (
    "fp8q_version",
    "fp8q_status_string",
    "fp8q_last_error",
    "fp8q_amax",
    "fp8q_quantize_tensor",
    "fp8q_quantize_1x128",
    "fp8q_quantize_1x128_t",
    "fp8q_quantize_128x128",
    "fp8q_quantize_mx",
    "fp8q_dequantize_mx",
    "fp8q_delayed_scaler_init",
    "fp8q_delayed_scaler_init_stat",
    "fp8q_delayed_scaler_update",
    "fp8q_dequantize",
    "fp8q_gemm_blockscaled",
    "fp8q_gemm_blockscaled_fast",
    "fp8q_gemm_mx",
    "fp8q_gemm_blockscaled_q",
    "fp8q_quantize_tensor_dq",
    "fp8q_quantize_tensor_delayed",
    "fp8q_gemm_blockscaled_qt",
    "fp8q_rmsnorm_1x128",
    "fp8q_rmsnorm_bwd_workspace",
    "fp8q_rmsnorm_bwd",
    "fp8q_glu_blockscaled",
    "fp8q_glu_blockscaled_fast",
    "fp8q_glu_blockscaled_q",
    "fp8q_glu_blockscaled_q_workspace",
    "fp8q_glu_bwd_q",
    "fp8q_gemm_blockscaled_few",
    "fp8q_layernorm_1x128",
    "fp8q_layernorm_bwd_workspace",
    "fp8q_layernorm_bwd",
    "fp8q_linear_blockscaled",
    "fp8q_linear_blockscaled_fast",
    "fp8q_linear_blockscaled_q",
    "fp8q_linear_blockscaled_q_fast",
    "fp8q_linear_blockscaled_workspace",
    "fp8q_linear_bwd_q_workspace",
    "fp8q_linear_bwd_q",
)


class Fp8qError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"fp8q status {status}: {msg}")
        self.status = status


class Scaler(ctypes.Structure):
    """Host image of fp8q_scaler (for checkpointing a device-resident state)."""

    _fields_ = [("ring", ctypes.c_float * 1024), ("window", ctypes.c_int32), ("count", ctypes.c_int32),
                ("pos", ctypes.c_int32), ("max_val", ctypes.c_float), ("eps", ctypes.c_float),
                ("margin", ctypes.c_float), ("scale", ctypes.c_float), ("stat", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("amax_acc", ctypes.c_float), ("ema", ctypes.c_double)]


STAT_MAX, STAT_MEAN, STAT_EMA = 0, 1, 2


SCALER_BYTES = ctypes.sizeof(Scaler)
SCALER_SCALE_OFFSET = Scaler.scale.offset

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libfp8q.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m block_scaled_precision_amax_amd.build` (hipcc, gfx950)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        sig = {
            "fp8q_version": (i32, []),
            "fp8q_status_string": (ctypes.c_char_p, [i32]),
            "fp8q_last_error": (ctypes.c_char_p, []),
            "fp8q_amax": (i32, [vp, i32, i64, vp, vp]),
            "fp8q_quantize_tensor": (i32, [vp, i32, i64, i32, vp, vp, vp, vp]),
            "fp8q_quantize_1x128": (i32, [vp, i32, i64, i64, i64, i32, f32, vp, i64, vp, i64, vp]),
            "fp8q_quantize_1x128_t": (i32, [vp, i32, i64, i64, i64, i32, f32, vp, i64, vp, i64, vp]),
            "fp8q_quantize_128x128": (i32, [vp, i32, i64, i64, i64, i32, f32, vp, i64, vp, i64, vp]),
            "fp8q_quantize_mx": (i32, [vp, i32, i64, i64, i64, i32, vp, i64, vp, i64, vp]),
            "fp8q_dequantize_mx": (i32, [vp, i32, i64, i64, i64, vp, i64, vp, i32, i64, vp]),
            "fp8q_delayed_scaler_init": (i32, [vp, i32, f32, f32, f32, vp]),
            "fp8q_delayed_scaler_init_stat": (i32, [vp, i32, f32, f32, f32, i32, f32, vp]),
            "fp8q_delayed_scaler_update": (i32, [vp, vp, vp]),
            "fp8q_dequantize": (i32, [vp, i32, i64, i64, i64, vp, i32, i64, vp, i32, i64, vp]),
            "fp8q_gemm_blockscaled": (i32, [vp, i32, i64, vp, i64, i64, vp, i32, i64, vp, i32, i64, i64,
                                            vp, i32, i64, i64, i64, i64, vp]),
            "fp8q_gemm_blockscaled_fast": (i32, [vp, i32, i64, vp, i64, i64, vp, i32, i64, vp, i32, i64, i64,
                                                 vp, i32, i64, i64, i64, i64, vp]),
            "fp8q_gemm_mx": (i32, [vp, i32, i64, vp, i64, vp, i32, i64, vp, i64, vp, i32, i64, i64, i64, i64, vp]),
            "fp8q_quantize_tensor_dq": (i32, [vp, i32, i64, i32, vp, vp, vp, vp, i32, vp]),
            "fp8q_quantize_tensor_delayed": (i32, [vp, i32, i64, i32, vp, vp, vp, i32, vp]),
            "fp8q_gemm_blockscaled_qt": (i32, [vp, i32, i64, vp, i64, i64, vp, i32, i64, vp, i32, i64, i64, i32, f32,
                                               vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, i64, vp]),
            "fp8q_gemm_blockscaled_q": (i32, [vp, i32, i64, vp, i64, i64, vp, i32, i64, vp, i32, i64, i64, i32, f32,
                                              vp, i64, vp, i64, i64, i64, i64, vp]),
            "fp8q_rmsnorm_1x128": (i32, [vp, i32, i64, vp, i64, vp, i32, i64, i64, f32, vp, i64, vp, i64, i32, f32, vp,
                                         i64, vp, i64, vp, vp]),
            "fp8q_rmsnorm_bwd_workspace": (i64, [i64, i64]),
            "fp8q_rmsnorm_bwd": (i32, [vp, i32, i64, vp, i64, vp, i32, vp, vp, i64, i64, i64, vp, i64, vp, vp, i64, vp]),
            "fp8q_glu_blockscaled": (i32, [vp, i32, i64, vp, i64, i64, vp, vp, i32, i64, vp, vp, i64, i64, i32, vp, i32,
                                           i64, vp, i64, i64, i64, i64, vp]),
            "fp8q_glu_blockscaled_fast": (i32, [vp, i32, i64, vp, i64, i64, vp, vp, i32, i64, vp, vp, i64, i64, i32, vp,
                                                i32, i64, vp, i64, i64, i64, i64, vp]),
            "fp8q_glu_blockscaled_q": (i32, [vp, i32, i64, vp, i64, i64, vp, vp, i32, i64, vp, vp, i64, i64, i32, i32,
                                             f32, vp, i64, vp, i64, vp, i64, i64, i64, i64, vp, i64, vp]),
            "fp8q_glu_blockscaled_q_workspace": (i64, [i64, i64]),
            "fp8q_glu_bwd_q": (i32, [vp, i32, i64, vp, i64, i32, i32, f32, vp, i64, vp, i64, vp, i64, vp, i64, i32, vp,
                                     i64, vp, i64, i64, i64, vp]),
            "fp8q_gemm_blockscaled_few": (i32, [vp, i32, i64, vp, i64, i64, vp, i32, i64, vp, i32, i64, i64, vp, i32,
                                                i64, i64, i64, i64, vp]),
            "fp8q_layernorm_1x128": (i32, [vp, i32, i64, vp, i64, vp, vp, i32, i64, i64, f32, vp, i64, vp, i64, i32, f32,
                                           vp, i64, vp, i64, vp, vp, vp]),
            "fp8q_layernorm_bwd_workspace": (i64, [i64, i64]),
            "fp8q_layernorm_bwd": (i32, [vp, i32, i64, vp, i64, vp, i32, vp, vp, vp, i64, i64, i64, vp, i64, vp, vp, vp,
                                         i64, vp]),
            "fp8q_linear_blockscaled_workspace": (i64, [i32, i32, i64, i64, i64]),
            "fp8q_linear_bwd_q_workspace": (i64, [i64, i64]),
            "fp8q_linear_bwd_q": (i32, [vp, i32, i64, vp, i64, i32, i32, f32, vp, i64, vp, i64, vp, i64, vp, i64, i32, vp,
                                        i64, vp, i64, vp, i64, i64, vp, i64, vp]),
            **{f"fp8q_linear_blockscaled{form}": (i32, [vp, i32, i64, vp, i64, i64, vp, i32, i64, vp, i64, i64, vp, i32, i32,
                                                        vp, i64, vp, i32, i64, vp, i64, i64, i64, i64, vp, i64, vp])
               for form in ("", "_fast")},
            **{f"fp8q_linear_blockscaled_q{form}": (i32, [vp, i32, i64, vp, i64, i64, vp, i32, i64, vp, i64, i64, vp, i32,
                                                          i32, i32, f32, vp, i64, vp, i64, vp, i64, i64, i64, i64, vp, i64,
                                                          vp])
               for form in ("", "_fast")},
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


# ---------------------------------------------------------------- marshalling helpers
def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_DTYPES: dict = {}  # torch's dtypes, filled by the first call (torch is imported only then)


def _dt(t) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        import torch

        _DTYPES.update({torch.float32: F32, torch.bfloat16: BF16})
        d = _DTYPES.get(t.dtype)
        if d is None:
            raise TypeError(f"fp8q inputs are float32 or bfloat16, got {t.dtype}")
    return d


# Operands whose element type is fixed: a narrower tensor's end would be passed, another type misread.  Each kind's
# torch dtypes are filled in by the first check.
_FLOAT: list = []
_BFLOAT: list = []
_CODES: list = []


def _refuse(t, kind, name) -> None:
    if not kind:
        import torch

        _FLOAT.append(torch.float32)
        _BFLOAT.extend((torch.bfloat16, torch.int16, torch.uint16))
        _CODES.extend((torch.uint8, torch.int8, torch.float8_e4m3fn, torch.float8_e5m2))
    if t.dtype not in kind:
        raise TypeError(f"this operand is {name}, got {t.dtype}")


def _f32(t) -> int | None:
    if t is None or isinstance(t, int):
        return t
    if t.dtype not in _FLOAT:
        _refuse(t, _FLOAT, "float32")
    return t.data_ptr()


def _bf16(t) -> int | None:
    if t is None or isinstance(t, int):
        return t
    if t.dtype not in _BFLOAT:
        _refuse(t, _BFLOAT, "bfloat16")
    return t.data_ptr()


def _codes(t) -> int | None:
    if t is None or isinstance(t, int):
        return t
    if t.dtype not in _CODES:
        _refuse(t, _CODES, "FP8 codes")
    return t.data_ptr()


_raw_stream = None


def _stream(stream, t=None) -> int | None:
    global _raw_stream
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    if t is not None and not isinstance(t, int) and t.is_cuda:
        # the handle alone: building a Stream object takes longer than a small launch
        if _raw_stream is None:
            import torch

            _raw_stream = torch._C._cuda_getCurrentRawStream
        return _raw_stream(t.get_device())
    import torch

    dev = t.device if (t is not None and not isinstance(t, int)) else None
    return torch.cuda.current_stream(dev).cuda_stream


def _workspace(nbytes, handle, stream, t):
    """Scratch memory on t's device (the current one for a raw pointer) from the pool of the stream that uses it: the
    allocator hands a block out again as soon as its own stream's work is enqueued, so one of another stream's may still
    be in use there."""
    import torch

    dev = torch.device("cuda", torch.cuda.current_device()) if isinstance(t, int) else t.device
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if isinstance(stream, int):  # handle 0 is no external stream to torch
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)


def _check(rc: int) -> None:
    if rc != OK:
        raise Fp8qError(rc, lib().fp8q_last_error().decode(errors="replace"))


# ---------------------------------------------------------------- entry points
def fp8q_version() -> int:
    return lib().fp8q_version()


def fp8q_amax(x, n, amax, stream=None) -> None:
    _check(lib().fp8q_amax(_ptr(x), _dt(x), n, _ptr(amax), _stream(stream, x)))


def fp8q_quantize_tensor(x, n, f, scale, q, amax_out=None, stream=None) -> None:
    _check(lib().fp8q_quantize_tensor(_ptr(x), _dt(x), n, f, _ptr(scale), _ptr(q), _ptr(amax_out),
                                      _stream(stream, x)))


def fp8q_quantize_1x128(x, rows, cols, ldx, f, eps, q, ldq, scales, ld_s, stream=None) -> None:
    _check(lib().fp8q_quantize_1x128(_ptr(x), _dt(x), rows, cols, ldx, f, eps, _ptr(q), ldq, _ptr(scales),
                                     ld_s, _stream(stream, x)))


def fp8q_quantize_1x128_t(x, rows, cols, ldx, f, eps, q, ldq, scales, ld_s, stream=None) -> None:
    _check(lib().fp8q_quantize_1x128_t(_ptr(x), _dt(x), rows, cols, ldx, f, eps, _ptr(q), ldq, _ptr(scales),
                                       ld_s, _stream(stream, x)))


def fp8q_quantize_128x128(x, rows, cols, ldx, f, eps, q, ldq, scales, ld_s, stream=None) -> None:
    _check(lib().fp8q_quantize_128x128(_ptr(x), _dt(x), rows, cols, ldx, f, eps, _ptr(q), ldq,
                                       _ptr(scales), ld_s, _stream(stream, x)))


def fp8q_quantize_mx(x, rows, cols, ldx, f, q, ldq, scales, ld_s, stream=None) -> None:
    _check(lib().fp8q_quantize_mx(_ptr(x), _dt(x), rows, cols, ldx, f, _ptr(q), ldq, _ptr(scales), ld_s,
                                  _stream(stream, x)))


def fp8q_dequantize_mx(q, f, rows, cols, ldq, scales, ld_s, y, ldy, stream=None) -> None:
    _check(lib().fp8q_dequantize_mx(_ptr(q), f, rows, cols, ldq, _ptr(scales), ld_s, _ptr(y), _dt(y), ldy,
                                    _stream(stream, q)))


def fp8q_delayed_scaler_init(state, window, max_val, eps, margin, stream=None) -> None:
    _check(lib().fp8q_delayed_scaler_init(_ptr(state), window, max_val, eps, margin, _stream(stream, state)))


def fp8q_delayed_scaler_init_stat(state, window, max_val, eps, margin, stat, alpha=0.0, stream=None) -> None:
    _check(lib().fp8q_delayed_scaler_init_stat(_ptr(state), window, max_val, eps, margin, stat, alpha,
                                               _stream(stream, state)))


def fp8q_delayed_scaler_update(state, amax=None, stream=None) -> None:
    _check(lib().fp8q_delayed_scaler_update(_ptr(state), _ptr(amax), _stream(stream, state)))


def fp8q_dequantize(q, f, rows, cols, ldq, scales, g, ld_s, y, ldy, stream=None) -> None:
    _check(lib().fp8q_dequantize(_ptr(q), f, rows, cols, ldq, _ptr(scales), g, ld_s, _ptr(y), _dt(y), ldy,
                                 _stream(stream, q)))


def fp8q_gemm_blockscaled(A, fa, lda, sA, sA_sm, sA_skb, B, fb, ldb, sB, gb, sB_sn, sB_skb, C, ldc, M, N,
                          K, stream=None) -> None:
    _check(lib().fp8q_gemm_blockscaled(_ptr(A), fa, lda, _ptr(sA), sA_sm, sA_skb, _ptr(B), fb, ldb, _ptr(sB),
                                       gb, sB_sn, sB_skb, _ptr(C), _dt(C), ldc, M, N, K, _stream(stream, A)))


def fp8q_gemm_blockscaled_fast(A, fa, lda, sA, sA_sm, sA_skb, B, fb, ldb, sB, gb, sB_sn, sB_skb, C, ldc, M, N,
                               K, stream=None) -> None:
    _check(lib().fp8q_gemm_blockscaled_fast(_ptr(A), fa, lda, _ptr(sA), sA_sm, sA_skb, _ptr(B), fb, ldb,
                                            _ptr(sB), gb, sB_sn, sB_skb, _ptr(C), _dt(C), ldc, M, N, K,
                                            _stream(stream, A)))


def fp8q_gemm_mx(A, fa, lda, sA, ld_sa, B, fb, ldb, sB, ld_sb, C, ldc, M, N, K, stream=None) -> None:
    _check(lib().fp8q_gemm_mx(_ptr(A), fa, lda, _ptr(sA), ld_sa, _ptr(B), fb, ldb, _ptr(sB), ld_sb, _ptr(C), _dt(C),
                              ldc, M, N, K, _stream(stream, A)))


def fp8q_gemm_blockscaled_q(A, fa, lda, sA, sA_sm, sA_skb, B, fb, ldb, sB, gb, sB_sn, sB_skb, fc, eps, Cq, ldcq, Cs,
                            ld_cs, M, N, K, stream=None) -> None:
    _check(lib().fp8q_gemm_blockscaled_q(_ptr(A), fa, lda, _ptr(sA), sA_sm, sA_skb, _ptr(B), fb, ldb, _ptr(sB), gb,
                                         sB_sn, sB_skb, fc, eps, _ptr(Cq), ldcq, _ptr(Cs), ld_cs, M, N, K,
                                         _stream(stream, A)))


def fp8q_quantize_tensor_dq(x, n, f, scale, q, y, amax_out=None, stream=None) -> None:
    _check(lib().fp8q_quantize_tensor_dq(_ptr(x), _dt(x), n, f, _ptr(scale), _ptr(q), _ptr(amax_out), _ptr(y),
                                         _dt(y), _stream(stream, x)))


def fp8q_quantize_tensor_delayed(x, n, f, state, q, y=None, stream=None) -> None:
    _check(lib().fp8q_quantize_tensor_delayed(_ptr(x), _dt(x), n, f, _ptr(state), _ptr(q), _ptr(y),
                                              _dt(y) if y is not None else F32, _stream(stream, x)))


def fp8q_gemm_blockscaled_qt(A, fa, lda, sA, sA_sm, sA_skb, B, fb, ldb, sB, gb, sB_sn, sB_skb, fc, eps, Cqt, ldcqt,
                             Cst, ld_cst, Cq, ldcq, Cs, ld_cs, M, N, K, stream=None) -> None:
    _check(lib().fp8q_gemm_blockscaled_qt(_ptr(A), fa, lda, _ptr(sA), sA_sm, sA_skb, _ptr(B), fb, ldb, _ptr(sB), gb,
                                          sB_sn, sB_skb, fc, eps, _ptr(Cqt), ldcqt, _ptr(Cst), ld_cst, _ptr(Cq), ldcq,
                                          _ptr(Cs), ld_cs, M, N, K, _stream(stream, A)))


def _same_dt(t, *others) -> int:
    """The element type of t, which the tensors among `others` must share."""
    dtype = t.dtype
    for o in others:
        if o is not None and o.__class__ is not int and o.dtype is not dtype:
            raise TypeError(f"these operands share one dtype, got {t.dtype} and {o.dtype}")
    return _dt(t)


def fp8q_rmsnorm_1x128(x, ldx, res, ldr, w, rows, cols, norm_eps, z, ldz, y, ldy, f, eps, q, ldq, scales, ld_s,
                       rstd=None, stream=None) -> None:
    _check(lib().fp8q_rmsnorm_1x128(_ptr(x), _same_dt(x, res, z, y), ldx, _ptr(res), ldr, _ptr(w), _dt(w), rows, cols,
                                    norm_eps, _ptr(z), ldz, _ptr(y), ldy, f, eps, _codes(q), ldq, _f32(scales), ld_s,
                                    _f32(rstd), _stream(stream, x)))


def fp8q_rmsnorm_bwd_workspace(rows, cols) -> int:
    return lib().fp8q_rmsnorm_bwd_workspace(rows, cols)


def fp8q_rmsnorm_bwd(dy, lddy, z, ldz, w, rstd, dres, lddr, rows, cols, dx, lddx, dw=None, ws=None, ws_bytes=0,
                     stream=None) -> None:
    _check(lib().fp8q_rmsnorm_bwd(_ptr(dy), _same_dt(dy, z, dres, dx), lddy, _ptr(z), ldz, _ptr(w), _dt(w), _f32(rstd),
                                  _ptr(dres), lddr, rows, cols, _ptr(dx), lddx, _f32(dw), _ptr(ws), ws_bytes,
                                  _stream(stream, dy)))


def fp8q_glu_blockscaled(A, fa, lda, sA, sA_sm, sA_skb, Bg, Bu, fb, ldb, sBg, sBu, sB_sn, sB_skb, act, H, ldh, gu, ldgu,
                         M, F, K, stream=None) -> None:
    _check(lib().fp8q_glu_blockscaled(_codes(A), fa, lda, _f32(sA), sA_sm, sA_skb, _codes(Bg), _codes(Bu), fb, ldb, _f32(sBg),
                                      _f32(sBu), sB_sn, sB_skb, act, _ptr(H), _dt(H), ldh, _bf16(gu), ldgu, M, F, K,
                                      _stream(stream, A)))


def fp8q_glu_blockscaled_fast(A, fa, lda, sA, sA_sm, sA_skb, Bg, Bu, fb, ldb, sBg, sBu, sB_sn, sB_skb, act, H, ldh, gu,
                              ldgu, M, F, K, stream=None) -> None:
    _check(lib().fp8q_glu_blockscaled_fast(_codes(A), fa, lda, _f32(sA), sA_sm, sA_skb, _codes(Bg), _codes(Bu), fb, ldb,
                                           _f32(sBg), _f32(sBu), sB_sn, sB_skb, act, _ptr(H), _dt(H), ldh, _bf16(gu),
                                           ldgu, M, F, K, _stream(stream, A)))


def fp8q_glu_blockscaled_q_workspace(M, F) -> int:
    return lib().fp8q_glu_blockscaled_q_workspace(M, F)


def fp8q_glu_blockscaled_q(A, fa, lda, sA, sA_sm, sA_skb, Bg, Bu, fb, ldb, sBg, sBu, sB_sn, sB_skb, act, fc, eps, Hq,
                           ldhq, Hs, ld_hs, gu, ldgu, M, F, K, ws=None, ws_bytes=0, stream=None) -> None:
    """Without `ws`, the few bytes a call of few rows needs come from torch's allocator."""
    handle = _stream(stream, A)
    if ws is None:
        ws_bytes = lib().fp8q_glu_blockscaled_q_workspace(M, F)
        if ws_bytes:
            ws = _workspace(ws_bytes, handle, stream, A)
    _check(lib().fp8q_glu_blockscaled_q(_codes(A), fa, lda, _f32(sA), sA_sm, sA_skb, _codes(Bg), _codes(Bu), fb, ldb,
                                        _f32(sBg), _f32(sBu), sB_sn, sB_skb, act, fc, eps, _codes(Hq), ldhq, _f32(Hs),
                                        ld_hs, _bf16(gu), ldgu, M, F, K, _ptr(ws), ws_bytes, handle))


def fp8q_glu_bwd_q(dH, lddh, gu, ldgu, act, fc, eps, Dq, lddq, Ds, ld_ds, Dt, lddt, Dst, ld_dst, fh, Ht, ldht, Hst,
                   ld_hst, M, F, stream=None) -> None:
    _check(lib().fp8q_glu_bwd_q(_ptr(dH), _dt(dH), lddh, _bf16(gu), ldgu, act, fc, eps, _codes(Dq), lddq, _f32(Ds), ld_ds,
                                _codes(Dt), lddt, _f32(Dst), ld_dst, fh, _codes(Ht), ldht, _f32(Hst), ld_hst, M, F,
                                _stream(stream, dH)))


def fp8q_gemm_blockscaled_few(A, fa, lda, sA, sA_sm, sA_skb, B, fb, ldb, sB, gb, sB_sn, sB_skb, C, ldc, M, N, K,
                              stream=None) -> None:
    _check(lib().fp8q_gemm_blockscaled_few(_codes(A), fa, lda, _f32(sA), sA_sm, sA_skb, _codes(B), fb, ldb, _f32(sB), gb,
                                           sB_sn, sB_skb, _ptr(C), _dt(C), ldc, M, N, K, _stream(stream, A)))


_native = None
_get_device = None


def _entries():
    """The module that marshals the calls below (csrc/fp8q_binding.cpp): pointers, fixed types and devices are read and
    checked there."""
    global _native, _get_device, _raw_stream
    if _native is None:
        import torch

        lib()
        try:
            from . import _fp8q_call as m
        except ImportError as e:
            raise ImportError(f"{e}: build it with `python -m block_scaled_precision_amax_amd.build`") from e
        m.types((torch.float32,), (torch.bfloat16, torch.int16, torch.uint16),
                (torch.uint8, torch.int8, torch.float8_e4m3fn, torch.float8_e5m2))
        _get_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        _native = m
    return _native


def _launch(fn, stream, t, *args, plan=None) -> None:
    """fn(device of t, *args, stream's handle) with that device as the current one, on which kernels are launched.  A host
    tensor's address, or one of another device, would fault in the kernel: fn refuses both.  With `plan`, the linear
    layer's (fast, codes, M, N, K), the workspace that the call needs on that device follows the arguments."""
    if t.__class__ is int or t is None:  # a raw pointer: what the tensors say, else the current device
        t = next((a for a in args if hasattr(a, "get_device")), None)
    dev = -1 if t is None else t.get_device()
    if dev >= 0 and _get_device() != dev:
        import torch

        with torch.cuda.device(dev):
            return _launch(fn, stream, t, *args, plan=plan)
    if dev >= 0:
        handle = _raw_stream(dev) if stream is None else stream if isinstance(stream, int) else stream.cuda_stream
    else:
        handle = _stream(stream) if t is None else 0
    if plan is not None:
        n = (_lib or lib()).fp8q_linear_blockscaled_workspace(*plan)
        # none for a host tensor, which fn refuses
        args += (_workspace(n, handle, stream, 0 if t is None else t) if n and (dev >= 0 or t is None) else None, n)
    rc = fn(dev, *args, handle)
    if rc:
        _check(rc)


def fp8q_layernorm_1x128(x, ldx, res, ldr, w, b, rows, cols, norm_eps, z, ldz, y, ldy, f, eps, q, ldq, scales, ld_s,
                         mean=None, rstd=None, stream=None) -> None:
    """w and b, of one dtype, may each be None (ones, zeros)."""
    wdt = F32 if w is None and b is None else _same_dt(b if w is None else w, b)
    _launch((_native or _entries()).fp8q_layernorm_1x128, stream, x, x, _same_dt(x, res, z, y), ldx, res, ldr, w, b, wdt, rows,
            cols, norm_eps, z, ldz, y, ldy, f, eps, q, ldq, scales, ld_s, mean, rstd)


def fp8q_layernorm_bwd_workspace(rows, cols) -> int:
    return lib().fp8q_layernorm_bwd_workspace(rows, cols)


def fp8q_layernorm_bwd(dy, lddy, z, ldz, w, mean, rstd, dres, lddr, rows, cols, dx, lddx, dw=None, db=None, ws=None,
                       ws_bytes=0, stream=None) -> None:
    _launch((_native or _entries()).fp8q_layernorm_bwd, stream, dy, dy, _same_dt(dy, z, dres, dx), lddy, z, ldz, w,
            F32 if w is None else _dt(w), mean, rstd, dres, lddr, rows, cols, dx, lddx, dw, db, ws, ws_bytes)


def fp8q_linear_blockscaled_workspace(fast, codes, M, N, K) -> int:
    return lib().fp8q_linear_blockscaled_workspace(fast, codes, M, N, K)


def _linear(fn, stream, A, plan, ws, ws_bytes, *args) -> None:
    if ws is None:
        _launch(fn, stream, A, *args, plan=plan)
    else:
        _launch(fn, stream, A, *args, ws, ws_bytes)


def fp8q_linear_blockscaled(A, fa, lda, sA, sA_sm, sA_skb, B, fb, ldb, sB, sB_sn, sB_skb, bias, act, res, ldr, C, ldc, pre,
                            ldpre, M, N, K, ws=None, ws_bytes=0, stream=None) -> None:
    """Without `ws`, what workspace the call needs comes from torch's allocator; so in the forms below."""
    _linear((_native or _entries()).fp8q_linear_blockscaled, stream, A, (0, 0, M, N, K), ws, ws_bytes, A, fa, lda, sA, sA_sm,
            sA_skb, B, fb, ldb, sB, sB_sn, sB_skb, bias, F32 if bias is None else _dt(bias), act, res, ldr, C, _same_dt(C, res),
            ldc, pre, ldpre, M, N, K)


def fp8q_linear_blockscaled_fast(A, fa, lda, sA, sA_sm, sA_skb, B, fb, ldb, sB, sB_sn, sB_skb, bias, act, res, ldr, C, ldc,
                                 pre, ldpre, M, N, K, ws=None, ws_bytes=0, stream=None) -> None:
    _linear((_native or _entries()).fp8q_linear_blockscaled_fast, stream, A, (1, 0, M, N, K), ws, ws_bytes, A, fa, lda, sA,
            sA_sm, sA_skb, B, fb, ldb, sB, sB_sn, sB_skb, bias, F32 if bias is None else _dt(bias), act, res, ldr, C,
            _same_dt(C, res), ldc, pre, ldpre, M, N, K)


def fp8q_linear_blockscaled_q(A, fa, lda, sA, sA_sm, sA_skb, B, fb, ldb, sB, sB_sn, sB_skb, bias, act, fc, eps, Cq, ldcq, Cs,
                              ld_cs, pre, ldpre, M, N, K, ws=None, ws_bytes=0, stream=None) -> None:
    _linear((_native or _entries()).fp8q_linear_blockscaled_q, stream, A, (0, 1, M, N, K), ws, ws_bytes, A, fa, lda, sA, sA_sm,
            sA_skb, B, fb, ldb, sB, sB_sn, sB_skb, bias, F32 if bias is None else _dt(bias), act, fc, eps, Cq, ldcq, Cs, ld_cs,
            pre, ldpre, M, N, K)


def fp8q_linear_blockscaled_q_fast(A, fa, lda, sA, sA_sm, sA_skb, B, fb, ldb, sB, sB_sn, sB_skb, bias, act, fc, eps, Cq,
                                   ldcq, Cs, ld_cs, pre, ldpre, M, N, K, ws=None, ws_bytes=0, stream=None) -> None:
    _linear((_native or _entries()).fp8q_linear_blockscaled_q_fast, stream, A, (1, 1, M, N, K), ws, ws_bytes, A, fa, lda, sA,
            sA_sm, sA_skb, B, fb, ldb, sB, sB_sn, sB_skb, bias, F32 if bias is None else _dt(bias), act, fc, eps, Cq, ldcq, Cs,
            ld_cs, pre, ldpre, M, N, K)


def fp8q_linear_bwd_q_workspace(M, N) -> int:
    return lib().fp8q_linear_bwd_q_workspace(M, N)


def fp8q_linear_bwd_q(dC, lddc, pre, ldpre, act, fc, eps, Dq, lddq, Ds, ld_ds, Dt, lddt, Dst, ld_dst, fh, Ht, ldht, Hst,
                      ld_hst, dbias, M, N, ws=None, ws_bytes=0, stream=None) -> None:
    _launch((_native or _entries()).fp8q_linear_bwd_q, stream, dC, dC, _dt(dC), lddc, pre, ldpre, act, fc, eps, Dq, lddq, Ds,
            ld_ds, Dt, lddt, Dst, ld_dst, fh, Ht, ldht, Hst, ld_hst, dbias, M, N, ws, ws_bytes)
