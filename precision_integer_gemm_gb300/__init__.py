"""Python binding of libigemm.so (exact int4 x int4 and W4A8 GEMM on sm_103a).

Argument marshalling only: each function passes device pointers, sizes and
the CUDA stream to the C entry point of the same name (include/igemm.h) and
raises IgemmError when it returns a non-zero status.  All work runs in the
library's CUDA kernels; if the shared library is missing, loading fails with
an error instead of falling back to anything else.

Tensors are torch CUDA tensors (or raw integer device addresses).  `stream`
defaults to torch's current stream on the current device.
"""

from __future__ import annotations

import ctypes
import os

from .build import LIB_PATH, build as build_library

__all__ = [
    "IgemmError", "load", "i4i4_gemm", "i4i4_gemm_noalloc", "w4a8_gemm", "i4i4_gemm_host", "w4a8_gemm_host", "w4a8_gemm_scaled", "fp8_gemm", "pack_int4",
    "fp8_blockscaled_gemm", "fp8_gemm_e5m2", "fp8_blockscaled_gemm_e5m2", "fp8_gemm_host", "fp8_gemm_e5m2_host",
    "fp8_blockscaled_gemm_host", "fp8_blockscaled_gemm_e5m2_host", "unpack_int4",
    "igemm_strerror",
    "igemm_last_status", "igemm_watchdog_selftest", "igemm_kernels_launched", "igemm_time_next_gemm",
    "igemm_skinny_plan", "igemm_ss_plan", "igemm_route",
    "pack_mxfp4", "pack_nvfp4", "igemm_mxfp4", "igemm_nvfp4",
    "igemm_mxfp4_grouped", "igemm_nvfp4_grouped", "igemm_moe_route", "igemm_moe_combine",
    "fp4_code_bytes", "mxfp4_scale_pitch", "nvfp4_scale_pitch",
    "pack_bsfp8", "igemm_bsfp8", "igemm_bsfp8_grouped", "bsfp8_code_bytes", "bsfp8_scale_pitch",
    "igemm_moe_route_scored", "igemm_moe_route_scored_grad",
    "EXPORTED_SYMBOLS", "LIB_PATH", "build_library",
]

EXPORTED_SYMBOLS = ("i4i4_gemm", "i4i4_gemm_noalloc", "w4a8_gemm", "i4i4_gemm_host", "w4a8_gemm_host", "w4a8_gemm_scaled", "fp8_gemm",
                    "fp8_gemm_e5m2", "fp8_blockscaled_gemm", "fp8_blockscaled_gemm_e5m2", "fp8_gemm_host",
                    "fp8_gemm_e5m2_host", "fp8_blockscaled_gemm_host", "fp8_blockscaled_gemm_e5m2_host", "pack_int4", "unpack_int4", "igemm_strerror", "igemm_last_status",
                    "igemm_watchdog_selftest", "igemm_kernels_launched",
                    "igemm_time_next_gemm", "igemm_skinny_plan", "igemm_ss_plan", "igemm_route",
                    "pack_mxfp4", "pack_nvfp4", "igemm_mxfp4", "igemm_nvfp4", "igemm_mxfp4_grouped",
                    "igemm_nvfp4_grouped", "igemm_moe_route", "igemm_moe_combine",
                    "pack_bsfp8", "igemm_bsfp8", "igemm_bsfp8_grouped", "igemm_moe_route_scored",
                    "igemm_moe_route_scored_grad")

IGEMM_OK = 0
IGEMM_INVALID_ARGUMENT = 1
IGEMM_UNSUPPORTED_SHAPE = 2
IGEMM_MISALIGNED = 3
IGEMM_OVERFLOW_BOUND = 4
IGEMM_CUDA_ERROR = 5
IGEMM_DEVICE_TIMEOUT = 6
IGEMM_WORKSPACE_LIMIT = 7
NOALLOC_WORKSPACE_BYTES = 32 << 20

_lib = None


class IgemmError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {igemm_strerror(code)} (status {code})")


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libigemm.so (the in-tree build); raises if it has not been built."""
    global _lib
    if path is not None:
        return _bind(ctypes.CDLL(path))
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OSError(f"{LIB_PATH} is missing: build it with precision_integer_gemm_gb300.build_library()")
        _lib = _bind(ctypes.CDLL(LIB_PATH))
    return _lib


def _bind(lib: ctypes.CDLL) -> ctypes.CDLL:
    p = ctypes.c_void_p
    i = ctypes.c_int
    i64 = ctypes.c_int64
    lib.i4i4_gemm.argtypes = [p, p, p, i, i, i, p]
    lib.i4i4_gemm.restype = i
    lib.i4i4_gemm_noalloc.argtypes = [p, p, p, i, i, i, p]
    lib.i4i4_gemm_noalloc.restype = i
    lib.w4a8_gemm_scaled.argtypes = [p, p, p, p, p, i, i, i, p]
    lib.w4a8_gemm_scaled.restype = i
    for name in ("fp8_gemm", "fp8_gemm_e5m2", "fp8_gemm_host", "fp8_gemm_e5m2_host"):
        getattr(lib, name).argtypes = [p, p, p, i, i, i, p]
        getattr(lib, name).restype = i
    for name in ("fp8_blockscaled_gemm", "fp8_blockscaled_gemm_e5m2", "fp8_blockscaled_gemm_host",
                 "fp8_blockscaled_gemm_e5m2_host"):
        getattr(lib, name).argtypes = [p, p, p, p, p, i, i, i, p]
        getattr(lib, name).restype = i
    lib.w4a8_gemm.argtypes = [p, p, p, i, i, i, p]
    lib.w4a8_gemm.restype = i
    for name in ("i4i4_gemm_host", "w4a8_gemm_host"):
        getattr(lib, name).argtypes = [p, p, p, i, i, i, p]
        getattr(lib, name).restype = i
    lib.pack_int4.argtypes = [p, p, i64, i64, p]
    lib.pack_int4.restype = i
    lib.unpack_int4.argtypes = [p, p, i64, i64, p]
    lib.unpack_int4.restype = i
    lib.igemm_strerror.argtypes = [i]
    lib.igemm_strerror.restype = ctypes.c_char_p
    lib.igemm_last_status.argtypes = [p]
    lib.igemm_last_status.restype = i
    lib.igemm_time_next_gemm.argtypes = [p, p]
    lib.igemm_time_next_gemm.restype = i
    lib.igemm_skinny_plan.argtypes = [i, i, i, i, i, i, i, ctypes.POINTER(ctypes.c_int)]
    lib.igemm_skinny_plan.restype = i
    lib.igemm_ss_plan.argtypes = [i, i, i, i, i, ctypes.POINTER(ctypes.c_int)]
    lib.igemm_ss_plan.restype = i
    lib.igemm_route.argtypes = [i, i, i, i, i, i, i, ctypes.POINTER(ctypes.c_int)]
    lib.igemm_route.restype = i
    lib.igemm_kernels_launched.argtypes = []
    lib.igemm_kernels_launched.restype = ctypes.c_uint64
    lib.pack_mxfp4.argtypes = [p, i, i64, i, p, i, p, p, i, i, p]
    lib.pack_nvfp4.argtypes = [p, i, i64, i, p, i, p, p, p, i, i, p]
    lib.igemm_mxfp4.argtypes = [p, p, p, p, p, i, i, i, i, p]
    lib.igemm_nvfp4.argtypes = [p, p, p, p, p, p, i, i, i, i, p]
    lib.igemm_mxfp4_grouped.argtypes = [p, p, p, p, p, p, i, i, i, i, i, p]
    lib.igemm_nvfp4_grouped.argtypes = [p, p, p, p, p, p, p, i, i, i, i, i, p]
    lib.igemm_moe_route.argtypes = [p, i, p, p, p, p, p, i, i, i, i, p]
    lib.igemm_moe_combine.argtypes = [p, p, p, p, i, i, i, i, p]
    lib.pack_bsfp8.argtypes = [p, i, i64, i, p, i, i, i, p, p, i, i, p]
    lib.igemm_bsfp8.argtypes = [p, p, p, p, p, i, i, i, i, i, p]
    lib.igemm_bsfp8_grouped.argtypes = [p, p, p, p, p, p, i, i, i, i, i, i, p]
    f = ctypes.c_float
    lib.igemm_moe_route_scored.argtypes = [p, i, p, p, p, p, p, p, i, i, i, i, i, i, i, i, f, p]
    lib.igemm_moe_route_scored_grad.argtypes = [p, i, p, p, p, i, i, i, i, i, f, p]
    for name in ("pack_mxfp4", "pack_nvfp4", "igemm_mxfp4", "igemm_nvfp4", "igemm_mxfp4_grouped",
                 "igemm_nvfp4_grouped", "igemm_moe_route", "igemm_moe_combine", "pack_bsfp8", "igemm_bsfp8",
                 "igemm_bsfp8_grouped", "igemm_moe_route_scored", "igemm_moe_route_scored_grad"):
        getattr(lib, name).restype = i
    lib.igemm_watchdog_selftest.argtypes = [ctypes.c_uint32, p]
    lib.igemm_watchdog_selftest.restype = i
    return lib


def _arg(x, nbytes: int, on_device: bool, what: str) -> int | None:
    """Address of an array argument after the checks a raw pointer cannot get:
    a tensor must live where the entry point reads it (CUDA memory, or host
    memory for the *_host entry points), be contiguous and hold at least
    `nbytes` bytes.  None and raw integer addresses pass through unchecked."""
    if x is None or isinstance(x, int):
        return x
    if bool(x.is_cuda) != on_device:
        raise ValueError(f"{what} must be a {'CUDA' if on_device else 'host (CPU)'} tensor")
    if not x.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    have = x.numel() * x.element_size()
    if have < nbytes:
        raise ValueError(f"{what} holds {have} bytes; the call needs {nbytes}")
    return x.data_ptr()


def _n(*dims: int) -> int:
    """Product of sizes, 0 if any is negative (the library rejects those itself)."""
    out = 1
    for d in dims:
        if d < 0:
            return 0
        out *= d
    return out


_raw_stream = None  # device index -> handle of torch's current stream there
_current_device = None


def _stream(stream) -> int | None:
    global _raw_stream, _current_device
    if stream is None:
        if _raw_stream is None:
            import torch
            _current_device = torch.cuda.current_device
            # (the handle alone: building a Stream object takes 2 us of a small call)
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda i: torch.cuda.current_stream(i).cuda_stream)
        return _raw_stream(_current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(code: int, where: str) -> None:
    if code != IGEMM_OK:
        raise IgemmError(code, where)


def _int_gemm_args(A, Bp, C, M, N, K, a_bytes, on_device, where):
    return (_arg(A, a_bytes, on_device, f"{where}: A"),
            _arg(Bp, _n(N, K) // 2, on_device, f"{where}: Bp"),
            _arg(C, 4 * _n(M, N), on_device, f"{where}: C"))


def i4i4_gemm(Ap, Bp, C, M: int, N: int, K: int, stream=None) -> None:
    """C[M,N] (int32) = A . B^T for packed int4 Ap [M,K/2] and Bp [N,K/2]."""
    a, b, c = _int_gemm_args(Ap, Bp, C, M, N, K, _n(M, K) // 2, True, "i4i4_gemm")
    _check(load().i4i4_gemm(a, b, c, M, N, K, _stream(stream)), "i4i4_gemm")


def i4i4_gemm_noalloc(Ap, Bp, C, M: int, N: int, K: int, stream=None) -> None:
    """Same as i4i4_gemm, with the library's fixed 32 MiB device workspace
    instead of allocated memory (for callers that cannot allocate during a
    call); larger problems raise with IGEMM_WORKSPACE_LIMIT.  Calls that
    overlap on the GPU share that workspace and race."""
    a, b, c = _int_gemm_args(Ap, Bp, C, M, N, K, _n(M, K) // 2, True, "i4i4_gemm_noalloc")
    _check(load().i4i4_gemm_noalloc(a, b, c, M, N, K, _stream(stream)), "i4i4_gemm_noalloc")


def w4a8_gemm(A, Bp, C, M: int, N: int, K: int, stream=None) -> None:
    """C[M,N] (int32) = A . B^T for int8 A [M,K] and packed int4 Bp [N,K/2]."""
    a, b, c = _int_gemm_args(A, Bp, C, M, N, K, _n(M, K), True, "w4a8_gemm")
    _check(load().w4a8_gemm(a, b, c, M, N, K, _stream(stream)), "w4a8_gemm")


def i4i4_gemm_host(Ap, Bp, C, M: int, N: int, K: int, stream=None) -> None:
    """i4i4_gemm with Ap, Bp and C in host memory (CPU tensors, pinned for overlap);
    C is complete once `stream` has reached the end of the call."""
    a, b, c = _int_gemm_args(Ap, Bp, C, M, N, K, _n(M, K) // 2, False, "i4i4_gemm_host")
    _check(load().i4i4_gemm_host(a, b, c, M, N, K, _stream(stream)), "i4i4_gemm_host")


def w4a8_gemm_host(A, Bp, C, M: int, N: int, K: int, stream=None) -> None:
    """w4a8_gemm with A, Bp and C in host memory (CPU tensors, pinned for overlap);
    C is complete once `stream` has reached the end of the call."""
    a, b, c = _int_gemm_args(A, Bp, C, M, N, K, _n(M, K), False, "w4a8_gemm_host")
    _check(load().w4a8_gemm_host(a, b, c, M, N, K, _stream(stream)), "w4a8_gemm_host")


def w4a8_gemm_scaled(A, Bp, scale_a, scale_b, C, M: int, N: int, K: int, stream=None) -> None:
    """C[M,N] (bfloat16) = per-channel dequantised W4A8 product: bf16(float(A . B^T) * scale_a[m] * scale_b[n])."""
    w = "w4a8_gemm_scaled"
    a, b, _ = _int_gemm_args(A, Bp, None, M, N, K, _n(M, K), True, w)
    _check(load().w4a8_gemm_scaled(a, b, _arg(scale_a, 4 * _n(M), True, f"{w}: scale_a"),
                                   _arg(scale_b, 4 * _n(N), True, f"{w}: scale_b"),
                                   _arg(C, 2 * _n(M, N), True, f"{w}: C"), M, N, K, _stream(stream)), w)


def _fp8_args(A, B, C, M, N, K, on_device, where):
    return (_arg(A, _n(M, K), on_device, f"{where}: A"), _arg(B, _n(N, K), on_device, f"{where}: B"),
            _arg(C, 4 * _n(M, N), on_device, f"{where}: C"))


def _fp8bs_args(A, B, SFA, SFB, C, M, N, K, on_device, where):
    kb = -(-K // 128) if K > 0 else 0
    return (_arg(A, _n(M, K), on_device, f"{where}: A"), _arg(B, _n(N, K), on_device, f"{where}: B"),
            _arg(SFA, 4 * _n(M, kb), on_device, f"{where}: SFA"), _arg(SFB, 4 * _n(N, kb), on_device, f"{where}: SFB"),
            _arg(C, 4 * _n(M, N), on_device, f"{where}: C"))


def fp8_gemm(A, B, C, M: int, N: int, K: int, stream=None) -> None:
    """C[M,N] (float32) = A . B^T for E4M3 byte matrices A [M,K] and B [N,K]."""
    _check(load().fp8_gemm(*_fp8_args(A, B, C, M, N, K, True, "fp8_gemm"), M, N, K, _stream(stream)), "fp8_gemm")


def fp8_gemm_e5m2(A, B, C, M: int, N: int, K: int, stream=None) -> None:
    """C[M,N] (float32) = A . B^T for E5M2 byte matrices A [M,K] and B [N,K]."""
    _check(load().fp8_gemm_e5m2(*_fp8_args(A, B, C, M, N, K, True, "fp8_gemm_e5m2"), M, N, K, _stream(stream)),
           "fp8_gemm_e5m2")


def fp8_blockscaled_gemm(A, B, SFA, SFB, C, M: int, N: int, K: int, stream=None) -> None:
    """C[M,N] (float32) = sum over 128-k blocks kb of SFA[m,kb] * SFB[n,kb] * (A . B^T over the block),
    for E4M3 byte matrices A [M,K], B [N,K] and float32 scales SFA [M,ceil(K/128)], SFB [N,ceil(K/128)]."""
    _check(load().fp8_blockscaled_gemm(*_fp8bs_args(A, B, SFA, SFB, C, M, N, K, True, "fp8_blockscaled_gemm"), M, N,
                                       K, _stream(stream)), "fp8_blockscaled_gemm")


def fp8_blockscaled_gemm_e5m2(A, B, SFA, SFB, C, M: int, N: int, K: int, stream=None) -> None:
    """fp8_blockscaled_gemm for E5M2 byte matrices A [M,K] and B [N,K]."""
    _check(load().fp8_blockscaled_gemm_e5m2(*_fp8bs_args(A, B, SFA, SFB, C, M, N, K, True,
                                                          "fp8_blockscaled_gemm_e5m2"), M, N, K, _stream(stream)),
           "fp8_blockscaled_gemm_e5m2")


def fp8_gemm_host(A, B, C, M: int, N: int, K: int, stream=None) -> None:
    """fp8_gemm with A, B and C in host memory (CPU tensors, pinned for overlap)."""
    _check(load().fp8_gemm_host(*_fp8_args(A, B, C, M, N, K, False, "fp8_gemm_host"), M, N, K, _stream(stream)),
           "fp8_gemm_host")


def fp8_gemm_e5m2_host(A, B, C, M: int, N: int, K: int, stream=None) -> None:
    """fp8_gemm_e5m2 with A, B and C in host memory (CPU tensors, pinned for overlap)."""
    _check(load().fp8_gemm_e5m2_host(*_fp8_args(A, B, C, M, N, K, False, "fp8_gemm_e5m2_host"), M, N, K,
                                     _stream(stream)), "fp8_gemm_e5m2_host")


def fp8_blockscaled_gemm_host(A, B, SFA, SFB, C, M: int, N: int, K: int, stream=None) -> None:
    """fp8_blockscaled_gemm with A, B, SFA, SFB and C in host memory."""
    _check(load().fp8_blockscaled_gemm_host(*_fp8bs_args(A, B, SFA, SFB, C, M, N, K, False,
                                                          "fp8_blockscaled_gemm_host"), M, N, K, _stream(stream)),
           "fp8_blockscaled_gemm_host")


def fp8_blockscaled_gemm_e5m2_host(A, B, SFA, SFB, C, M: int, N: int, K: int, stream=None) -> None:
    """fp8_blockscaled_gemm_e5m2 with A, B, SFA, SFB and C in host memory."""
    _check(load().fp8_blockscaled_gemm_e5m2_host(*_fp8bs_args(A, B, SFA, SFB, C, M, N, K, False,
                                                               "fp8_blockscaled_gemm_e5m2_host"), M, N, K,
                                                 _stream(stream)), "fp8_blockscaled_gemm_e5m2_host")


def pack_int4(logical, packed, rows: int, K: int, stream=None) -> None:
    """packed [rows,K/2] = two int4 values per byte of logical [rows,K] (low nibble = even k)."""
    _check(load().pack_int4(_arg(logical, _n(rows, K), True, "pack_int4: logical"),
                            _arg(packed, _n(rows, K) // 2, True, "pack_int4: packed"), rows, K, _stream(stream)),
           "pack_int4")


def unpack_int4(packed, logical, rows: int, K: int, stream=None) -> None:
    """logical [rows,K] int8 = the sign-extended nibbles of packed [rows,K/2] (low nibble = even k)."""
    _check(load().unpack_int4(_arg(packed, _n(rows, K) // 2, True, "unpack_int4: packed"),
                              _arg(logical, _n(rows, K), True, "unpack_int4: logical"), rows, K, _stream(stream)),
           "unpack_int4")


# ---------------------------------------------------------------- 4-bit floating point, mixture of experts
_TYPES = {"torch.float32": (0, 4), "torch.bfloat16": (1, 2), "torch.float16": (2, 2)}
_type_of = {}  # torch dtype -> (igemm_type, bytes), filled as dtypes are met
_names = {}    # torch dtype -> its name


def fp4_code_bytes(K: int) -> int:
    """Bytes of a row of K packed e2m1 codes (whole blocks of 32)."""
    return -(-K // 32) * 16


def mxfp4_scale_pitch(K: int) -> int:
    """Bytes of a row of mxfp4 scales: one per 32 k, rounded up to 16."""
    return -(-K // 512) * 16


def nvfp4_scale_pitch(K: int) -> int:
    """Bytes of a row of nvfp4 scales: one per 16 k, rounded up to 16."""
    return -(-K // 256) * 16


def _type(x, what: str) -> tuple[int, int]:
    """(igemm_type, bytes per element) of a tensor."""
    t = _type_of.get(x.dtype)
    if t is None:
        t = _TYPES.get(str(x.dtype))
        if t is None:
            raise ValueError(f"{what}: a tensor of float32, bfloat16 or float16 is wanted, not of {x.dtype}")
        _type_of[x.dtype] = t
    return t


def _dev(x, nbytes: int, where: str, name: str):
    """_arg for device memory, its message made only when it is needed."""
    if x is None or isinstance(x, int):
        return x
    if x.is_cuda and x.is_contiguous() and x.nbytes >= nbytes:
        return x.data_ptr()
    return _arg(x, nbytes, True, f"{where}: {name}")


def _typed(x, dtype: str, count: int, where: str, name: str):
    """_dev for `count` 4-byte elements of torch type `dtype`."""
    if x is None or isinstance(x, int):
        return x
    if _names.get(x.dtype) != dtype:
        _names[x.dtype] = str(x.dtype)
        if _names[x.dtype] != dtype:
            raise ValueError(f"{where}: {name} must be {dtype}, not {x.dtype}")
    # (_dev's checks again: a call of it for each argument is a tenth of a small call's time)
    if x.is_cuda and x.is_contiguous() and x.nbytes >= 4 * count:
        return x.data_ptr()
    return _arg(x, 4 * count, True, f"{where}: {name}")


def _pack_operand(where, x, rows, K, index):
    """(type, leading dimension, transposed, rows) of the matrix x that `rows` rows of K are packed from."""
    t, _ = _type(x, where)
    if not x.is_cuda or x.dim() != 2:
        raise ValueError(f"{where}: x must be a CUDA matrix")
    (r, c), (sr, sc) = x.shape, x.stride()
    if c != K or (index is None and r != rows):
        raise ValueError(f"{where}: x is {tuple(x.shape)}; the call packs {rows} rows of {K}")
    # a dimension of one element has no stride of its own
    if c == 1 or sc == 1:
        transposed, ld = 0, (sr if r > 1 else max(sr, c))
    elif r == 1 or sr == 1:
        transposed, ld = 1, sc
    else:
        raise ValueError(f"{where}: x must have unit stride along one dimension")
    if ld < (r if transposed else c):
        raise ValueError(f"{where}: x has overlapping rows")
    if transposed and index is not None:
        raise ValueError(f"{where}: rows of a transposed x cannot be gathered")
    return t, ld, transposed, r


def _pack_fp4(fn, where, x, extra, codes, scales, rows, K, index, pitch, stream):
    t, ld, transposed, r = _pack_operand(where, x, rows, K, index)
    n = _n(rows)
    _check(fn(x.data_ptr(), t, ld, transposed, _typed(index, "torch.int32", n, where, "index"), r, *extra,
              _dev(codes, n * fp4_code_bytes(K), where, "codes"), _dev(scales, n * pitch, where, "scales"), rows, K,
              _stream(stream)), where)


def pack_mxfp4(x, codes, scales, rows: int, K: int, index=None, stream=None) -> None:
    """codes [rows, fp4_code_bytes(K)], scales [rows, mxfp4_scale_pitch(K)] (uint8) = x quantised to e2m1 with one
    power-of-two scale per 32 k.  x: CUDA matrix [rows, K] (float32, bfloat16 or float16) with unit stride along
    one dimension; with `index` (int32 [rows]) row r is x[index[r]], zeros where index[r] is out of range."""
    _pack_fp4(load().pack_mxfp4, "pack_mxfp4", x, (), codes, scales, rows, K, index, mxfp4_scale_pitch(K), stream)


def pack_nvfp4(x, tensor_scale, codes, scales, rows: int, K: int, index=None, stream=None) -> None:
    """pack_mxfp4 with one e4m3 scale per 16 k, relative to tensor_scale (float32 [1] on the device, None: 1);
    scales [rows, nvfp4_scale_pitch(K)]."""
    _pack_fp4(load().pack_nvfp4, "pack_nvfp4", x, (_typed(tensor_scale, "torch.float32", 1, "pack_nvfp4", "tensor_scale"),),
              codes, scales, rows, K, index, nvfp4_scale_pitch(K), stream)


def _fp4_args(A, B, SFA, SFB, C, M, E, N, K, pitch, where):
    kb = fp4_code_bytes(K)
    t, size = _type(C, where)
    m, n = _n(M), _n(E, N)  # (rows of A and of B)
    return ((_dev(A, m * kb, where, "A"), _dev(B, n * kb, where, "B"),
             _dev(SFA, m * pitch, where, "SFA"), _dev(SFB, n * pitch, where, "SFB")),
            (_dev(C, size * _n(M, N), where, "C"), t))


def igemm_mxfp4(A, B, SFA, SFB, C, M: int, N: int, K: int, stream=None) -> None:
    """C[M,N] (float32, bfloat16 or float16) = A . B^T of mxfp4 matrices (codes and scales as pack_mxfp4 writes them)."""
    w = "igemm_mxfp4"
    ops, c = _fp4_args(A, B, SFA, SFB, C, M, 1, N, K, mxfp4_scale_pitch(K), w)
    _check(load().igemm_mxfp4(*ops, *c, M, N, K, _stream(stream)), w)


def igemm_nvfp4(A, B, SFA, SFB, alpha, C, M: int, N: int, K: int, stream=None) -> None:
    """C[M,N] (float32, bfloat16 or float16) = alpha * A . B^T of nvfp4 matrices; alpha: float32 [1] on the device
    (the product of the operands' tensor scales), None: 1."""
    w = "igemm_nvfp4"
    ops, c = _fp4_args(A, B, SFA, SFB, C, M, 1, N, K, nvfp4_scale_pitch(K), w)
    _check(load().igemm_nvfp4(*ops, _typed(alpha, "torch.float32", 1, w, "alpha"), *c, M, N, K, _stream(stream)), w)


def igemm_mxfp4_grouped(A, B, SFA, SFB, offsets, C, rows: int, E: int, N: int, K: int, stream=None) -> None:
    """Rows offsets[e] .. offsets[e+1]-1 of C [rows, N] = those rows of A times the transpose of B[e] (B: E matrices
    of N rows); offsets: int32 [E+1] on the device.  Rows of no group are left as they were."""
    w = "igemm_mxfp4_grouped"
    ops, c = _fp4_args(A, B, SFA, SFB, C, rows, E, N, K, mxfp4_scale_pitch(K), w)
    _check(load().igemm_mxfp4_grouped(*ops, _typed(offsets, "torch.int32", _n(E + 1), w, "offsets"), *c, rows, E, N,
                                      K, _stream(stream)), w)


def igemm_nvfp4_grouped(A, B, SFA, SFB, offsets, alpha, C, rows: int, E: int, N: int, K: int, stream=None) -> None:
    """igemm_mxfp4_grouped for nvfp4 matrices; alpha: float32 [E] on the device, None: 1."""
    w = "igemm_nvfp4_grouped"
    ops, c = _fp4_args(A, B, SFA, SFB, C, rows, E, N, K, nvfp4_scale_pitch(K), w)
    _check(load().igemm_nvfp4_grouped(*ops, _typed(offsets, "torch.int32", _n(E + 1), w, "offsets"),
                                      _typed(alpha, "torch.float32", _n(E), w, "alpha"), *c, rows, E, N, K,
                                      _stream(stream)), w)


def igemm_moe_route(logits, experts, weights, offsets, tokens, slots, T: int, E: int, k: int, normalize: bool = True,
                    stream=None) -> None:
    """The k largest of logits [T,E] per token: experts [T,k] (int32, -1: none left), softmax weights [T,k] (float32,
    over the chosen or, normalize False, over all E), and the pairs sorted by expert: offsets [E+1], tokens [T*k]
    (sorted place -> token, -1 past the last), slots [T,k] (pair -> sorted place, -1), int32."""
    w = "igemm_moe_route"
    t, size = _type(logits, w)
    pairs = _n(T, k)
    _check(load().igemm_moe_route(
        _dev(logits, size * _n(T, E), w, "logits"), t, _typed(experts, "torch.int32", pairs, w, "experts"),
        _typed(weights, "torch.float32", pairs, w, "weights"),
        _typed(offsets, "torch.int32", _n(E + 1), w, "offsets"), _typed(tokens, "torch.int32", pairs, w, "tokens"),
        _typed(slots, "torch.int32", pairs, w, "slots"), T, E, k, 1 if normalize else 0, _stream(stream)), w)


SCORES = {"softmax": 0, "sigmoid": 1}


def _score(score: str, where: str) -> int:
    s = SCORES.get(score)
    if s is None:
        raise ValueError(f"{where}: score must be 'softmax' or 'sigmoid', not {score!r}")
    return s


def igemm_moe_route_scored(logits, bias, experts, weights, offsets, tokens, slots, T: int, E: int, k: int,
                           score: str = "softmax", groups: int = 1, group_k: int = 1, group_top: int = 1,
                           normalize: bool = True, scale: float = 1.0, stream=None) -> None:
    """igemm_moe_route by scores: softmax or sigmoid of logits [T,E] plus bias (float32 [E], None: 0; for the choice
    only), the group_k best of `groups` equal runs of experts (by the sum of their group_top largest), the k best
    experts in them; weights = scale * score, over the sum of the chosen scores (normalize)."""
    w = "igemm_moe_route_scored"
    t, size = _type(logits, w)
    if T < 0 or E < 0 or k < 0:
        scores = pairs = e = 0  # (the library rejects those itself)
    else:
        scores, pairs, e = T * E, T * k, E
    _check(load().igemm_moe_route_scored(
        _dev(logits, size * scores, w, "logits"), t, _typed(bias, "torch.float32", e, w, "bias"),
        _typed(experts, "torch.int32", pairs, w, "experts"), _typed(weights, "torch.float32", pairs, w, "weights"),
        _typed(offsets, "torch.int32", e + 1, w, "offsets"), _typed(tokens, "torch.int32", pairs, w, "tokens"),
        _typed(slots, "torch.int32", pairs, w, "slots"), T, E, k, _score(score, w), groups, group_k, group_top,
        1 if normalize else 0, scale, _stream(stream)), w)


def igemm_moe_route_scored_grad(logits, experts, dweights, dlogits, T: int, E: int, k: int, score: str = "softmax",
                                normalize: bool = True, scale: float = 1.0, stream=None) -> None:
    """dlogits [T,E] (of logits' type) = gradient of the logits for dweights [T,k] (float32), that of the weights which
    igemm_moe_route_scored gave the choices experts [T,k] with the same score, normalize and scale."""
    w = "igemm_moe_route_scored_grad"
    t, size = _type(logits, w)
    if dlogits.dtype != logits.dtype:
        raise ValueError(f"{w}: dlogits must have logits' type")
    if T < 0 or E < 0 or k < 0:
        scores = pairs = 0  # (the library rejects those itself)
    else:
        scores, pairs = T * E, T * k
    _check(load().igemm_moe_route_scored_grad(
        _dev(logits, size * scores, w, "logits"), t, _typed(experts, "torch.int32", pairs, w, "experts"),
        _typed(dweights, "torch.float32", pairs, w, "dweights"), _dev(dlogits, size * scores, w, "dlogits"), T, E, k,
        _score(score, w), 1 if normalize else 0, scale, _stream(stream)), w)


def igemm_moe_combine(Y, slots, weights, out, T: int, k: int, N: int, stream=None) -> None:
    """out [T,N] = sum over j of weights[t,j] * Y[slots[t,j]] (Y [T*k,N] and out of one type; slots of -1 add nothing)."""
    w = "igemm_moe_combine"
    t, size = _type(Y, w)
    if out.dtype != Y.dtype:
        raise ValueError(f"{w}: out must have Y's type")
    pairs = _n(T, k)
    _check(load().igemm_moe_combine(
        _dev(Y, size * _n(pairs, N), w, "Y"), _typed(slots, "torch.int32", pairs, w, "slots"),
        _typed(weights, "torch.float32", pairs, w, "weights"), _dev(out, size * _n(T, N), w, "out"), t, T,
        k, N, _stream(stream)), w)


# ---------------------------------------------------------------- block-scaled fp8
FP8_FORMATS = {"e4m3": 0, "e5m2": 1}


def bsfp8_code_bytes(K: int) -> int:
    """Bytes of a row of K fp8 codes (whole 16-byte units)."""
    return -(-K // 16) * 16


def bsfp8_scale_pitch(K: int) -> int:
    """float32 scales of a row of K values: one per 128 k, rounded up to four."""
    return -(-K // 512) * 4


def _fp8_format(format: str, where: str) -> int:
    f = FP8_FORMATS.get(format)
    if f is None:
        raise ValueError(f"{where}: format must be 'e4m3' or 'e5m2', not {format!r}")
    return f


def pack_bsfp8(x, codes, scales, rows: int, K: int, tile_rows: int = 1, format: str = "e4m3", index=None,
               stream=None) -> None:
    """codes [rows, bsfp8_code_bytes(K)] (a byte each), scales [ceil(rows/tile_rows), bsfp8_scale_pitch(K)] (float32) =
    x quantised to fp8 with one scale per tile_rows (1: activations, 128: weights) x 128 k.  x and index as for
    pack_mxfp4 (index with tile_rows 1 only)."""
    w = "pack_bsfp8"
    t, ld, transposed, r = _pack_operand(w, x, rows, K, index)
    n = rows if rows > 0 else 0
    tiles = n if tile_rows == 1 else -(-n // 128)
    _check(load().pack_bsfp8(x.data_ptr(), t, ld, transposed, _typed(index, "torch.int32", n, w, "index"), r, tile_rows,
                             _fp8_format(format, w), _dev(codes, n * bsfp8_code_bytes(K), w, "codes"),
                             _typed(scales, "torch.float32", tiles * bsfp8_scale_pitch(K), w, "scales"), rows, K,
                             _stream(stream)), w)


def _bsfp8_args(A, B, SFA, SFB, C, M, E, N, K, where):
    t, size = _type(C, where)
    if M < 0 or E < 0 or N < 0 or K < 0:
        m = rows = tiles = c = kb = pitch = 0  # (the library rejects those itself)
    else:
        kb, pitch = -(-K // 16) * 16, -(-K // 512) * 4
        m, rows, tiles, c = M, E * N, E * -(-N // 128), size * M * N
    return ((_dev(A, m * kb, where, "A"), _dev(B, rows * kb, where, "B"),
             _typed(SFA, "torch.float32", m * pitch, where, "SFA"), _typed(SFB, "torch.float32", tiles * pitch, where, "SFB")),
            (_dev(C, c, where, "C"), t))


def igemm_bsfp8(A, B, SFA, SFB, C, M: int, N: int, K: int, format: str = "e4m3", stream=None) -> None:
    """C[M,N] (float32, bfloat16 or float16) = A . B^T of block-scaled fp8 matrices: A as pack_bsfp8 writes it with
    tile_rows 1, B with tile_rows 128."""
    w = "igemm_bsfp8"
    ops, c = _bsfp8_args(A, B, SFA, SFB, C, M, 1, N, K, w)
    _check(load().igemm_bsfp8(*ops, *c, _fp8_format(format, w), M, N, K, _stream(stream)), w)


def igemm_bsfp8_grouped(A, B, SFA, SFB, offsets, C, rows: int, E: int, N: int, K: int, format: str = "e4m3",
                        stream=None) -> None:
    """Rows offsets[e] .. offsets[e+1]-1 of C [rows, N] = those rows of A times the transpose of B[e] (B [E, N, ...], SFB
    [E, ceil(N/128), ...]); offsets: int32 [E+1] on the device.  Rows of no group are left as they were."""
    w = "igemm_bsfp8_grouped"
    ops, c = _bsfp8_args(A, B, SFA, SFB, C, rows, E, N, K, w)
    _check(load().igemm_bsfp8_grouped(*ops, _typed(offsets, "torch.int32", _n(E + 1), w, "offsets"), *c,
                                      _fp8_format(format, w), rows, E, N, K, _stream(stream)), w)


def igemm_strerror(code: int) -> str:
    return load().igemm_strerror(code).decode()


def igemm_last_status(stream=None) -> int:
    return int(load().igemm_last_status(_stream(stream)))


def igemm_time_next_gemm(start, stop) -> None:
    """Arm two CUDA events (torch.cuda.Event with timing, already recorded
    once so that they exist, or raw handles) around the GEMM kernel of this
    thread's next GEMM call."""
    h = [e if isinstance(e, int) else e.cuda_event for e in (start, stop)]
    _check(load().igemm_time_next_gemm(h[0], h[1]), "igemm_time_next_gemm")


def igemm_skinny_plan(variant: str, M: int, N: int, K: int, sms: int, pairs: int, quads: int) -> dict:
    """The K split a skinny (M <= 64) i4i4_gemm / w4a8_gemm call would use on a GPU with
    `sms` SMs and room for `pairs` / `quads` clusters of two / four (host only)."""
    out = (ctypes.c_int * 4)()
    v = {"i4i4": 0, "w4a8": 1}[variant]
    _check(load().igemm_skinny_plan(v, M, N, K, sms, pairs, quads, out), "igemm_skinny_plan")
    return {"split": out[0], "slice_k": out[1], "ctas": out[2], "cluster": out[3]}


ROUTES = ("skinny", "small", "codes", "in-kernel", "packed")


def igemm_route(variant: str, M: int, N: int, K: int, sms: int = 152, pairs: int = 76, quads: int = 36) -> str:
    """The path an i4i4_gemm / w4a8_gemm call of this shape takes on a GPU with `sms`
    SMs and room for `pairs` / `quads` skinny clusters (host only)."""
    out = ctypes.c_int()
    v = {"i4i4": 0, "w4a8": 1}[variant]
    _check(load().igemm_route(v, M, N, K, sms, pairs, quads, ctypes.byref(out)), "igemm_route")
    return ROUTES[out.value]


def igemm_ss_plan(variant: str, M: int, N: int, K: int, clusters: int) -> dict:
    """The prepared-codes kernel's plan for an i4i4_gemm / w4a8_gemm call on a GPU
    where `clusters` CTA pairs fit, with the host check of its coverage (host only)."""
    out = (ctypes.c_int * 7)()
    v = {"i4i4": 0, "w4a8": 1}[variant]
    _check(load().igemm_ss_plan(v, M, N, K, clusters, out), "igemm_ss_plan")
    return {"split": out[0], "kb_per_split": out[1], "units": out[2], "tail_tiles": out[3],
            "tail_kb": out[4], "clusters": out[5], "covered": bool(out[6])}


def igemm_kernels_launched() -> int:
    """Kernels this library has enqueued in this process so far."""
    return int(load().igemm_kernels_launched())


def igemm_watchdog_selftest(limit_us: int, stream=None) -> None:
    _check(load().igemm_watchdog_selftest(limit_us, _stream(stream)), "igemm_watchdog_selftest")
