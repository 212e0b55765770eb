"""ctypes binding of libswiglu_b200.so (the C ABI of include/swiglu.h).

Argument marshalling only: torch tensors become device pointers and the
current CUDA stream becomes a cudaStream_t; the library does all the work.
The library is loaded on first use; if it is missing or cannot be loaded the
call raises -- there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libswiglu_b200.so")

# enum swiglu_dtype
SWIGLU_BF16 = 0
SWIGLU_FP32 = 1
# enum swiglu_status
SWIGLU_OK = 0
SWIGLU_ERR_NULL_POINTER = 1
SWIGLU_ERR_BAD_DIM = 2
SWIGLU_ERR_MISALIGNED_DIM = 3
SWIGLU_ERR_MISALIGNED_PTR = 4
SWIGLU_ERR_BAD_DTYPE = 5
SWIGLU_ERR_UNSUPPORTED_DEVICE = 6
SWIGLU_ERR_CUDA = 7
SWIGLU_ERR_TIMEOUT = 8
SWIGLU_ERR_OVERLAP = 9
SWIGLU_ERR_NO_DEVICE = 10
SWIGLU_ERR_BAD_FLAGS = 11
SWIGLU_ERR_BAD_EPILOGUE = 12
SWIGLU_ERR_BAD_BLOCK = 13
SWIGLU_ERR_WORKSPACE = 14
# enum swiglu_block
SWIGLU_BLOCK_ROW = 0
SWIGLU_BLOCK_TILE = 1
# enum swiglu_activation
SWIGLU_ACT_SILU = 0
SWIGLU_ACT_GELU_TANH = 1
# enum swiglu_flags
SWIGLU_FLAG_WEIGHTS_STABLE = 1
# enum swiglu_route
ROUTE_NONE = 0
ROUTE_ZERO_K = 1
ROUTE_DECODE_BF16 = 2
ROUTE_GEMM_BF16 = 3
ROUTE_GEMM_TF32X3 = 4
ROUTE_BWD_GEMM_BF16 = 5
ROUTE_BWD_GEMM_TF32X3 = 6
ROUTE_STREAM_TC_BF16 = 7

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int


class Epilogue(ctypes.Structure):
    """struct swiglu_epilogue."""
    _fields_ = [("activation", ctypes.c_int), ("gate_multiplier", ctypes.c_float),
                ("G", ctypes.c_void_p), ("U", ctypes.c_void_p)]


class BlockNormParams(ctypes.Structure):
    """struct swiglu_block_norm_params."""
    _fields_ = [("post_weight", ctypes.c_void_p), ("pre_weight", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("gate_rows", ctypes.c_int64),
                ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float)]


_NORM = ctypes.POINTER(BlockNormParams)

# name -> (restype, argtypes), mirroring include/swiglu.h
SIGNATURES = {
    "swiglu_fwd": (_I, [_P, _P, _P, _P, _I64, _I64, _I64, _I, _P]),
    "swiglu_fwd_ex": (_I, [_P, _P, _P, _P, _I64, _I64, _I64, _I, ctypes.c_uint, _P]),
    "swiglu_fwd_epilogue": (_I, [_P, _P, _P, _P, _I64, _I64, _I64, _I, ctypes.POINTER(Epilogue),
                                 ctypes.c_uint, _P]),
    "dswiglu_bwd_epilogue": (_I, [_P, _P, _P, _P, _P, _I64, _I, _I, ctypes.c_float, _P]),
    "dswiglu_bwd": (_I, [_P, _P, _P, _P, _P, _I64, _P]),
    "dswiglu_bwd_dtype": (_I, [_P, _P, _P, _P, _P, _I64, _I, _P]),
    "swiglu_fwd_fp8": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, ctypes.POINTER(Epilogue), _P]),
    "swiglu_bwd_dx": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P]),
    "swiglu_bwd_dx_noalloc": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P]),
    "swiglu_bwd_dw": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P]),
    "swiglu_bwd_gemms": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P]),
    "swiglu_quant_b128": (_I, [_P, _P, _P, _I64, _I64, _I, _I, _I, _P]),
    "swiglu_gemm_b128": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _P]),
    "swiglu_fwd_b128": (_I, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, ctypes.POINTER(Epilogue),
                             _P]),
    "swiglu_block_norm": (_I, [_P, _P, _NORM, _P, _P, _P, _P, _I64, _I64, _I, _P]),
    "swiglu_block_norm_bwd_workspace": (_I64, [_NORM, _I64, _I64, _I]),
    "swiglu_block_norm_bwd": (_I, [_P, _P, _P, _P, _P, _P, _NORM, _P, _P, _P, _P, _P, _P, _I64, _I64,
                                   _I64, _I, _P]),
    "swiglu_route_for": (_I, [_I64, _I64, _I64, _I]),
    "swiglu_last_route": (_I, []),
    "swiglu_status_string": (ctypes.c_char_p, [_I]),
    "swiglu_sync_status": (_I, [_P]),
    "swiglu_read_floor": (_I, [_P, _P, _I64, _P, _P]),
    "swiglu_selftest_wait_timeout": (_I, [_P]),
    "swiglu_read_floor_sink_words": (_I64, []),
}

_lock = threading.Lock()
_lib = None


class SwigluError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m up_projection_b200.build` (nvcc, sm_100a)")
            handle = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(handle, name)
                f.restype = res
                f.argtypes = args
            _lib = handle
            _bind(handle)
    return _lib


# csrc/binding.cpp: the calls of the operators around the projection that are in
# order, done natively (None: not built, built for another torch, or not loaded
# yet).  A native call returns None for what it leaves to the functions below.
_native = None


def _bind(handle):
    global _native
    try:
        from . import _binding
        from .build import binding_stamp
    except ImportError:
        return
    if getattr(_binding, "built_for", None) != binding_stamp():
        return  # its inlined tensor code is another torch's
    _binding.bind(*(ctypes.cast(getattr(handle, n), ctypes.c_void_p).value for n in (
        "swiglu_block_norm", "swiglu_block_norm_bwd_workspace", "swiglu_block_norm_bwd",
        "swiglu_quant_b128", "swiglu_gemm_b128", "swiglu_fwd_b128")))
    _native = _binding


def status_string(status: int) -> str:
    return lib().swiglu_status_string(int(status)).decode()


# (the raw handle of the current stream and the current device, without the
# Stream object torch.cuda.current_stream() builds: 3 us less per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_raw_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _drawn(stream, *tensors) -> int:
    """The call's stream as a handle, after outputs and scratch were drawn on
    the current one.  Another stream first waits for what may still use their
    memory there, and keeps it until its own work is done.  (Not where one of
    the two captures: its memory is the graph's, and waiting would draw the
    other in.)"""
    s = _stream(stream)
    if stream is None:
        return s
    current = torch.cuda.current_stream()
    if s != current.cuda_stream:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(s) if s else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            captures = torch.cuda.is_current_stream_capturing()
        if captures == torch.cuda.is_current_stream_capturing():
            stream.wait_stream(current)
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    return s


def _check(fn: str, st: int):
    if st != SWIGLU_OK:
        raise SwigluError(fn, st)


_DT = {torch.bfloat16: SWIGLU_BF16, torch.float32: SWIGLU_FP32}


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}; use bfloat16 or float32")
    return _DT[t.dtype]


def _dev(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def swiglu_fwd(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor,
               H: torch.Tensor | None = None, stream=None,
               weights_stable: bool = False, activation: int = SWIGLU_ACT_SILU,
               gate_multiplier: float = 1.0, return_gu: bool = False):
    """H = silu(X Wg^T) * (X Wu^T) through the C ABI.  X [..., K] (leading
    dims are flattened to M rows, as the TensorRT-LLM fused up-projection
    does), Wg/Wu [N, K]; bf16 or fp32, all contiguous on one GPU.

    weights_stable=True promises that no earlier work on the stream writes
    Wg or Wu (SWIGLU_FLAG_WEIGHTS_STABLE): the weight-streaming kernels (bf16
    decode at M <= 8, the tcgen05 stream at 9 <= M <= 128) may then start
    streaming them while the preceding kernel finishes.

    activation / gate_multiplier select the epilogue variant
    H = act(gate_multiplier * G) * U (SWIGLU_ACT_SILU or
    SWIGLU_ACT_GELU_TANH).  return_gu=True also stores G = X Wg^T and
    U = X Wu^T (training forward) and returns (H, G, U)."""
    # (the checks are ordered for the per-call cost of the decode path: one
    # pass of cheap attribute reads, the detailed messages only on failure)
    if not (X.is_cuda and Wg.is_cuda and Wu.is_cuda and X.is_contiguous()
            and Wg.is_contiguous() and Wu.is_contiguous()):
        for t, n in ((X, "X"), (Wg, "Wg"), (Wu, "Wu")):
            _dev(t, n)
    dt = X.dtype
    if Wg.dtype != dt or Wu.dtype != dt:
        raise TypeError("X, Wg and Wu must share a dtype")
    code = _DT.get(dt)
    if code is None:
        _dtype_code(X)
    xs = X.shape
    K = xs[-1]
    ws = Wg.shape
    N = ws[0]
    if len(ws) != 2 or ws[1] != K or Wu.shape != ws:
        raise ValueError(f"weights must be [N, K] = [{N}, {K}]")
    M = X.numel() // K if K else math.prod(xs[:-1])
    if H is None:
        H = torch.empty((*xs[:-1], N), dtype=dt, device=X.device)
    elif not (H.is_cuda and H.is_contiguous()):
        _dev(H, "H")
    elif H.dtype != dt or H.numel() != M * N:
        raise ValueError("H has the wrong dtype or size")
    flags = SWIGLU_FLAG_WEIGHTS_STABLE if weights_stable else 0
    G = U = None
    if return_gu:
        G = torch.empty_like(H)
        U = torch.empty_like(H)
    if activation == SWIGLU_ACT_SILU and gate_multiplier == 1.0 and not return_gu:
        st = lib().swiglu_fwd_ex(X.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), H.data_ptr(),
                                 M, K, N, code, flags, _stream(stream))
    else:
        epi = Epilogue(int(activation), float(gate_multiplier),
                       G.data_ptr() if G is not None else None,
                       U.data_ptr() if U is not None else None)
        st = lib().swiglu_fwd_epilogue(X.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), H.data_ptr(),
                                       M, K, N, code, ctypes.byref(epi), flags,
                                       _stream(stream))
    _check("swiglu_fwd", st)
    return (H, G, U) if return_gu else H


def dswiglu_bwd(dH: torch.Tensor, G: torch.Tensor, U: torch.Tensor,
                dG: torch.Tensor | None = None, dU: torch.Tensor | None = None,
                stream=None, activation: int = SWIGLU_ACT_SILU, gate_multiplier: float = 1.0):
    """(dG, dU) of h = act(gate_multiplier g) * u through the C ABI (bf16 or
    fp32); the defaults are the plain dSwiGLU."""
    for t, n in ((dH, "dH"), (G, "G"), (U, "U")):
        _dev(t, n)
    if not (dH.dtype == G.dtype == U.dtype) or dH.shape != G.shape or G.shape != U.shape:
        raise ValueError("dH, G, U must share dtype and shape")
    dG = torch.empty_like(G) if dG is None else dG
    dU = torch.empty_like(U) if dU is None else dU
    _dev(dG, "dG")
    _dev(dU, "dU")
    st = lib().dswiglu_bwd_epilogue(dH.data_ptr(), G.data_ptr(), U.data_ptr(), dG.data_ptr(),
                                    dU.data_ptr(), G.numel(), _dtype_code(G), int(activation),
                                    float(gate_multiplier), _stream(stream))
    _check("dswiglu_bwd", st)
    return dG, dU


def swiglu_fwd_fp8(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, stream=None,
                   activation: int = SWIGLU_ACT_SILU, gate_multiplier: float = 1.0):
    """Quantised forward through the C ABI: returns (Hq, Hs) with Hq the
    e4m3 codes [..., N] (torch.uint8) and Hs the UE8M0 scale codes
    [..., ceil(N/32)] (torch.uint8) of H = act(gate_multiplier G) U; the
    value of element n is e4m3(Hq) * 2^(Hs[n // 32] - 127).  bf16 inputs."""
    for t, n in ((X, "X"), (Wg, "Wg"), (Wu, "Wu")):
        _dev(t, n)
    if not (X.dtype == Wg.dtype == Wu.dtype == torch.bfloat16):
        raise TypeError("swiglu_fwd_fp8 takes bfloat16 X, Wg, Wu")
    K = X.shape[-1]
    N = Wg.shape[0]
    if Wg.shape != (N, K) or Wu.shape != (N, K):
        raise ValueError(f"weights must be [N, K] = [{N}, {K}]")
    lead = X.shape[:-1]
    M = 1
    for d in lead:
        M *= d
    Hq = torch.empty((*lead, N), dtype=torch.uint8, device=X.device)
    Hs = torch.empty((*lead, (N + 31) // 32), dtype=torch.uint8, device=X.device)
    epi = Epilogue(int(activation), float(gate_multiplier), None, None)
    st = lib().swiglu_fwd_fp8(X.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), Hq.data_ptr(),
                              Hs.data_ptr(), M, K, N, ctypes.byref(epi), _stream(stream))
    _check("swiglu_fwd_fp8", st)
    return Hq, Hs


def _bwd_shapes(dG, dU, name_w, W):
    for t, n in ((dG, "dG"), (dU, "dU"), (W, name_w)):
        _dev(t, n)
    if not (dG.dtype == dU.dtype == W.dtype) or dG.dtype not in _DT:
        raise TypeError("the backward GEMMs take bfloat16 or float32 tensors of one dtype")
    if dG.shape != dU.shape:
        raise ValueError("dG and dU must have the same shape")
    N = dG.shape[-1]
    M = 1
    for d in dG.shape[:-1]:
        M *= d
    return M, N


def swiglu_bwd_dx(dG: torch.Tensor, dU: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor,
                  dX: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dX = dG Wg + dU Wu through the C ABI (bf16, or fp32 by 3xTF32).  dG, dU [..., N] (leading
    dims flattened to M rows), Wg, Wu [N, K]; dX has dG's leading dims."""
    M, N = _bwd_shapes(dG, dU, "Wg", Wg)
    _dev(Wu, "Wu")
    K = Wg.shape[-1]
    if Wg.shape != (N, K) or Wu.shape != (N, K) or Wu.dtype != Wg.dtype:
        raise ValueError(f"weights must be [N, K] = [{N}, {K}] of dG's dtype")
    if dX is None:
        dX = torch.empty((*dG.shape[:-1], K), dtype=dG.dtype, device=dG.device)
    else:
        _dev(dX, "dX")
        if dX.dtype != dG.dtype or dX.numel() != M * K:
            raise ValueError("dX has the wrong dtype or size")
    st = lib().swiglu_bwd_dx(dG.data_ptr(), dU.data_ptr(), Wg.data_ptr(), Wu.data_ptr(),
                             dX.data_ptr(), M, K, N, _dtype_code(dG), _stream(stream))
    _check("swiglu_bwd_dx", st)
    return dX


def swiglu_bwd_dw(dG: torch.Tensor, dU: torch.Tensor, X: torch.Tensor,
                  dWg: torch.Tensor | None = None, dWu: torch.Tensor | None = None,
                  stream=None):
    """(dWg, dWu) = (dG^T X, dU^T X) through the C ABI (bf16, or fp32 by 3xTF32).  dG, dU
    [..., N] and X [..., K] with the same leading dims (M rows)."""
    M, N = _bwd_shapes(dG, dU, "X", X)
    K = X.shape[-1]
    if X.numel() != M * K:
        raise ValueError("X must have dG's leading dims")
    dWg = torch.empty((N, K), dtype=X.dtype, device=X.device) if dWg is None else dWg
    dWu = torch.empty((N, K), dtype=X.dtype, device=X.device) if dWu is None else dWu
    for t, n in ((dWg, "dWg"), (dWu, "dWu")):
        _dev(t, n)
        if t.dtype != X.dtype or t.numel() != N * K:
            raise ValueError(f"{n} has the wrong dtype or size")
    st = lib().swiglu_bwd_dw(dG.data_ptr(), dU.data_ptr(), X.data_ptr(), dWg.data_ptr(),
                             dWu.data_ptr(), M, K, N, _dtype_code(dG), _stream(stream))
    _check("swiglu_bwd_dw", st)
    return dWg, dWu


def swiglu_bwd_gemms(dG: torch.Tensor, dU: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor,
                     X: torch.Tensor, stream=None):
    """(dX, dWg, dWu) of the projection in one call (bf16 or fp32; for fp32
    one balanced launch runs all three GEMMs)."""
    M, N = _bwd_shapes(dG, dU, "Wg", Wg)
    for t, n in ((Wu, "Wu"), (X, "X")):
        _dev(t, n)
    K = Wg.shape[-1]
    if Wg.shape != (N, K) or Wu.shape != (N, K) or X.shape[-1] != K or X.numel() != M * K:
        raise ValueError("shapes: dG, dU [.., N], Wg, Wu [N, K], X [.., K] with dG's leading dims")
    if not (Wu.dtype == X.dtype == dG.dtype):
        raise TypeError("all tensors must share one dtype")
    dX = torch.empty((*dG.shape[:-1], K), dtype=dG.dtype, device=dG.device)
    dWg = torch.empty((N, K), dtype=dG.dtype, device=dG.device)
    dWu = torch.empty((N, K), dtype=dG.dtype, device=dG.device)
    st = lib().swiglu_bwd_gemms(dG.data_ptr(), dU.data_ptr(), Wg.data_ptr(), Wu.data_ptr(),
                                X.data_ptr(), dX.data_ptr(), dWg.data_ptr(), dWu.data_ptr(),
                                M, K, N, _dtype_code(dG), _stream(stream))
    _check("swiglu_bwd_gemms", st)
    return dX, dWg, dWu


def _here(*tensors):
    """All on the current device, whose stream and kernels the call uses."""
    i = _raw_device()
    for t in tensors:
        if t is not None and t.get_device() != i:
            raise ValueError(f"all tensors must be on the current device (cuda:{i})")


def _device_of(t: torch.Tensor, name: str) -> int:
    """The current device, which the contiguous tensor t is on."""
    dev = t.get_device()
    if dev < 0 or not t.is_contiguous():
        _dev(t, name)
    if dev != _raw_device():
        _here(t)
    return dev


def _fits(t: torch.Tensor, device: int, dtype: torch.dtype, shape) -> bool:
    """One cheap pass over what every operand needs (messages only on failure)."""
    return t.get_device() == device and t.dtype is dtype and t.shape == shape and t.is_contiguous()


def _codes(t: torch.Tensor, name: str, device: int):
    if t.get_device() != device or not t.is_contiguous():
        _dev(t, name)
        _here(t)
    if t.dtype is not torch.uint8 and t.dtype is not torch.float8_e4m3fn:
        raise TypeError(f"{name} must hold e4m3 codes (uint8 or float8_e4m3fn)")


def _row_scales(s: torch.Tensor, name: str, rows: int, kb: int, device: int):
    """The 1 x 128 scales [rows, kb], stored [kb, rows padded to 4]."""
    if s.get_device() != device or s.dtype is not torch.float32 or s.shape != (rows, kb):
        if s.is_cuda:
            _here(s)
        raise ValueError(f"{name} must be a float32 CUDA tensor [{rows}, {kb}]")
    if rows and kb and ((rows > 1 and s.stride(0) != 1) or
                        (kb > 1 and s.stride(1) != (rows + 3) // 4 * 4)):
        raise ValueError(f"{name} must be stored with its rows innermost, padded to a multiple of "
                         "4 (as swiglu_quant_b128 returns it)")


def swiglu_quant_b128(X: torch.Tensor, block: str = "row", transpose: bool = False, stream=None):
    """e4m3 codes and fp32 power-of-two scales of X [..., C] (leading dims
    flattened to R rows; bf16 or fp32; C a multiple of 16) in blocks of 128:
    block "row" (1 x 128) or "tile" (128 x 128).  Returns (Q, S): Q torch.uint8
    codes of X's shape, S [R, ceil(C/128)] ("row", rows innermost in memory) or
    [ceil(R/128), ceil(C/128)].  transpose=True quantises X^T instead, blocks
    along R: Q [C, R rounded up to 16] with zero codes behind R, S
    [C, ceil(R/128)] or [ceil(C/128), ceil(R/128)]."""
    tile = block == "tile"
    if not tile and block != "row":
        raise ValueError('block must be "row" or "tile"')
    if stream is None and _native is not None:
        r = _native.quant_b128(X, tile, transpose)
        if r is not None:
            if type(r) is int:
                _check("swiglu_quant_b128", r)
            return r
    if not (X.is_cuda and X.is_contiguous()):
        _dev(X, "X")
    code = _DT.get(X.dtype)
    if code is None:
        _dtype_code(X)
    _here(X)
    shape = X.shape
    C = shape[-1]
    R = X.numel() // C if C else math.prod(shape[:-1])
    rows, cols = (C, (R + 15) // 16 * 16) if transpose else (R, C)
    Q = X.new_empty((rows, cols) if transpose else shape, dtype=torch.uint8)
    kb = (cols + 127) // 128
    if tile:
        S = X.new_empty(((rows + 127) // 128, kb), dtype=torch.float32)
    elif rows & 3 or not kb:
        S = X.new_empty((kb, (rows + 3) // 4 * 4), dtype=torch.float32)[:, :rows].t()
    else:
        S = X.new_empty_strided((rows, kb), (1, rows), dtype=torch.float32)
    st = lib().swiglu_quant_b128(X.data_ptr(), Q.data_ptr(), S.data_ptr(), R, C, code,
                                 1 if tile else 0, 1 if transpose else 0, _drawn(stream, Q, S))
    if st:
        _check("swiglu_quant_b128", st)
    return Q, S


def swiglu_gemm_b128(A: torch.Tensor, As: torch.Tensor, B: torch.Tensor, Bs: torch.Tensor,
                     out_dtype: torch.dtype = torch.bfloat16, Y: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Y = A B^T of block-scaled e4m3 operands (swiglu_quant_b128 makes them):
    A [..., K] codes with 1 x 128 scales As [M, KB], B [N, K] codes with scales
    Bs [ceil(N/128), KB] (128 x 128 blocks) or [N, KB] (1 x 128, rows innermost
    in memory); KB = ceil(K/128), K a multiple of 16, N of 8.  Y bf16 or fp32
    with A's leading dims."""
    if stream is None and _native is not None and (out_dtype is torch.bfloat16 or out_dtype is torch.float32):
        r = _native.gemm_b128(A, As, B, Bs, out_dtype is torch.float32, Y)
        if r is not None:
            if type(r) is int:
                _check("swiglu_gemm_b128", r)
            return r
    dev = _device_of(A, "A")
    _codes(A, "A", dev)
    _codes(B, "B", dev)
    shape = A.shape
    K = shape[-1]
    M = shape[0] if len(shape) == 2 else math.prod(shape[:-1])
    N = B.shape[0]
    if B.shape != (N, K):
        raise ValueError(f"B must be [N, K] = [{N}, {K}]")
    kb = (K + 127) // 128
    _row_scales(As, "As", M, kb, dev)
    tiles = ((N + 127) // 128, kb)
    if Bs.shape == tiles:
        block = SWIGLU_BLOCK_TILE
        if not _fits(Bs, dev, torch.float32, tiles):
            _refuse(Bs, "Bs", f"float32 [{tiles[0]}, {kb}]")
    else:
        block = SWIGLU_BLOCK_ROW
        _row_scales(Bs, "Bs", N, kb, dev)
    code = _DT.get(out_dtype)
    if code is None:
        raise TypeError(f"unsupported out_dtype {out_dtype}; use bfloat16 or float32")
    drawn = None
    if Y is None:
        Y = drawn = A.new_empty((M, N) if len(shape) == 2 else (*shape[:-1], N), dtype=out_dtype)
    else:
        _dev(Y, "Y")
        _here(Y)
        if Y.dtype != out_dtype or Y.numel() != M * N:
            raise ValueError("Y has the wrong dtype or size")
    st = lib().swiglu_gemm_b128(A.data_ptr(), As.data_ptr(), B.data_ptr(), Bs.data_ptr(),
                                Y.data_ptr(), M, N, K, block, code, _drawn(stream, drawn))
    if st:
        _check("swiglu_gemm_b128", st)
    return Y


def swiglu_fwd_b128(X: torch.Tensor, Xs: torch.Tensor, Wg: torch.Tensor, Wgs: torch.Tensor,
                    Wu: torch.Tensor, Wus: torch.Tensor, H: torch.Tensor | None = None, stream=None,
                    activation: int = SWIGLU_ACT_SILU, gate_multiplier: float = 1.0,
                    return_gu: bool = False):
    """swiglu_fwd on block-scaled e4m3 operands: X [..., K] codes with 1 x 128
    scales Xs [M, KB], Wg, Wu [N, K] codes with 128 x 128 scales
    [ceil(N/128), KB].  Returns H bf16 [..., N], or (H, G, U)."""
    if stream is None and _native is not None:
        r = _native.fwd_b128(X, Xs, Wg, Wgs, Wu, Wus, H, activation, gate_multiplier, return_gu)
        if r is not None:
            if type(r) is int:
                _check("swiglu_fwd_b128", r)
            return r
    dev = _device_of(X, "X")
    _codes(X, "X", dev)
    _codes(Wg, "Wg", dev)
    _codes(Wu, "Wu", dev)
    shape = X.shape
    K = shape[-1]
    M = shape[0] if len(shape) == 2 else math.prod(shape[:-1])
    w = Wg.shape
    N = w[0]
    if w != (N, K) or Wu.shape != w:
        raise ValueError(f"weights must be [N, K] = [{N}, {K}]")
    kb = (K + 127) // 128
    _row_scales(Xs, "Xs", M, kb, dev)
    tiles = ((N + 127) // 128, kb)
    if not _fits(Wgs, dev, torch.float32, tiles):
        _refuse(Wgs, "Wgs", f"float32 [{tiles[0]}, {kb}]")
    if not _fits(Wus, dev, torch.float32, tiles):
        _refuse(Wus, "Wus", f"float32 [{tiles[0]}, {kb}]")
    drawn = None
    if H is None:
        H = drawn = X.new_empty((M, N) if len(shape) == 2 else (*shape[:-1], N), dtype=torch.bfloat16)
    else:
        _dev(H, "H")
        _here(H)
        if H.dtype != torch.bfloat16 or H.numel() != M * N:
            raise ValueError("H has the wrong dtype or size")
    G = U = epi = None   # (no epilogue: silu, multiplier 1, neither G nor U)
    if return_gu:
        G = torch.empty_like(H)
        U = torch.empty_like(H)
    if return_gu or activation != SWIGLU_ACT_SILU or gate_multiplier != 1.0:
        epi = ctypes.byref(Epilogue(int(activation), float(gate_multiplier),
                                    G.data_ptr() if return_gu else None, U.data_ptr() if return_gu else None))
    st = lib().swiglu_fwd_b128(X.data_ptr(), Xs.data_ptr(), Wg.data_ptr(), Wgs.data_ptr(),
                               Wu.data_ptr(), Wus.data_ptr(), H.data_ptr(), M, K, N, epi,
                               _drawn(stream, drawn, G, U))
    if st:
        _check("swiglu_fwd_b128", st)
    return (H, G, U) if return_gu else H


def _refuse(t: torch.Tensor, name: str, what: str):
    """What _fits found wrong with an operand."""
    _dev(t, name)
    _here(t)
    raise ValueError(f"{name} must be {what}")


def _norm_params(dev, dt, D, post_weight, pre_weight, gate, residual_scale, eps):
    """The checked parameter struct of the block norm calls."""
    w1 = w2 = g = None
    rows = 1
    if post_weight is not None:
        if not _fits(post_weight, dev, dt, (D,)):
            _refuse(post_weight, "post_weight", f"[{D}] of Y's dtype")
        w1 = post_weight.data_ptr()
    if pre_weight is not None:
        if not _fits(pre_weight, dev, dt, (D,)):
            _refuse(pre_weight, "pre_weight", f"[{D}] of Y's dtype")
        w2 = pre_weight.data_ptr()
    if gate is not None:
        if gate.dim() == 2:
            rows = gate.shape[0]
            ok = rows > 0 and _fits(gate, dev, dt, (rows, D))
        else:
            ok = _fits(gate, dev, dt, (D,))
        if not ok:
            _refuse(gate, "gate", f"[{D}] or [rows, {D}] of Y's dtype, with a row at least")
        g = gate.data_ptr()
    return BlockNormParams(w1, w2, g, rows, residual_scale, eps)


def _norm_shape(Y):
    """Device, dtype, its code, M and D of a block norm's Y."""
    dev = _device_of(Y, "Y")
    dt = Y.dtype
    code = _DT.get(dt)
    if code is None:
        _dtype_code(Y)
    shape = Y.shape
    D = shape[-1]
    return dev, dt, code, shape, Y.numel() // D if D else 0, D


def swiglu_block_norm(Y: torch.Tensor, R: torch.Tensor, post_weight: torch.Tensor | None = None,
                      pre_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                      residual_scale: float = 1.0, eps: float = 1e-6, return_stats: bool = False,
                      Rn: torch.Tensor | None = None, stream=None):
    """The boundary between two blocks in one pass, for rows of D elements:
    P = post_weight * Y / rms(Y), Rn = R + residual_scale * gate * P,
    N = pre_weight * Rn / rms(Rn), rms(x) = sqrt(mean(x^2) + eps).  Y is the
    block's output and R the residual stream [..., D] (bf16 or fp32).  Without
    post_weight P = Y; without pre_weight N is None; gate is [D], or
    [rows, D] with rows dividing the number of rows M (row m uses gate row
    m // (M / rows)).  Returns (Rn, N), with return_stats=True (training)
    (Rn, N, rstd_post, rstd_pre), fp32 [M], for swiglu_block_norm_bwd.  Rn may
    be given as the output buffer, R itself included (in place)."""
    if stream is None and _native is not None:
        r = _native.block_norm(Y, R, post_weight, pre_weight, gate, residual_scale, eps, return_stats, Rn)
        if r is not None:
            if type(r) is int:
                _check("swiglu_block_norm", r)
            return r
    dev, dt, code, shape, M, D = _norm_shape(Y)
    if not _fits(R, dev, dt, shape):
        _refuse(R, "R", "of Y's dtype and shape")
    p = _norm_params(dev, dt, D, post_weight, pre_weight, gate, residual_scale, eps)
    drawn = None
    if Rn is None:
        Rn = drawn = torch.empty_like(R)
    elif not _fits(Rn, dev, dt, shape):
        _refuse(Rn, "Rn", "of Y's dtype and shape")
    N = torch.empty_like(Y) if pre_weight is not None else None
    r1 = r2 = None
    if return_stats:
        if post_weight is not None:
            r1 = Y.new_empty((M,), dtype=torch.float32)
        if pre_weight is not None:
            r2 = Y.new_empty((M,), dtype=torch.float32)
    st = lib().swiglu_block_norm(Y.data_ptr(), R.data_ptr(), ctypes.byref(p), Rn.data_ptr(),
                                 N.data_ptr() if N is not None else None,
                                 r1.data_ptr() if r1 is not None else None,
                                 r2.data_ptr() if r2 is not None else None, M, D, code,
                                 _drawn(stream, drawn, N, r1, r2))
    if st:
        _check("swiglu_block_norm", st)
    return (Rn, N, r1, r2) if return_stats else (Rn, N)


def _stat(t, name, dev, M):
    """Address of a row statistic the backward reads."""
    if t is None:
        raise ValueError(f"{name} is missing")
    if not _fits(t, dev, torch.float32, (M,)):
        _refuse(t, name, f"float32 [{M}]")
    return t.data_ptr()


def swiglu_block_norm_bwd(dRn: torch.Tensor | None, dN: torch.Tensor | None, Y: torch.Tensor,
                          Rn: torch.Tensor, rstd_post: torch.Tensor | None,
                          rstd_pre: torch.Tensor | None, post_weight: torch.Tensor | None = None,
                          pre_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                          residual_scale: float = 1.0, stream=None):
    """Gradients of swiglu_block_norm's Rn and N: returns (dY, dR, d_post,
    d_pre, d_gate), the last three None without their parameter (d_gate has
    gate's shape).  dRn or dN may be None for zero (dN only without
    pre_weight); Rn, rstd_post, rstd_pre as the forward returned them."""
    if stream is None and _native is not None:
        r = _native.block_norm_bwd(dRn, dN, Y, Rn, rstd_post, rstd_pre, post_weight, pre_weight, gate,
                                   residual_scale)
        if r is not None:
            if type(r) is int:
                _check("swiglu_block_norm_bwd", r)
            return r
    dev, dt, code, shape, M, D = _norm_shape(Y)
    if (dN is None) != (pre_weight is None):
        raise ValueError("dN and pre_weight go together")
    pR = pN = p1 = p2 = d1 = d2 = dgp = dw1 = dw2 = dg = ws = wsp = None
    if not _fits(Rn, dev, dt, shape):
        _refuse(Rn, "Rn", "of Y's dtype and shape")
    if dRn is not None:
        if not _fits(dRn, dev, dt, shape):
            _refuse(dRn, "dRn", "of Y's dtype and shape")
        pR = dRn.data_ptr()
    if dN is not None:
        if not _fits(dN, dev, dt, shape):
            _refuse(dN, "dN", "of Y's dtype and shape")
        pN = dN.data_ptr()
    p = _norm_params(dev, dt, D, post_weight, pre_weight, gate, residual_scale, 0.0)
    if post_weight is not None:
        p1 = _stat(rstd_post, "rstd_post", dev, M)
        dw1 = torch.empty_like(post_weight)
        d1 = dw1.data_ptr()
    if pre_weight is not None:
        p2 = _stat(rstd_pre, "rstd_pre", dev, M)
        dw2 = torch.empty_like(pre_weight)
        d2 = dw2.data_ptr()
    if gate is not None:
        dg = torch.empty_like(gate)
        dgp = dg.data_ptr()
    dY = torch.empty_like(Y)
    dR = torch.empty_like(Y)
    c = lib()
    ref = ctypes.byref(p)
    need = c.swiglu_block_norm_bwd_workspace(ref, M, D, code)
    if need > 0:
        ws = Y.new_empty((need,), dtype=torch.uint8)
        wsp = ws.data_ptr()
    else:
        need = 0
    st = c.swiglu_block_norm_bwd(pR, pN, Y.data_ptr(), Rn.data_ptr(), p1, p2, ref, dY.data_ptr(),
                                 dR.data_ptr(), d1, d2, dgp, wsp, need, M, D, code,
                                 _drawn(stream, dY, dR, dw1, dw2, dg, ws))
    if st:
        _check("swiglu_block_norm_bwd", st)
    return dY, dR, dw1, dw2, dg


def swiglu_route_for(M: int, K: int, N: int, dtype: int) -> int:
    return lib().swiglu_route_for(M, K, N, dtype)


def swiglu_last_route() -> int:
    return lib().swiglu_last_route()


def swiglu_sync_status(stream=None) -> int:
    return lib().swiglu_sync_status(_stream(stream))


def swiglu_read_floor(A: torch.Tensor, B: torch.Tensor, sink: torch.Tensor,
                      stream=None) -> None:
    """Bench-only: stream-read A and B (same byte size) once."""
    _dev(A, "A")
    _dev(B, "B")
    nbytes = A.numel() * A.element_size()
    if B.numel() * B.element_size() != nbytes:
        raise ValueError("A and B must have the same size in bytes")
    st = lib().swiglu_read_floor(A.data_ptr(), B.data_ptr(), nbytes, sink.data_ptr(),
                                 _stream(stream))
    _check("swiglu_read_floor", st)
