"""Host side of the operators around the projection (block norms, e4m3
quantisation in blocks of 128, block-scaled products): argument checks of the
C entry points and the launch plans, without a GPU."""
import ctypes

import pytest
import torch

import up_projection_b200 as up
from test_host_plans import _build_and_run
from up_projection_b200 import _capi

A = [(i + 1) << 24 for i in range(16)]   # distinct, aligned, far apart
NULL, DIM, MDIM, MPTR, DTYPE, OVER, EPI, BLOCK = (
    _capi.SWIGLU_ERR_NULL_POINTER, _capi.SWIGLU_ERR_BAD_DIM, _capi.SWIGLU_ERR_MISALIGNED_DIM,
    _capi.SWIGLU_ERR_MISALIGNED_PTR, _capi.SWIGLU_ERR_BAD_DTYPE, _capi.SWIGLU_ERR_OVERLAP,
    _capi.SWIGLU_ERR_BAD_EPILOGUE, _capi.SWIGLU_ERR_BAD_BLOCK)


def test_product_plans_keep_memory_bounds():
    """Shared memory, TMA boxes, TMEM columns and tiles of the block-scaled
    products' plans, many rows and few (gemm_b128_plan_check.cu,
    gemm_b128_stream_plan_check.cu)."""
    csrc = "up_projection_b200/csrc/"
    _build_and_run(["tests/gemm_b128_plan_check.cu", csrc + "gemm_b128_stream.cu", csrc + "tmap.cu"], 100000)
    _build_and_run(["tests/gemm_b128_stream_plan_check.cu", csrc + "tmap.cu"], 100000)


def test_norm_ring_plans_keep_memory_bounds():
    """Row rings, sums and items of the block norms (block_norm_plan_check.cu)."""
    _build_and_run(["tests/block_norm_plan_check.cu"], 20000)


# swiglu_quant_b128(X, Q, S, R, C, dtype, block, transpose)
@pytest.mark.parametrize("args,code", [
    ((A[0], A[1], A[2], 4, 64, 2, 0, 0), DTYPE),
    ((A[0], A[1], A[2], 4, 64, 0, 2, 0), BLOCK),
    ((A[0], A[1], A[2], -1, 64, 0, 0, 0), DIM),
    ((A[0], A[1], A[2], 1 << 31, 64, 0, 0, 0), DIM),
    ((A[0], A[1], A[2], (1 << 31) - 1, 1 << 30, 0, 0, 0), DIM),     # too many blocks
    ((A[0], A[1], A[2], 4, 72, 0, 0, 0), MDIM),
    ((None, A[1], A[2], 4, 64, 0, 0, 0), NULL),
    ((A[0], A[1], None, 4, 64, 0, 0, 0), NULL),
    ((A[0], A[1] + 8, A[2], 4, 64, 0, 0, 0), MPTR),
    ((A[0], A[1], A[2] + 4, 4, 64, 0, 0, 0), MPTR),
    ((A[0], A[0] + 256, A[2], 4, 64, 0, 0, 0), OVER),               # Q inside X
    ((A[0], A[1], A[1] + 240, 4, 64, 0, 0, 0), OVER),               # S in Q's last bytes
    ((A[0], A[1], A[1] + 1008, 4, 64, 0, 0, 1), OVER),              # transposed Q is padded to 16
    ((None, None, None, 0, 64, 0, 0, 0), 0),
    ((None, None, None, 4, 0, 1, 1, 1), 0),
])
def test_quant_refusals(args, code):
    assert _capi.lib().swiglu_quant_b128(*args, None) == code


# swiglu_gemm_b128(A, As, B, Bs, Y, M, N, K, b_block, out_dtype)
@pytest.mark.parametrize("args,code", [
    ((*A[:5], 4, 64, 64, 0, 2), DTYPE),
    ((*A[:5], 4, 64, 64, 3, 0), BLOCK),
    ((*A[:5], -4, 64, 64, 0, 0), DIM),
    ((*A[:5], 4, 1 << 31, 64, 0, 0), DIM),
    ((*A[:5], (1 << 31) - 128, (1 << 31) - 8, 64, 0, 0), DIM),      # too many tiles
    ((*A[:5], 4, 60, 64, 0, 1), MDIM),
    ((*A[:5], 4, 64, 72, 0, 0), MDIM),
    ((A[0], None, A[2], A[3], A[4], 4, 64, 64, 0, 0), NULL),
    ((A[0], A[1], A[2], A[3], None, 4, 64, 64, 0, 0), NULL),
    ((A[0], A[1] + 4, A[2], A[3], A[4], 4, 64, 64, 0, 0), MPTR),
    ((A[0] + 1, A[1], A[2], A[3], A[4], 4, 64, 64, 0, 0), MPTR),
    ((A[0], A[1], A[2], A[3], A[3], 4, 64, 64, 1, 0), OVER),
    ((A[0], A[1], A[2], A[3], A[2] - 16, 4, 64, 64, 1, 0), OVER),
    ((None, None, None, None, None, 0, 64, 64, 0, 0), 0),
    ((None, None, None, None, None, 4, 0, 64, 0, 0), 0),
])
def test_gemm_refusals(args, code):
    assert _capi.lib().swiglu_gemm_b128(*args, None) == code


# swiglu_fwd_b128(X, Xs, Wg, Wgs, Wu, Wus, H, M, K, N, epi)
def test_fwd_refusals():
    f = _capi.lib().swiglu_fwd_b128
    ok = tuple(A[:7])
    assert f(*ok, 4, 64, 60, None, None) == MDIM
    assert f(*ok, 4, 72, 64, None, None) == MDIM
    assert f(*ok, 4, 64, -64, None, None) == DIM
    assert f(*ok[:6], None, 4, 64, 64, None, None) == NULL
    assert f(*ok[:5], None, ok[6], 4, 64, 64, None, None) == NULL
    assert f(*ok[:6], ok[6] + 2, 4, 64, 64, None, None) == MPTR
    assert f(*ok[:6], ok[4], 4, 64, 64, None, None) == OVER
    for epi in (_capi.Epilogue(5, 1.0, None, None), _capi.Epilogue(0, float("inf"), None, None),
                _capi.Epilogue(0, 1.0, A[8], None)):
        assert f(*ok, 4, 64, 64, ctypes.byref(epi), None) == EPI
    same = _capi.Epilogue(0, 1.0, A[8], A[8] + 16)
    assert f(*ok, 4, 64, 64, ctypes.byref(same), None) == OVER
    assert f(*[None] * 7, 0, 64, 64, None, None) == 0


def _p(post=None, pre=None, gate=None, rows=1, scale=1.0, eps=1e-6):
    return ctypes.byref(_capi.BlockNormParams(post, pre, gate, rows, scale, eps))


# swiglu_block_norm(Y, R, p, Rn, N, rstd_post, rstd_pre, M, D, dtype)
@pytest.mark.parametrize("args,code", [
    ((A[0], A[1], None, A[2], A[3], None, None, 4, 64, 0), NULL),
    ((A[0], A[1], _p(A[8], A[9]), A[2], A[3], None, None, 4, 64, 3), DTYPE),
    ((A[0], A[1], _p(A[8], A[9]), A[2], A[3], None, None, -1, 64, 0), DIM),
    ((A[0], A[1], _p(A[8], A[9]), A[2], A[3], None, None, 4, 16392, 0), DIM),
    ((A[0], A[1], _p(A[8], A[9]), A[2], A[3], None, None, 4, 8196, 1), DIM),
    ((A[0], A[1], _p(A[8], A[9]), A[2], A[3], None, None, 4, 68, 0), MDIM),
    ((A[0], A[1], _p(A[8], A[9], scale=float("nan")), A[2], A[3], None, None, 4, 64, 0), EPI),
    ((A[0], A[1], _p(A[8], A[9], eps=-1e-6), A[2], A[3], None, None, 4, 64, 0), EPI),
    ((A[0], A[1], _p(A[8], A[9], A[10], 3), A[2], A[3], None, None, 4, 64, 0), DIM),
    ((A[0], A[1], _p(A[8], A[9], A[10], 0), A[2], A[3], None, None, 4, 64, 0), DIM),
    ((A[0], A[1], _p(A[8], A[9], A[10], 8), A[2], A[3], None, None, 4, 64, 0), DIM),
    ((A[0], None, _p(A[8], A[9]), A[2], A[3], None, None, 4, 64, 0), NULL),
    ((A[0], A[1], _p(A[8], A[9]), A[2], None, None, None, 4, 64, 0), NULL),
    ((A[0], A[1], _p(A[8], A[9] + 2), A[2], A[3], None, None, 4, 64, 0), MPTR),
    ((A[0], A[1], _p(A[8], A[9]), A[2], A[3], A[4] + 4, None, 4, 64, 0), MPTR),
    ((A[0], A[1], _p(A[8], A[9]), A[0], A[3], None, None, 4, 64, 0), OVER),       # Rn on Y
    ((A[0], A[1], _p(A[8], A[9]), A[1] + 16, A[3], None, None, 4, 64, 0), OVER),  # Rn beside R
    ((A[0], A[1], _p(A[8], A[9]), A[2], A[2], None, None, 4, 64, 0), OVER),       # N on Rn
    ((A[0], A[1], _p(A[8], A[9]), A[2], A[1], None, None, 4, 64, 0), OVER),       # N on R
    ((None, None, _p(), None, None, None, None, 0, 64, 0), 0),
])
def test_norm_refusals(args, code):
    assert _capi.lib().swiglu_block_norm(*args, None) == code


# swiglu_block_norm_bwd(dRn, dN, Y, Rn, r1, r2, p, dY, dR, d_post, d_pre, d_gate, ws, bytes, M, D, dtype)
def test_norm_bwd_refusals():
    f = _capi.lib().swiglu_block_norm_bwd
    good = dict(dRn=A[0], dN=A[1], Y=A[2], Rn=A[3], r1=A[4], r2=A[5], p=_p(A[6], A[7]), dY=A[8],
                dR=A[9], d1=A[10], d2=A[11], dg=None, ws=A[12], nb=1 << 22, M=4, D=64, dt=0)

    def call(**kw):
        return f(*{**good, **kw}.values(), None)

    assert call(dt=7) == DTYPE
    assert call(D=60) == MDIM
    assert call(D=1 << 15) == DIM
    assert call(dN=None) == NULL
    assert call(r1=None) == NULL
    assert call(d2=None) == NULL
    assert call(p=_p(A[6], A[7], A[13], 2)) == NULL                   # a gate without d_gate
    assert call(p=_p(), dRn=None) == NULL                              # no gradient at all
    assert call(dR=A[9] + 8) == MPTR
    assert call(dY=A[0]) == OVER
    assert call(dR=A[8]) == OVER
    assert call(d1=A[6]) == OVER
    lib = _capi.lib()
    assert lib.swiglu_block_norm_bwd_workspace(_p(A[0]), 4, 60, 0) == -1
    assert lib.swiglu_block_norm_bwd_workspace(_p(A[0]), 0, 64, 0) == 0


def test_python_refusals():
    """Argument checks of the binding that need no device."""
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    u = torch.zeros((4, 64), dtype=torch.uint8)
    s = torch.zeros((4, 1))
    with pytest.raises(ValueError):
        up.swiglu_quant_b128(x)                       # not a CUDA tensor
    with pytest.raises(ValueError):
        up.swiglu_gemm_b128(u, s, u, s)
    with pytest.raises(ValueError):
        up.swiglu_fwd_b128(u, s, u, s, u, s)
    with pytest.raises(ValueError):
        up.swiglu_block_norm(x, x)
    with pytest.raises(ValueError):
        up.swiglu_block_norm_bwd(x, None, x, x, None, None)
    for code in (13, 14):
        assert _capi.status_string(code) != "unknown status"


def test_no_device_is_an_error():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    lib = _capi.lib()
    none = _capi.SWIGLU_ERR_NO_DEVICE
    assert lib.swiglu_quant_b128(A[0], A[1], A[2], 4, 64, 0, 0, 0, None) == none
    assert lib.swiglu_gemm_b128(*A[:5], 4, 64, 64, 0, 0, None) == none
    assert lib.swiglu_gemm_b128(None, None, None, None, A[4], 4, 64, 0, 0, 0, None) == none
    assert lib.swiglu_fwd_b128(*A[:7], 4, 64, 64, None, None) == none
    assert lib.swiglu_block_norm(A[0], A[1], _p(A[8], A[9]), A[2], A[3], None, None, 4, 64, 0,
                                 None) == none


def test_native_binding_leaves_other_calls_alone():
    """The native calls return None for what is not a call in order: CPU
    tensors, other objects, other numbers of arguments."""
    _capi.lib()
    b = _capi._native
    assert b is not None
    x, s = torch.zeros(4, 64), torch.zeros(4, 1)
    q = torch.zeros(4, 64, dtype=torch.uint8)
    assert b.quant_b128(x, False, False) is None and b.quant_b128(x) is None and b.quant_b128([1.0], True, True) is None
    assert b.block_norm(x, x, None, None, None, 1.0, 1e-6, False, None) is None
    assert b.block_norm(None, None, None, None, None, 1.0, 1e-6, False, None) is None
    assert b.block_norm(x, x, None, None, None, "1", None, False, None) is None
    assert b.block_norm_bwd(x, None, x, x, None, None, None, None, None, 1.0) is None
    assert b.gemm_b128(q, s, q, s, False, None) is None and b.gemm_b128(None, s, q, s, True, 3) is None
    assert b.fwd_b128(q, s, q, s, q, s, None, 0, 1.0, False) is None
    with pytest.raises((TypeError, ValueError)):
        b.bind(0, 0, 0, 0, 0, 0)
