"""Contracts of the operators around the projection that hold by construction
or on the host, without a GPU."""
import ctypes
import os
import re

import pytest
import torch

from test_host_plans import _build_and_run
from up_projection_b200 import _capi

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "up_projection_b200", "csrc")


def _code(path):
    """A source file without its comments."""
    with open(path) as f:
        s = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", s, flags=re.S)


def test_early_started_kernels_read_with_plain_loads():
    """A kernel that starts while the one before it runs may read what that one
    writes: no read-only loads, named or inferred from const __restrict__."""
    early = [n for n in sorted(os.listdir(CSRC))
             if n.endswith(".cu") and re.search(r'#include "(pdl|b128)\.cuh"', _code(os.path.join(CSRC, n)))]
    assert early == ["block_norm.cu", "gemm_b128.cu", "gemm_b128_stream.cu", "quant_b128.cu"]
    for n in early + ["b128.cuh", "pdl.cuh"]:
        found = re.findall(r"__ldg|ld_nc\w*|\.nc\b|__restrict__", _code(os.path.join(CSRC, n)))
        assert not found, (n, found)


def _params(post=None, pre=None, gate=None, rows=1):
    return ctypes.byref(_capi.BlockNormParams(post, pre, gate, rows, 1.0, 1e-6))


@pytest.mark.parametrize("D", [1 << 60, 1 << 61, 1 << 62, (1 << 63) - 16, (1 << 62) + 64])
@pytest.mark.parametrize("dtype", [_capi.SWIGLU_BF16, _capi.SWIGLU_FP32])
def test_norm_row_lengths_whose_bytes_wrap_are_refused(D, dtype):
    """D times the element size wraps 64 bits to something small."""
    lib, a = _capi.lib(), [(i + 1) << 24 for i in range(16)]
    dim = _capi.SWIGLU_ERR_BAD_DIM
    assert lib.swiglu_block_norm(a[0], a[1], _params(a[2], a[3]), a[4], a[5], None, None, 4, D, dtype, None) == dim
    assert lib.swiglu_block_norm_bwd(*a[:6], _params(a[6], a[7]), *a[8:12], None, a[12], 1 << 22, 4, D, dtype,
                                     None) == dim
    assert lib.swiglu_block_norm_bwd_workspace(_params(a[6], a[7]), 4, D, dtype) == -1


@pytest.mark.parametrize("rows", [1 << 31, 1 << 55, (1 << 63) - 1])
def test_gate_rows_whose_bytes_wrap_are_refused(rows):
    """No rows: any number of gate rows divides them, up to the largest M."""
    lib, a = _capi.lib(), [(i + 1) << 24 for i in range(16)]
    dim = _capi.SWIGLU_ERR_BAD_DIM
    p = _params(gate=a[6], rows=rows)
    assert lib.swiglu_block_norm(a[0], a[1], p, a[4], None, None, None, 0, 64, 0, None) == dim
    assert lib.swiglu_block_norm_bwd(*a[:6], p, a[8], a[9], None, None, a[10], None, 0, 0, 64, 0, None) == dim


def test_gate_without_rows_is_refused():
    """Its null address would read as no gate at all.  (CPU tensors stand for a
    device's here: the check looks at shapes.)"""
    g = torch.ones((0, 64))
    assert g.data_ptr() == 0
    with pytest.raises(ValueError, match="gate"):
        _capi._norm_params(-1, torch.float32, 64, None, None, g, 1.0, 1e-6)
    assert _capi._norm_params(-1, torch.float32, 64, None, None, torch.ones((2, 64)), 1.0, 1e-6).gate_rows == 2


def test_status_words_are_read_once_and_written_only_if_set():
    """Each kernel file adds a word to swiglu_sync_status; a word that is clear
    costs one read (status_check.cu)."""
    _build_and_run(["tests/status_check.cu"], 6)
    for n in sorted(os.listdir(CSRC)):
        if n.endswith(".cu"):
            code = _code(os.path.join(CSRC, n))
            assert code.count("_status_fetch_and_clear(unsigned int *host_out") == code.count("return fetch_and_clear(g_"), n
