"""Contracts of the operators around the projection that hold by construction
or on the host, without a GPU."""
import os
import re

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
