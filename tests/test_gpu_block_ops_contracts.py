"""Contracts of the operators around the projection on a B200 that the tests of
their results do not reach."""
import pytest
import torch

import block_ref as ref
import up_projection_b200 as up
from gpu_util import dev
from test_gpu_block_ops import rand
from up_projection_b200 import _capi

pytestmark = pytest.mark.gpu


def _stream_calls():
    """name -> (call on a stream, bytes of its first output)."""
    M, D, N = 512, 1024, 520
    bf = torch.bfloat16
    x, w = rand((M, D), 1, bf), rand((D,), 2, bf)
    (a, sa), (b, sb) = up.swiglu_quant_b128(x), up.swiglu_quant_b128(rand((N, D), 3, bf), "tile")
    Rn, _, r1, r2 = up.swiglu_block_norm(x, x, w, w, return_stats=True)
    return {
        "quant": (lambda s: up.swiglu_quant_b128(x, stream=s), M * D),
        "gemm": (lambda s: (up.swiglu_gemm_b128(a, sa, b, sb, stream=s),), 2 * M * N),
        "gated": (lambda s: up.swiglu_fwd_b128(a, sa, b, sb, b, sb, return_gu=True, stream=s), 2 * M * N),
        "norm": (lambda s: up.swiglu_block_norm(x, x, w, w, return_stats=True, stream=s), 2 * M * D),
        "norm_bwd": (lambda s: up.swiglu_block_norm_bwd(x, x, x, Rn, r1, r2, w, w, stream=s), 2 * M * D),
    }


@pytest.mark.parametrize("name", ["quant", "gemm", "gated", "norm", "norm_bwd"])
@pytest.mark.parametrize("handle", [False, True])
def test_outputs_drawn_for_another_stream_wait_for_their_memory(name, handle):
    """Outputs are drawn on the current stream: their memory may be that of
    tensors whose last reader there has not run yet."""
    call, nbytes = _stream_calls()[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = [t.clone() for t in call(None) if t is not None]
    torch.cuda.synchronize()
    for _ in range(3):
        old = [torch.full((nbytes,), 85, dtype=torch.uint8, device=dev()) for _ in range(6)]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)            # some 10 ms
        copies = [t.clone() for t in old]
        del old                                  # back to the allocator, still to be read
        got = call(side.cuda_stream if handle else side)
        torch.cuda.synchronize()
        assert all(bool((c == 85).all()) for c in copies)
        for g, t in zip(got, want):
            assert torch.equal(g, t)


def test_call_on_a_stream_that_captures_beside_the_current_one():
    """The current stream does not capture, the call's does: no wait between
    them, which would end the capture."""
    x = rand((64, 256), 1, torch.bfloat16)
    want = up.swiglu_quant_b128(x)
    side = torch.cuda.Stream()
    up.swiglu_quant_b128(x, stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        g.capture_begin(capture_error_mode="relaxed")
    got = up.swiglu_quant_b128(x, stream=side)
    with torch.cuda.stream(side):
        g.capture_end()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_call_on_another_stream_stays_out_of_a_capture():
    """The current stream captures, the call's does not: it runs at once, and
    the capture ends as it would without it."""
    M, D = 64, 256
    x, w = rand((M, D), 1, torch.bfloat16), rand((D,), 2, torch.bfloat16)
    Rn, _, r1, r2 = up.swiglu_block_norm(x, x, w, w, return_stats=True)
    want = up.swiglu_block_norm_bwd(x, x, x, Rn, r1, r2, w, w)
    side = torch.cuda.Stream()
    up.swiglu_block_norm_bwd(x, x, x, Rn, r1, r2, w, w, stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = up.swiglu_block_norm_bwd(x, x, x, Rn, r1, r2, w, w, stream=side)
        y = x + 1
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want) if b is not None)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, x + 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("R,C", [(1, 16), (5, 144), (121, 272), (130, 400), (250, 128), (268, 272)])
def test_transposed_codes_behind_the_rows_are_zero(R, C, block, dtype):
    """Columns R.. of a transposed Q are 0, also in a block that holds NaN or
    Inf (whose own codes are 0x7F)."""
    x = rand((R, C), R + C, torch.float32)
    x[R - 1, 0] = float("nan")
    x[0, C // 2] = float("inf")
    x[R // 2, C - 1] = float("-inf")
    x = x.to(dtype)
    q, s = up.swiglu_quant_b128(x, block=block, transpose=True)
    wq, ws = ref.quant(x, block, True)
    wq[:, R:] = 0
    assert q.shape == (C, (R + 15) // 16 * 16)
    assert torch.equal(q, wq)
    assert torch.equal(torch.nan_to_num(s.double(), nan=-1.0), torch.nan_to_num(ws, nan=-1.0))


@pytest.mark.parametrize("native", [True, False])
@pytest.mark.parametrize("M", [0, 6])
def test_gate_without_rows_is_refused(M, native, monkeypatch):
    """A gate [0, D] is no gate row for any row, not a call without a gate."""
    _capi.lib()
    if not native:
        monkeypatch.setattr(_capi, "_native", None)
    x, g, w = (torch.ones((n, 64), device=dev()) for n in (M, 0, 1))
    with pytest.raises(ValueError):
        up.swiglu_block_norm(x, x, gate=g)
    with pytest.raises(ValueError):
        up.swiglu_block_norm_bwd(x, None, x, x, None, None, gate=g)
    assert torch.equal(up.swiglu_block_norm(x, x, gate=w)[0], x + x)


def _one_product_per_block(M, N, kb, seed):
    """Operands whose blocks hold one product 1 x 1 each, scaled by powers of
    two of such different sizes that the order of the fp32 sums shows."""
    one = torch.tensor(1.0, device=dev()).to(torch.float8_e4m3fn).view(torch.uint8)
    A = torch.zeros((M, kb * 128), dtype=torch.uint8, device=dev())
    B = torch.zeros((N, kb * 128), dtype=torch.uint8, device=dev())
    A[:, ::128] = one
    B[:, ::128] = one
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    sign = torch.randint(0, 2, (M, kb), generator=g, device="cuda").float() * 2 - 1
    As = sign * torch.rand((M, kb), generator=g, device="cuda") * torch.exp2(
        torch.randint(0, 30, (M, kb), generator=g, device="cuda").float())
    return A, ref.row_scales(As), B


@pytest.mark.parametrize("M", [65, 300])
@pytest.mark.parametrize("block", ["tile", "row"])
def test_many_rows_add_their_blocks_in_order(M, block):
    N, kb = 136, 19
    A, As, B = _one_product_per_block(M, N, kb, M)
    Bs = torch.ones((2, kb), device=dev()) if block == "tile" else ref.row_scales(torch.ones((N, kb), device=dev()))
    Y = up.swiglu_gemm_b128(A, As, B, Bs, out_dtype=torch.float32)
    want = torch.zeros((M,), device=dev())
    for b in range(kb):
        want = want + As[:, b]
    assert torch.equal(Y, want[:, None].expand(M, N))
    assert not torch.equal(As.double().sum(1).float(), want)    # (the order does show)


@pytest.mark.parametrize("M", [1, 8, 20, 32, 33, 64])
def test_few_rows_give_the_same_bits_every_time(M):
    N, kb = 520, 40
    A, As, B = _one_product_per_block(M, N, kb, M)
    Bs = torch.ones(((N + 127) // 128, kb), device=dev())
    Y = [up.swiglu_gemm_b128(A, As, B, Bs, out_dtype=torch.float32) for _ in range(4)]
    assert all(torch.equal(y, Y[0]) for y in Y)
    # each partial sum and each join is off by half a unit of at most the terms' sum
    bound = kb * 2.0 ** -24 * As.double().abs().sum(1)
    assert bool(((Y[0].double() - As.double().sum(1)[:, None]).abs() <= bound[:, None]).all())


@pytest.mark.parametrize("M", [4, 40, 200])
def test_scales_meet_before_the_sums(M):
    """Far apart, the scales' product is what counts; beyond fp32's range it is
    infinite, below the subnormals zero."""
    N, kb = 136, 17
    A, _, B = _one_product_per_block(M, N, kb, 0)
    a, b = torch.ones((M, kb), device=dev()), torch.ones((2, kb), device=dev())
    a[:, 3], b[:, 3] = 2.0 ** 110, 2.0 ** -108
    a[:, 4], b[:, 4] = 2.0 ** -120, 2.0 ** 121
    a[:, 5], b[:, 5] = 2.0 ** -100, 2.0 ** -100
    Y = up.swiglu_gemm_b128(A, ref.row_scales(a), B, b, out_dtype=torch.float32)
    assert bool((Y == kb - 3 + 4 + 2).all())
    a[0, 7], b[0, 7] = 2.0 ** 100, 2.0 ** 100
    A[0, 7 * 128] = 0                           # the block's sum is 0
    Y = up.swiglu_gemm_b128(A, ref.row_scales(a), B, b, out_dtype=torch.float32)
    assert bool(torch.isnan(Y[0, :128]).all()) and bool(torch.isfinite(Y[1:, 128:]).all())
