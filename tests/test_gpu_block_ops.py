"""Operators around the projection on a B200 against their plain fp64 forms:
e4m3 quantisation in blocks of 128, the block-scaled products, block norms and
their backward, and a run of them as an MLP block.

Tolerances.  An output is rounded once: eps/2 of its type relative to the
value (bf16 2^-8, fp32 2^-24).  An fp32 sum of n terms is off by at most
n 2^-24 of the sum of their magnitudes; `terms` below is that n with a few
operations per term added.  The tensor cores' fp32 accumulation may lose up to
one unit (2^-23) of the running sum per addition: 127 additions in a block."""
import math

import pytest
import torch

import block_ref as ref
import up_projection_b200 as up
from gpu_util import assert_guards_intact, dev, guarded_empty
from up_projection_b200 import _capi

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rand(shape, seed, dtype=torch.float32, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    ok = err <= bound + 1e-37
    assert bool(ok.all()), (f"{what}: {int((~ok).sum())} of {ok.numel()} outside, worst "
                            f"{float((err / (bound + 1e-37)).max())} of the bound")


def synced():
    assert up.swiglu_sync_status() == 0


# ------------------------------------------------------------- quantisation

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block,transpose", [("row", False), ("tile", False), ("row", True), ("tile", True)])
@pytest.mark.parametrize("R,C", [(1, 16), (3, 128), (16, 144), (17, 512), (127, 528), (128, 1536),
                                 (130, 2064), (300, 272)])
def test_quant_matches_definition(R, C, dtype, block, transpose):
    x = rand((R, C), R + C) * torch.exp(2 * rand((R, 1), 5)) * torch.exp(rand((1, C), 6))
    x[:, ::7] = 0
    x = x.to(DT[dtype])
    q, s = up.swiglu_quant_b128(x, block=block, transpose=transpose)
    rq, rs = ref.quant(x, block, transpose)
    assert q.shape == rq.shape and s.shape == rs.shape
    assert torch.equal(s.double(), rs)
    assert torch.equal(q, rq)


@pytest.mark.parametrize("block,transpose", [("row", False), ("tile", False), ("row", True), ("tile", True)])
def test_quant_special_values(block, transpose):
    """Blocks of zeros, of the smallest and largest magnitudes, at the scale's
    boundary 448 * 2^e, and with NaN or infinities."""
    x = rand((256, 384), 3, std=0.01)
    x[:, 128:256] = 0
    x[5, 128] = -0.0
    x[130, 300] = float("inf")
    x[200, 3] = float("nan")
    x[0, 0:2] = torch.tensor([448.0, -448.0])
    x[1, 0] = 448.0000305
    x[2, 0] = 2.0 ** -149
    x[3, 0] = 2.0 ** -126
    x[4, 0] = 3.4028234e38
    x[140:150] *= 1e-38
    q, s = up.swiglu_quant_b128(x, block=block, transpose=transpose)
    rq, rs = ref.quant(x, block, transpose)
    assert torch.equal(torch.nan_to_num(s.double(), nan=-1.0), torch.nan_to_num(rs, nan=-1.0))
    assert torch.equal(q, rq)


def test_quant_every_code_and_tie():
    """Every e4m3 value and every midpoint between neighbours (ties to even)."""
    grid = torch.arange(127, dtype=torch.uint8, device=dev()).view(torch.float8_e4m3fn).double()
    mid = (grid[1:] + grid[:-1]) / 2
    v = torch.cat([grid, mid, -grid, -mid])
    x = torch.full((128, 512), 0.0, device=dev())
    x[:, :v.numel()] = v.float()
    x[:, 0::128] = 448.0                    # every block's scale is 1
    q, s = up.swiglu_quant_b128(x)
    rq, rs = ref.quant(x, "row", False)
    assert bool((s == 1).all()) and torch.equal(q, rq)


def test_quant_writes_inside_its_outputs():
    R, C = 131, 272
    x = rand((R, C), 1, torch.bfloat16)
    for tr, blk in ((0, 0), (0, 1), (1, 0), (1, 1)):
        qn = C * 144 if tr else R * C
        sn = {(0, 0): 3 * 132, (0, 1): 2 * 3, (1, 0): 2 * C, (1, 1): 3 * 2}[(tr, blk)]
        qf, q = guarded_empty(qn, torch.uint8, 77)
        sf, s = guarded_empty(sn, torch.float32)
        st = _capi.lib().swiglu_quant_b128(x.data_ptr(), q.data_ptr(), s.data_ptr(), R, C, 0, blk, tr,
                                           torch.cuda.current_stream().cuda_stream)
        assert st == 0
        synced()
        assert_guards_intact(qf, 77)
        assert_guards_intact(sf)
        if (tr, blk) == (0, 0):
            assert bool((s.view(3, 132)[:, 131] == 1234.5).all())   # the padding is left alone


# ----------------------------------------------------------------- products

SHAPES = [(1, 8, 16), (1, 136, 272), (3, 264, 128), (8, 1032, 1040), (9, 24, 4096), (64, 2056, 512),
          (127, 72, 144), (128, 4096, 384), (129, 520, 656), (300, 1160, 1168), (513, 2304, 256),
          (1100, 264, 2000)]


def operands(M, N, K, block, seed=0):
    """Codes of random values and arbitrary positive scales."""
    A, _ = ref.quant(rand((M, K), seed + 1), "row", False)
    B, _ = ref.quant(rand((N, K), seed + 2), "row", False)
    kb = (K + 127) // 128
    As = ref.row_scales(torch.exp(rand((M, kb), seed + 3)))
    if block == "tile":
        Bs = torch.exp(rand(((N + 127) // 128, kb), seed + 4))
    else:
        Bs = ref.row_scales(torch.exp(rand((N, kb), seed + 4)))
    return A, As, B, Bs


def product_terms(K):
    """Error of the sums relative to the terms' magnitudes: the additions of a
    block (2^-23 each), the two scale products, and the sums over the blocks."""
    return 127 * 2 * U24 + (2 + (K + 127) // 128) * U24


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("block", ["tile", "row"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_matches_fp64(M, N, K, block, out):
    A, As, B, Bs = operands(M, N, K, block, M)
    Y = up.swiglu_gemm_b128(A, As, B, Bs, out_dtype=DT[out])
    synced()
    want, mag = ref.product(A, As, B, Bs, block)
    within(Y, want, HALF[DT[out]] * want.abs() + product_terms(K) * (1 + HALF[DT[out]]) * mag, "Y")


@pytest.mark.parametrize("block", ["tile", "row"])
@pytest.mark.parametrize("M,N,K", SHAPES + [(200, 14336, 384), (40, 6912, 1536), (8, 4096, 4096), (20, 512, 8192), (1, 8, 4112),
                                            (33, 40000, 256), (2, 60000, 144), (70, 24000, 272)])
def test_gemm_integers_are_exact(M, N, K, block):
    """Small integers and power-of-two scales: every partial sum is exact in
    fp32, so the fp32 result has to be equal, bit for bit, and every scale has
    to meet its own block."""
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N)
    codes = torch.tensor([0.0, 1.0, 2.0, -1.0, -2.0], device=dev()).to(torch.float8_e4m3fn).view(torch.uint8)
    A = codes[torch.randint(0, 5, (M, K), generator=g, device="cuda")]
    B = codes[torch.randint(0, 5, (N, K), generator=g, device="cuda")]
    kb = (K + 127) // 128

    def pow2(r):
        return torch.exp2(torch.randint(-2, 3, (r, kb), generator=g, device="cuda").float())

    As = ref.row_scales(pow2(M))
    Bs = pow2((N + 127) // 128) if block == "tile" else ref.row_scales(pow2(N))
    Y = up.swiglu_gemm_b128(A, As, B, Bs, out_dtype=torch.float32)
    synced()
    assert torch.equal(Y.double(), ref.product(A, As, B, Bs, block)[0])


@pytest.mark.parametrize("gu", [False, True])
@pytest.mark.parametrize("act,alpha", [(up.SWIGLU_ACT_SILU, 1.0), (up.SWIGLU_ACT_GELU_TANH, -0.75)])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gated_matches_fp64(M, N, K, act, alpha, gu):
    A, As, Wg, Gs = operands(M, N, K, "tile", M)
    _, _, Wu, Us = operands(M, N, K, "tile", M + 50)
    As = As / math.sqrt(K)           # G and U of order one
    As = ref.row_scales(As)
    r = up.swiglu_fwd_b128(A, As, Wg, Gs, Wu, Us, activation=act, gate_multiplier=alpha, return_gu=gu)
    synced()
    G, AG = ref.product(A, As, Wg, Gs, "tile")
    U, AU = ref.product(A, As, Wu, Us, "tile")
    c = product_terms(K)
    x = alpha * G
    k = math.sqrt(2 / math.pi)
    if act == up.SWIGLU_ACT_SILU:
        z, dz = x, torch.ones_like(x)
    else:
        z, dz = 2 * k * (x + 0.044715 * x ** 3), 2 * k * (1 + 3 * 0.044715 * x * x)
    s = torch.sigmoid(z)
    a, da = x * s, s + x * s * (1 - s) * dz
    # G is off by c AG, U by c AU, and the activation's exponential and
    # reciprocal by a few units of its argument's size (bf16 path)
    first = c * (da * alpha).abs() * AG * U.abs() + c * a.abs() * AU
    second = 4 * (c * alpha * AG) ** 2 * (1 + x.abs()) * U.abs()   # |act''| and the cubic's growth
    special = (8 + 4 * z.abs()) * U24 * (a * U).abs()
    H = r[0] if gu else r
    within(H, a * U, 2.0 ** -8 * (a * U).abs() + 1.01 * (first + second + special), "H")
    if gu:
        within(r[1], G, 2.0 ** -8 * G.abs() + 1.01 * c * AG, "G")
        within(r[2], U, 2.0 ** -8 * U.abs() + 1.01 * c * AU, "U")


@pytest.mark.parametrize("M", [1, 8, 20, 60, 128, 300])
@pytest.mark.parametrize("K", [384, 400])
@pytest.mark.parametrize("order", ["gate first", "up first", "one weight"])
def test_gated_weights_in_any_place(M, K, order):
    """The two weights behind one another in either order, or the same one:
    integer operands, so G and U are exact before their rounding."""
    N = 520
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K)
    codes = torch.tensor([0.0, 1.0, 2.0, -1.0, -2.0], device=dev()).to(torch.float8_e4m3fn).view(torch.uint8)
    A = codes[torch.randint(0, 5, (M, K), generator=g, device="cuda")]
    W = codes[torch.randint(0, 5, (2, N, K), generator=g, device="cuda")]
    kb = (K + 127) // 128
    s = [torch.exp2(torch.randint(-2, 3, ((N + 127) // 128, kb), generator=g, device="cuda").float()) for _ in range(2)]
    As = ref.row_scales(torch.exp2(torch.randint(-2, 3, (M, kb), generator=g, device="cuda").float()))
    i, j = {"gate first": (0, 1), "up first": (1, 0), "one weight": (0, 0)}[order]
    H, G, U = up.swiglu_fwd_b128(A, As, W[i], s[0], W[j], s[1], return_gu=True)
    synced()
    assert torch.equal(G, ref.product(A, As, W[i], s[0], "tile")[0].to(torch.bfloat16))
    assert torch.equal(U, ref.product(A, As, W[j], s[1], "tile")[0].to(torch.bfloat16))


def test_products_write_inside_their_outputs():
    M, N, K = 131, 264, 272
    s = torch.cuda.current_stream().cuda_stream
    lib = _capi.lib()
    for block in ("tile", "row"):
        A, As, B, Bs = operands(M, N, K, block)
        for code, dt in ((0, torch.bfloat16), (1, torch.float32)):
            full, y = guarded_empty(M * N, dt)
            assert lib.swiglu_gemm_b128(A.data_ptr(), As.data_ptr(), B.data_ptr(), Bs.data_ptr(),
                                        y.data_ptr(), M, N, K, 1 if block == "tile" else 0, code, s) == 0
            synced()
            assert_guards_intact(full)
            assert torch.equal(y.view(M, N), up.swiglu_gemm_b128(A, As, B, Bs, out_dtype=dt))


def test_products_nan_codes_and_scales():
    """A NaN code or scale makes its row (or column) NaN and no other; an
    infinite scale follows the formula; a zero scale gives zero."""
    M, N, K = 140, 264, 400
    A, As, B, Bs = operands(M, N, K, "tile", 9)
    A[3, 399] = 0x7F
    B[7, 0] = 0xFF
    As = As.clone()
    As[9, 1] = float("nan")
    As[10, 2] = 0.0
    As = ref.row_scales(As)
    Y = up.swiglu_gemm_b128(A, As, B, Bs, out_dtype=torch.float32)
    synced()
    nan = torch.zeros((M, N), dtype=torch.bool, device=dev())
    nan[3] = nan[9] = True
    nan[:, 7] = True
    assert torch.equal(torch.isnan(Y), nan)
    Az, Bz = A.clone(), B.clone()
    Az[3, 399] = Bz[7, 0] = 0
    Sz = As.clone()
    Sz[9, 1] = 0.0
    want, mag = ref.product(Az, ref.row_scales(Sz), Bz, Bs, "tile")
    within(Y[~nan], want[~nan], U24 * want[~nan].abs() + 1.01 * product_terms(K) * mag[~nan], "Y")


def test_products_empty_and_k_zero():
    e = torch.empty((0, 64), dtype=torch.uint8, device=dev())
    w = torch.zeros((16, 64), dtype=torch.uint8, device=dev())
    ws = torch.ones((1, 1), device=dev())
    assert up.swiglu_gemm_b128(e, torch.empty((0, 1), device=dev()), w, ws).shape == (0, 16)
    a = torch.empty((5, 0), dtype=torch.uint8, device=dev())
    as_ = torch.empty((5, 0), device=dev())
    b = torch.empty((16, 0), dtype=torch.uint8, device=dev())
    bs = torch.empty((1, 0), device=dev())
    y = torch.full((5, 16), 3.0, dtype=torch.bfloat16, device=dev())
    assert bool((up.swiglu_gemm_b128(a, as_, b, bs, Y=y) == 0).all())
    h, g, u = up.swiglu_fwd_b128(a, as_, b, bs, b, bs, return_gu=True)
    assert not bool(h.any()) and not bool(g.any()) and not bool(u.any())
    synced()


def test_products_refuse_other_layouts():
    A, As, B, Bs = operands(6, 24, 256, "row")
    with pytest.raises(ValueError):
        up.swiglu_gemm_b128(A, As.contiguous(), B, Bs)          # blocks innermost
    with pytest.raises(ValueError):
        up.swiglu_gemm_b128(A, As[:, :1], B, Bs)
    with pytest.raises(TypeError):
        up.swiglu_gemm_b128(A.int(), As, B, Bs)
    with pytest.raises(TypeError):
        up.swiglu_gemm_b128(A, As, B, Bs, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        up.swiglu_gemm_b128(A.t(), As, B, Bs)
    with pytest.raises(ValueError):
        up.swiglu_fwd_b128(A, As, B, Bs, B, Bs)                 # row scales of the weights


def test_gemm_is_deterministic_and_graph_safe():
    A, As, B, Bs = operands(300, 1160, 1168, "tile")
    first = up.swiglu_gemm_b128(A, As, B, Bs)
    out = torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            up.swiglu_gemm_b128(A, As, B, Bs, Y=out)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        out.zero_()
        g.replay()
        synced()
        assert torch.equal(out, first)


# -------------------------------------------------------------- block norms

NORM_SHAPES = [(1, 8), (1, 1536), (3, 64), (5, 264), (7, 2048), (33, 4096), (130, 520), (9, 5120),
               (4, 8192), (300, 128)]


def norm_inputs(M, D, dtype, post, pre, gate_rows, seed=0):
    dt = DT[dtype]
    v = dict(Y=rand((M, D), seed + 1, dt, 0.7), R=rand((M, D), seed + 2, dt, 2.0),
             post=rand((D,), seed + 3, dt, 0.2, 1.0) if post else None,
             pre=rand((D,), seed + 4, dt, 0.2, 1.0) if pre else None,
             gate=rand((gate_rows, D), seed + 5, dt, 0.5, 0.5) if gate_rows else None)
    if gate_rows == 1:
        v["gate"] = v["gate"].view(D)
    return v


def gate_count(M, kind):
    if kind == "rows":
        return M
    if kind == "groups":
        return max(k for k in (1, 2, 3, 5, 10, 11, 13) if M % k == 0)
    return {"none": 0, "channel": 1}[kind]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("post,pre,gate", [(True, True, "channel"), (False, True, "none"),
                                           (True, False, "groups"), (False, False, "rows"),
                                           (True, True, "rows"), (True, True, "none")])
@pytest.mark.parametrize("M,D", NORM_SHAPES + [(2, 16384)])
def test_norm_matches_fp64(M, D, dtype, post, pre, gate):
    if dtype == "f32" and D > 8192:
        D = 8192 - 4
    v = norm_inputs(M, D, dtype, post, pre, gate_count(M, gate), M + D)
    s, eps = -0.6, 1e-5
    Rn, N, r1, r2 = up.swiglu_block_norm(v["Y"], v["R"], v["post"], v["pre"], v["gate"], residual_scale=s,
                                         eps=eps, return_stats=True)
    wRn, wN, w1, w2, mag = ref.norm_fwd(v["Y"], v["R"], v["post"], v["pre"], v["gate"], s, eps)
    # a statistic: a sum of D squares (32 or fewer per thread, then a tree),
    # halved in relative terms by the root; a value: a few products more
    stat = (32 + 5 + 16 + 8) * U24
    h = HALF[DT[dtype]]
    within(Rn, wRn, h * wRn.abs() + (stat + 8 * U24) * (1 + h) * mag, "Rn")
    assert (N is None) == (not pre) and (r1 is None) == (not post) and (r2 is None) == (not pre)
    if post:
        within(r1, w1, stat * w1, "rstd_post")
    if pre:
        # R' is off by (stat + 8 u) mag, which moves r2 by its mean square share
        off = (stat + 8 * U24) * (mag * mag).mean(1).sqrt() * w2
        within(r2, w2, (stat + off) * w2, "rstd_pre")
        m = v["pre"].double().abs() * mag * w2[:, None]
        within(N, wN, h * wN.abs() + (1 + h) * ((stat + 8 * U24) * m + (stat + off)[:, None] * wN.abs()), "N")


def test_norm_in_place_and_given_output():
    v = norm_inputs(37, 1536, "bf16", True, True, 1)
    args = (v["Y"], v["R"], v["post"], v["pre"], v["gate"])
    Rn, N = up.swiglu_block_norm(*args)
    R2 = v["R"].clone()
    Rn2, N2 = up.swiglu_block_norm(v["Y"], R2, *args[2:], Rn=R2)
    assert Rn2 is R2 and torch.equal(R2, Rn) and torch.equal(N2, N)
    full, out = guarded_empty(37 * 1536, torch.bfloat16)
    Rn3, _ = up.swiglu_block_norm(*args, Rn=out.view(37, 1536))
    synced()
    assert torch.equal(Rn3, Rn)
    assert_guards_intact(full)


def test_norm_zero_rows_and_non_finite_rows():
    """A row of zeros has rstd 1/sqrt(eps); NaN and infinities stay in their row."""
    v = norm_inputs(6, 512, "f32", True, True, 0)
    v["Y"][1] = 0
    v["R"][1] = 0
    v["Y"][3, 7] = float("nan")
    v["R"][4, 9] = float("inf")
    Rn, N, r1, r2 = up.swiglu_block_norm(v["Y"], v["R"], v["post"], v["pre"], eps=1e-6, return_stats=True)
    synced()
    assert not bool(Rn[1].any()) and not bool(N[1].any())
    assert abs(float(r1[1]) - 1000) < 1e-2 and abs(float(r2[1]) - 1000) < 1e-2
    assert bool(torch.isnan(N[3]).all())
    assert float(r2[4]) == 0.0 and bool(torch.isnan(N[4, 9])) and not bool(N[4, :9].any())
    ok = [0, 1, 2, 5]
    assert bool(torch.isfinite(Rn[ok]).all()) and bool(torch.isfinite(N[ok]).all())


def test_norm_leading_dims_and_empty():
    v = norm_inputs(12, 256, "bf16", True, True, 3)
    Rn, N = up.swiglu_block_norm(v["Y"].view(3, 4, 256), v["R"].view(3, 4, 256), v["post"], v["pre"], v["gate"])
    R2, N2 = up.swiglu_block_norm(v["Y"], v["R"], v["post"], v["pre"], v["gate"])
    assert Rn.shape == (3, 4, 256) and torch.equal(Rn.view(12, 256), R2) and torch.equal(N.view(12, 256), N2)
    e = torch.empty((0, 256), dtype=torch.bfloat16, device=dev())
    Rn, N = up.swiglu_block_norm(e, e, v["post"], v["pre"])
    assert Rn.shape == N.shape == (0, 256)
    f = torch.empty((0,), device=dev())
    dY, dR, d1, d2, dg = up.swiglu_block_norm_bwd(e, e, e, e, f, f, v["post"], v["pre"], v["post"])
    synced()
    assert dY.shape == (0, 256) and not bool(d1.any()) and not bool(d2.any()) and not bool(dg.any())


def run_bwd(v, r1, r2, Rn, dRn, dN, s):
    got = up.swiglu_block_norm_bwd(dRn, dN, v["Y"], Rn, r1, r2, v["post"], v["pre"], v["gate"], residual_scale=s)
    return dict(zip(("dY", "dR", "d_post", "d_pre", "d_gate"), got))


def check_bwd(v, dtype, M, D, seed, with_dRn=True):
    s = 0.8
    Rn, _, r1, r2 = up.swiglu_block_norm(v["Y"], v["R"], v["post"], v["pre"], v["gate"], residual_scale=s,
                                         return_stats=True)
    dRn = rand((M, D), seed + 7, DT[dtype]) if with_dRn else None
    dN = rand((M, D), seed + 8, DT[dtype]) if v["pre"] is not None else None
    got = run_bwd(v, r1, r2, Rn, dRn, dN, s)
    synced()
    want = ref.norm_bwd(dRn, dN, v["Y"], Rn, r1, r2, v["post"], v["pre"], v["gate"], s)
    h = HALF[DT[dtype]]
    # row sums: 32 terms or fewer per thread, a tree of 5 + 16, a few products
    # each; the two means enter dY one through the other
    row = 2 * (32 + 5 + 16 + 12) * U24
    # column sums: at most M additions on top of the terms' own error
    col = row + (M + 40) * U24
    for k in ("dY", "dR"):
        within(got[k], want[k], h * want[k].abs() + (1 + h) * row * want["|%s|" % k], k)
    for k in ("d_post", "d_pre", "d_gate"):
        assert (got[k] is None) == (want[k] is None)
        if want[k] is not None:
            within(got[k], want[k], h * want[k].abs() + (1 + h) * col * want["|%s|" % k], k)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("post,pre,gate", [(True, True, "channel"), (False, True, "none"),
                                           (True, False, "groups"), (False, False, "rows"),
                                           (False, True, "channel"), (True, True, "rows"),
                                           (True, True, "groups"), (True, True, "none")])
@pytest.mark.parametrize("M,D", NORM_SHAPES + [(2, 16384), (700, 1536)])
def test_norm_bwd_matches_fp64(M, D, dtype, post, pre, gate):
    if dtype == "f32" and D > 8192:
        D = 8192 - 4
    check_bwd(norm_inputs(M, D, dtype, post, pre, gate_count(M, gate), M + D), dtype, M, D, M)


def test_norm_bwd_without_residual_gradient():
    check_bwd(norm_inputs(50, 768, "f32", True, True, 1), "f32", 50, 768, 1, with_dRn=False)


@pytest.mark.parametrize("M,groups", [(4096, 1), (4096, 16), (4000, 500), (3000, 1500)])
def test_norm_bwd_many_rows(M, groups):
    """Several workers per gate row, one per row, several rows per worker."""
    got = check_bwd(norm_inputs(M, 512, "f32", True, True, groups, 3), "f32", M, 512, 4)
    again = check_bwd(norm_inputs(M, 512, "f32", True, True, groups, 3), "f32", M, 512, 4)
    for k in got:
        assert torch.equal(got[k], again[k]), k


def test_norm_bwd_matches_differences():
    """The backward against central differences of the fp64 forward."""
    M, D, s, eps = 4, 64, 0.8, 1e-6
    v = norm_inputs(M, D, "f32", True, True, 2, 11)
    cR, cN = rand((M, D), 21), rand((M, D), 22)
    Rn, _, r1, r2 = up.swiglu_block_norm(v["Y"], v["R"], v["post"], v["pre"], v["gate"], residual_scale=s,
                                         eps=eps, return_stats=True)
    got = run_bwd(v, r1, r2, Rn, cR, cN, s)
    got = dict(Y=got["dY"], R=got["dR"], post=got["d_post"], pre=got["d_pre"], gate=got["d_gate"])

    def loss(u):
        Rn, N, *_ = ref.norm_fwd(u["Y"], u["R"], u["post"], u["pre"], u["gate"], s, eps)
        return float((Rn * cR.double()).sum() + (N * cN.double()).sum())

    u = {k: t.double() for k, t in v.items()}
    for name in u:
        for i in (0, 17, 63):
            step = 1e-5
            t = u[name].view(-1)
            old = float(t[i])
            t[i] = old + step
            up_ = loss(u)
            t[i] = old - step
            down = loss(u)
            t[i] = old
            num = (up_ - down) / (2 * step)
            # truncation ~ step^2, differences of sums ~ 1e2 in fp64 / step, fp32 result
            assert abs(float(got[name].reshape(-1)[i]) - num) <= 1e-5 * max(1.0, abs(num)) + 1e-6, name


def test_norm_bwd_other_stream_and_graph():
    """On another stream, and captured and replayed with new gradients: the
    eager call's bits."""
    M, D = 300, 1024
    v = norm_inputs(M, D, "bf16", True, True, 3)
    Rn, _, r1, r2 = up.swiglu_block_norm(v["Y"], v["R"], v["post"], v["pre"], v["gate"], return_stats=True)
    dRn, dN = rand((M, D), 5, torch.bfloat16), rand((M, D), 6, torch.bfloat16)
    want = run_bwd(v, r1, r2, Rn, dRn, dN, 1.0)
    synced()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = up.swiglu_block_norm_bwd(dRn, dN, v["Y"], Rn, r1, r2, v["post"], v["pre"], v["gate"], stream=side)
    side.synchronize()
    for a, b in zip(got, want.values()):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    sR, sN = torch.zeros_like(dRn), torch.zeros_like(dN)
    with torch.cuda.graph(g):
        got = up.swiglu_block_norm_bwd(sR, sN, v["Y"], Rn, r1, r2, v["post"], v["pre"], v["gate"])
    sR.copy_(dRn)
    sN.copy_(dN)
    g.replay()
    synced()
    for a, b in zip(got, want.values()):
        assert torch.equal(a, b)


def test_norm_bwd_workspace_is_checked():
    v = norm_inputs(40, 256, "bf16", True, True, 1)
    import ctypes
    p = _capi.BlockNormParams(v["post"].data_ptr(), v["pre"].data_ptr(), v["gate"].data_ptr(), 1, 1.0, 0.0)
    lib = _capi.lib()
    need = lib.swiglu_block_norm_bwd_workspace(ctypes.byref(p), 40, 256, 0)
    assert need > 0
    t = [torch.zeros((40, 256), dtype=torch.bfloat16, device=dev()) for _ in range(6)]
    r = [torch.zeros((40,), device=dev()) for _ in range(2)]
    d = [torch.zeros((256,), dtype=torch.bfloat16, device=dev()) for _ in range(3)]
    full, ws = guarded_empty(need, torch.uint8, 77)
    s = torch.cuda.current_stream().cuda_stream

    def call(w, n):
        return lib.swiglu_block_norm_bwd(t[0].data_ptr(), t[1].data_ptr(), t[2].data_ptr(), t[3].data_ptr(),
                                         r[0].data_ptr(), r[1].data_ptr(), ctypes.byref(p), t[4].data_ptr(),
                                         t[5].data_ptr(), *(x.data_ptr() for x in d), w, n, 40, 256, 0, s)

    assert call(None, need) == _capi.SWIGLU_ERR_WORKSPACE
    assert call(ws.data_ptr(), need - 1) == _capi.SWIGLU_ERR_WORKSPACE
    assert call(t[5].data_ptr(), need) == _capi.SWIGLU_ERR_OVERLAP
    assert call(ws.data_ptr(), need) == 0
    synced()
    assert_guards_intact(full, 77)


# ----------------------------------------------------------- an MLP block

def test_mlp_block_forward_and_backward():
    """norm -> gate/up -> down -> norm on 8-bit operands, and back: every step
    against its fp64 form on the step's own inputs."""
    M, D, F = 200, 512, 1040
    bf = torch.bfloat16
    x, res = rand((M, D), 1, bf, 0.5), rand((M, D), 2, bf)
    w1, w2 = rand((D,), 3, bf, 0.1, 1.0), rand((D,), 4, bf, 0.1, 1.0)
    Wg, Wu = rand((F, D), 5, bf, D ** -0.5), rand((F, D), 6, bf, D ** -0.5)
    Wd = rand((D, F), 7, bf, F ** -0.5)
    r0, n0 = up.swiglu_block_norm(x, res, None, w2)
    nq, ns = up.swiglu_quant_b128(n0)
    (gq, gs), (uq, us), (dq, ds) = (up.swiglu_quant_b128(w, block="tile") for w in (Wg, Wu, Wd))
    H, G, U = up.swiglu_fwd_b128(nq, ns, gq, gs, uq, us, return_gu=True)
    hq, hs = up.swiglu_quant_b128(H)
    y = up.swiglu_gemm_b128(hq, hs, dq, ds)
    r, n, s1, s2 = up.swiglu_block_norm(y, r0, w1, w2, residual_scale=0.5, return_stats=True)
    synced()
    wantG, mG = ref.product(nq, ns, gq, gs, "tile")
    within(G, wantG, 2.0 ** -8 * wantG.abs() + 1.01 * product_terms(D) * mG, "G")
    want, m = ref.product(hq, hs, dq, ds, "tile")
    within(y, want, 2.0 ** -8 * want.abs() + 1.01 * product_terms(F) * m, "y")
    # the quantised block is near the one of the unquantised operands: three
    # e4m3 roundings (2^-4 at most, about 2^-6 rms) of independent terms
    h = n0.double() @ Wg.double().t()
    h = h * torch.sigmoid(h) * (n0.double() @ Wu.double().t())
    plain = h @ Wd.double().t()
    assert float((y.double() - plain).norm() / plain.norm()) < 2.0 ** -3
    # backward through the norm, the down product and the gated pair
    dr, dn = rand((M, D), 8, bf), rand((M, D), 9, bf)
    dy, dr0, dw1, dw2, _ = up.swiglu_block_norm_bwd(dr, dn, y, r, s1, s2, w1, w2, residual_scale=0.5)
    dyq, dys = up.swiglu_quant_b128(dy)
    dqt, dst = up.swiglu_quant_b128(Wd, block="tile", transpose=True)    # [F, D]
    dH = up.swiglu_gemm_b128(dyq, dys, dqt, dst)
    dyt, dyts = up.swiglu_quant_b128(dy, transpose=True)                 # [D, M padded]
    ht, hts = up.swiglu_quant_b128(H, transpose=True)                    # [F, M padded]
    dWd = up.swiglu_gemm_b128(dyt, dyts, ht, hts, out_dtype=torch.float32)
    dG, dU = up.dswiglu_bwd(dH, G, U)
    synced()
    want, m = ref.product(dyq, dys, dqt, dst, "tile")
    within(dH, want, 2.0 ** -8 * want.abs() + 1.01 * product_terms(D) * m, "dH")
    want, m = ref.product(dyt, dyts, ht, hts, "row")
    within(dWd, want, U24 * want.abs() + 1.01 * product_terms(M) * m, "dWd")
    plain = dy.double().t() @ H.double()
    assert dWd.shape == Wd.shape and float((dWd.double() - plain).norm() / plain.norm()) < 2.0 ** -3
    plain = dy.double() @ Wd.double()
    assert float((dH.double() - plain).norm() / plain.norm()) < 2.0 ** -3
    assert bool(torch.isfinite(dG).all()) and bool(torch.isfinite(dU).all())


# ------------------------------------------------ many rows, calls in flight

@pytest.mark.parametrize("dtype,M,D", [("bf16", 1300, 4096), ("bf16", 1185, 4104), ("bf16", 700, 8192),
                                       ("f32", 605, 5120), ("f32", 2370, 2052), ("f32", 600, 8192)])
@pytest.mark.parametrize("post,pre,gate", [(True, True, "channel"), (False, True, "groups"),
                                           (True, False, "rows"), (False, False, "none")])
def test_norm_many_rows_matches_fp64(dtype, M, D, post, pre, gate):
    """Rows of 8 KB and more, several per block: rows through shared memory."""
    v = norm_inputs(M, D, dtype, post, pre, gate_count(M, gate), M + D)
    s, eps = 0.7, 1e-6
    Rn, N, r1, r2 = up.swiglu_block_norm(v["Y"], v["R"], v["post"], v["pre"], v["gate"], residual_scale=s,
                                         eps=eps, return_stats=True)
    wRn, wN, w1, w2, mag = ref.norm_fwd(v["Y"], v["R"], v["post"], v["pre"], v["gate"], s, eps)
    stat = (32 + 5 + 16 + 8) * U24   # as in test_norm_matches_fp64
    h = HALF[DT[dtype]]
    within(Rn, wRn, h * wRn.abs() + (stat + 8 * U24) * (1 + h) * mag, "Rn")
    if post:
        within(r1, w1, stat * w1, "rstd_post")
    if pre:
        off = (stat + 8 * U24) * (mag * mag).mean(1).sqrt() * w2
        within(r2, w2, (stat + off) * w2, "rstd_pre")
        m = v["pre"].double().abs() * mag * w2[:, None]
        within(N, wN, h * wN.abs() + (1 + h) * ((stat + 8 * U24) * m + (stat + off)[:, None] * wN.abs()), "N")


def test_norm_many_rows_in_place_and_non_finite():
    M, D = 1300, 4096
    v = norm_inputs(M, D, "bf16", True, True, 1)
    want, wn = up.swiglu_block_norm(v["Y"], v["R"], v["post"], v["pre"], v["gate"])
    bad = [0, 7, 649, 1299]
    Y = v["Y"].clone()
    Y[bad, 5] = torch.tensor([float("inf"), float("nan"), float("-inf"), float("nan")], dtype=torch.bfloat16,
                             device=dev())
    R = v["R"].clone()
    Rn, N = up.swiglu_block_norm(Y, R, v["post"], v["pre"], v["gate"], Rn=R)
    synced()
    good = torch.ones(M, dtype=torch.bool, device=dev())
    good[bad] = False
    assert Rn is R and torch.equal(Rn[good], want[good]) and torch.equal(N[good], wn[good])
    assert bool(torch.isnan(N[~good]).any(1).all())


@pytest.mark.parametrize("dtype,M,D,groups", [("bf16", 700, 8192, 1), ("bf16", 640, 8192, 10), ("bf16", 320, 16384, 1),
                                              ("bf16", 320, 16384, 2), ("bf16", 400, 12008, 0), ("bf16", 5000, 64, 5),
                                              ("bf16", 6000, 256, 1), ("f32", 500, 8188, 1), ("f32", 480, 8192, 3),
                                              ("f32", 1020, 1536, 12), ("f32", 4500, 16, 4500)])
def test_norm_bwd_row_lengths(dtype, M, D, groups):
    """The layouts of the row rings: one warp to 16 per row, 8 to 32 elements
    per thread, one stage to many."""
    check_bwd(norm_inputs(M, D, dtype, True, True, groups, M + D), dtype, M, D, M + 1)


def test_norm_bwd_non_finite_row_stays_in_its_row():
    M, D = 600, 4096
    v = norm_inputs(M, D, "bf16", True, True, 1)
    Rn, _, r1, r2 = up.swiglu_block_norm(v["Y"], v["R"], v["post"], v["pre"], v["gate"], return_stats=True)
    dRn, dN = rand((M, D), 5, torch.bfloat16), rand((M, D), 6, torch.bfloat16)
    want = run_bwd(v, r1, r2, Rn, dRn, dN, 1.0)
    bad = dN.clone()
    bad[[3, 599], 9] = float("inf")
    got = run_bwd(v, r1, r2, Rn, dRn, bad, 1.0)
    synced()
    good = torch.ones(M, dtype=torch.bool, device=dev())
    good[[3, 599]] = False
    for k in ("dY", "dR"):
        assert torch.equal(got[k][good], want[k][good])
    assert not bool(torch.isfinite(got["d_pre"][9])) and bool(torch.isfinite(got["d_pre"][10:]).all())


def mlp_step(x, res, w1, w2, Wg, Wu, Wd):
    """norm, gate and up, down, norm, all operands quantised on the way."""
    r0, n0 = up.swiglu_block_norm(x, res, None, w2)
    nq, ns = up.swiglu_quant_b128(n0)
    (gq, gs), (uq, us), (dq, ds) = (up.swiglu_quant_b128(w, block="tile") for w in (Wg, Wu, Wd))
    hq, hs = up.swiglu_quant_b128(up.swiglu_fwd_b128(nq, ns, gq, gs, uq, us))
    return up.swiglu_block_norm(up.swiglu_gemm_b128(hq, hs, dq, ds), r0, w1, w2, residual_scale=0.5)


def mlp_weights(D, F, seed):
    bf = torch.bfloat16
    return (rand((D,), seed + 3, bf, 0.1, 1.0), rand((D,), seed + 4, bf, 0.1, 1.0),
            rand((F, D), seed + 5, bf, D ** -0.5), rand((F, D), seed + 6, bf, D ** -0.5),
            rand((D, F), seed + 7, bf, F ** -0.5))


@pytest.mark.parametrize("M", [1, 8, 60, 200])
def test_steps_in_flight_keep_their_order(M):
    """Each kernel starts while the one before it drains; weights and
    activations are written by the kernels just before.  Steps without a wait
    between them, memory of one reused by the next, give the bits of steps
    that are waited for."""
    D, F = 512, 1040
    bf = torch.bfloat16
    steps = [(rand((M, D), 30 + i, bf, 0.5), rand((M, D), 60 + i, bf, 2.0), mlp_weights(D, F, 100 * i))
             for i in range(4)]
    want = []
    for x, res, w in steps:
        want.append(mlp_step(x, res, *w))
        synced()
    for _ in range(5):
        got = [mlp_step(x, res, *w) for x, res, w in steps]
        for g, t in zip(got, want):
            assert torch.equal(g[0], t[0]) and torch.equal(g[1], t[1])


@pytest.mark.parametrize("M", [8, 200])
def test_step_captured_and_on_two_streams(M):
    D, F = 512, 1040
    bf = torch.bfloat16
    w = mlp_weights(D, F, 0)
    a, b = ((rand((M, D), 30 + i, bf, 0.5), rand((M, D), 60 + i, bf, 2.0)) for i in range(2))
    want = [mlp_step(*a, *w), mlp_step(*b, *w)]
    synced()
    # two streams at once
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s, v in zip(side, (a, b)):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append([mlp_step(*v, *w) for _ in range(10)])
    torch.cuda.synchronize()
    for t, all_ in zip(want, got):
        for g in all_:
            assert torch.equal(g[0], t[0]) and torch.equal(g[1], t[1])
    # two graphs, replayed in turn and side by side
    graphs, outs, ins = [], [], []
    for v in (a, b):
        x, res = torch.zeros_like(v[0]), torch.zeros_like(v[1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mlp_step(x, res, *w))
        graphs.append(g)
        ins.append((x, res))
    for (x, res), v in zip(ins, (a, b)):
        x.copy_(v[0])
        res.copy_(v[1])
    torch.cuda.synchronize()
    for rounds in range(3):
        for s, g in zip(side, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for g, t in zip(outs, want):
            assert torch.equal(g[0], t[0]) and torch.equal(g[1], t[1])
            g[0].zero_()
            g[1].zero_()
        torch.cuda.synchronize()


# Row counts around the change of kernels (32 and 64 rows), short and long
# reductions.
TURNS = [(m, 520, k) for m in (31, 32, 33, 63, 64, 65) for k in (2032, 2048, 2064, 2192)] + [(64, 8, 14336),
                                                                                              (40, 20000, 2176)]


@pytest.mark.parametrize("block", ["tile", "row"])
@pytest.mark.parametrize("M,N,K", TURNS)
def test_gemm_row_counts_are_exact(M, N, K, block):
    test_gemm_integers_are_exact(M, N, K, block)


@pytest.mark.parametrize("order", ["gate first", "up first", "one weight"])
@pytest.mark.parametrize("M,K", [(33, 2192), (60, 2176), (64, 2192), (65, 2192), (128, 384)])
def test_gated_row_counts_are_exact(M, K, order):
    test_gated_weights_in_any_place(M, K, order)


@pytest.mark.parametrize("dtype,M,D", [("bf16", 4800, 512), ("bf16", 2400, 1032), ("bf16", 1200, 2048),
                                       ("bf16", 5000, 520), ("f32", 4800, 256), ("f32", 2500, 500),
                                       ("f32", 1300, 1024), ("bf16", 620, 4104)])
@pytest.mark.parametrize("post,pre,gate", [(True, True, "groups"), (False, True, "channel"),
                                           (True, False, "none"), (False, False, "rows")])
def test_norm_shorter_rows_through_rings(dtype, M, D, post, pre, gate):
    test_norm_many_rows_matches_fp64(dtype, M, D, post, pre, gate)


def test_native_and_ctypes_calls_agree(monkeypatch):
    """The native binding and the path through ctypes: the same outputs, layouts
    and refusals."""
    from up_projection_b200 import _capi
    v = norm_inputs(12, 256, "bf16", True, True, 3)
    for t in v.values():
        t.requires_grad_(True)
    x = rand((37, 400), 1, torch.bfloat16)

    def calls():
        Rn, N, r1, r2 = up.swiglu_block_norm(v["Y"], v["R"], v["post"], v["pre"], v["gate"], return_stats=True)
        out = [Rn, N, r1, r2, *up.swiglu_block_norm(v["Y"], v["R"])[:1],
               *up.swiglu_block_norm_bwd(Rn, N, v["Y"], Rn, r1, r2, v["post"], v["pre"], v["gate"]),
               *[t for t in up.swiglu_block_norm_bwd(Rn, None, v["Y"], Rn, None, None) if t is not None]]
        for block in ("row", "tile"):
            for transpose in (False, True):
                out += up.swiglu_quant_b128(x, block, transpose)
        q, s = up.swiglu_quant_b128(x.view(1, 37, 400))
        w, ws = up.swiglu_quant_b128(rand((264, 400), 2, torch.bfloat16), "tile")
        out += [q, s, up.swiglu_gemm_b128(q, s, w, ws), up.swiglu_gemm_b128(q, s, w, ws, out_dtype=torch.float32)]
        out += up.swiglu_fwd_b128(q, s, w, ws, w, ws, return_gu=True)
        out.append(up.swiglu_fwd_b128(q[0].view(torch.float8_e4m3fn), s, w, ws, w, ws, activation=up.SWIGLU_ACT_GELU_TANH,
                                      gate_multiplier=2))
        H = torch.empty((37, 264), dtype=torch.bfloat16, device=dev())
        assert up.swiglu_gemm_b128(q, s, w, ws, Y=H) is H and up.swiglu_fwd_b128(q, s, w, ws, w, ws, H=H) is H
        with pytest.raises(up.SwigluError):
            up.swiglu_block_norm(v["Y"], v["R"], v["post"], v["pre"], v["post"].expand(5, 256).contiguous())
        with pytest.raises(up.SwigluError):
            up.swiglu_block_norm(v["Y"], v["R"], residual_scale=float("inf"))
        with pytest.raises(up.SwigluError):
            up.swiglu_quant_b128(x[:, :392].contiguous())
        with pytest.raises(up.SwigluError):
            up.swiglu_gemm_b128(q, s, w[:9].contiguous(), ws[:1].contiguous())
        with pytest.raises(up.SwigluError):
            up.swiglu_fwd_b128(q, s, w, ws, w, ws, activation=9)
        for bad in ((v["Y"], v["R"][:6]), (v["Y"], v["R"].float()), (v["Y"].t(), v["R"]), (v["Y"].cpu(), v["R"])):
            with pytest.raises((ValueError, TypeError)):
                up.swiglu_block_norm(*bad)
        with pytest.raises(ValueError):
            up.swiglu_gemm_b128(q, s[:36], w, ws)
        synced()
        return out

    native = _capi._native
    assert native is not None
    a = calls()
    monkeypatch.setattr(_capi, "_native", None)
    b = calls()
    assert len(a) == len(b)
    for s, t in zip(a, b):
        assert s.dtype == t.dtype and s.shape == t.shape and s.stride() == t.stride() and torch.equal(s, t)
        assert not s.requires_grad and not t.requires_grad
