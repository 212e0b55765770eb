"""Plain fp64 forms of the operators around the projection, for the tests:
straight from the definitions in include/swiglu.h, on whatever device."""
import torch

BLOCK = 128


def norm_fwd(Y, R, post, pre, gate, scale, eps):
    """(R', N, r1, r2) and the magnitudes |R| + |s g P| of R' before
    cancellation, all fp64."""
    Y, R = Y.double(), R.double()
    M = Y.shape[0]
    P, r1, r2, N = Y, None, None, None
    if post is not None:
        r1 = 1 / torch.sqrt((Y * Y).mean(1) + eps)
        P = post.double() * Y * r1[:, None]
    if gate is not None:
        g = gate.double().reshape(-1, Y.shape[1])
        P = P * g.repeat_interleave(M // g.shape[0], 0)
    Rn = R + scale * P
    if pre is not None:
        r2 = 1 / torch.sqrt((Rn * Rn).mean(1) + eps)
        N = pre.double() * Rn * r2[:, None]
    return Rn, N, r1, r2, R.abs() + (scale * P).abs()


def norm_bwd(dRn, dN, Y, Rn, r1, r2, post, pre, gate, scale):
    """dict of dY, dR, d_post, d_pre, d_gate (None where absent) and of the
    magnitudes of their terms before cancellation ("|dY|", ...)."""
    Y, Rn = Y.double(), Rn.double()
    M, D = Y.shape
    z = torch.zeros_like(Y)
    dX = z if dRn is None else dRn.double()
    mX = dX.abs()
    o = dict(d_post=None, d_pre=None, d_gate=None)
    if pre is not None:
        n = Rn * r2.double()[:, None]
        a = pre.double() * dN.double()
        dX = dX + r2.double()[:, None] * (a - n * (a * n).mean(1, keepdim=True))
        mX = mX + r2.double()[:, None] * (a.abs() + n.abs() * (a * n).abs().mean(1, keepdim=True))
        o["d_pre"] = (dN.double() * n).sum(0)
        o["|d_pre|"] = (dN.double() * n).abs().sum(0)
    sg = torch.full_like(Y, scale)
    if gate is not None:
        g = gate.double().reshape(-1, D)
        sg = scale * g.repeat_interleave(M // g.shape[0], 0)
    y = Y if post is None else Y * r1.double()[:, None]
    w = 1.0 if post is None else post.double()
    if gate is not None:
        t = scale * w * dX * y
        o["d_gate"] = t.view(g.shape[0], M // g.shape[0], D).sum(1).view(gate.shape)
        o["|d_gate|"] = (scale * w * mX * y).abs().view(g.shape[0], M // g.shape[0], D).sum(1).view(gate.shape)
    if post is None:
        o["dY"], o["|dY|"] = sg * dX, (sg * mX).abs()
    else:
        r = r1.double()[:, None]
        b, m = sg * w * dX, (sg * w).abs() * mX
        o["dY"] = r * (b - y * (b * y).mean(1, keepdim=True))
        o["|dY|"] = r * (m + y.abs() * (m * y.abs()).mean(1, keepdim=True))
        o["d_post"] = (sg * dX * y).sum(0)
        o["|d_post|"] = (sg * mX * y).abs().sum(0)
    o["dR"], o["|dR|"] = dX, mX
    return o


def quant(X, block, transpose):
    """(codes uint8, scales fp64) by the definition: the scale's exponent by
    search, the code by comparing with every e4m3 value's neighbours."""
    x = X.double()
    if transpose:
        x = x.t()
    R, C = x.shape
    Cp = (C + 15) // 16 * 16
    cb, rb = (Cp + 127) // 128, (R + 127) // 128
    rows = rb * 128 if block == "tile" else R
    p = torch.zeros((rows, cb * 128), dtype=torch.float64, device=x.device)
    p[:R, :C] = x
    v = p.view(rb, 128, cb, 128) if block == "tile" else p.view(R, 1, cb, 128)
    a = v.abs().amax(dim=(1, 3), keepdim=True)
    bad = ~torch.isfinite(v).all(dim=3, keepdim=True).all(dim=1, keepdim=True)
    a = torch.where(bad, torch.ones_like(a), a)
    e = torch.floor(torch.log2(a.clamp_min(2.0 ** -1000))) - 10
    for _ in range(4):                       # up to the smallest with a <= 448 * 2^e
        e = torch.where(a > 448.0 * torch.exp2(e), e + 1, e)
    e = e.clamp(-126, 127)
    s = torch.where(a > 0, torch.exp2(e), torch.ones_like(a))
    q = torch.where(bad, torch.zeros_like(v), v) / s
    grid = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    mid = (grid[1:] + grid[:-1]) / 2
    m = q.abs().contiguous()
    lo = torch.bucketize(m, mid)             # first code whose upper midpoint is >= m
    at = mid[lo.clamp_max(125)]
    lo = torch.where((m == at) & (lo < 126) & (lo % 2 == 1), lo + 1, lo)
    code = lo.to(torch.uint8) | (torch.signbit(v) & torch.isfinite(v)).to(torch.uint8) * 128
    code = torch.where(bad.expand_as(code), torch.full_like(code, 0x7F), code)
    s = torch.where(bad, torch.full_like(s, float("nan")), s)
    code = code.reshape(rows, cb * 128)[:R, :Cp].contiguous()
    if transpose and Cp > C:
        code[:, C:] = torch.where(code[:, C:] == 0x7F, code[:, C:], torch.zeros_like(code[:, C:]))
    return code, s.reshape(s.shape[0], cb)


def values(q):
    return q.view(torch.float8_e4m3fn).double()


def spread(s, rows, cols, block):
    s = s.double().repeat_interleave(128, 1)[:, :cols]
    return s.repeat_interleave(128, 0)[:rows] if block == "tile" else s


def product(A, As, B, Bs, block):
    """(Y, sum of |terms|) fp64."""
    a = values(A) * spread(As, *A.shape, "row")
    b = values(B) * spread(Bs, *B.shape, block)
    return a @ b.t(), a.abs() @ b.abs().t()


def row_scales(s):
    """[rows, KB] values stored as the products take them."""
    rows, kb = s.shape
    st = torch.zeros((kb, (rows + 3) // 4 * 4), dtype=torch.float32, device=s.device)
    st[:, :rows] = s.t()
    return st[:, :rows].t()
