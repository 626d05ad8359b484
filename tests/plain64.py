"""Plain 64-bit forms of the MXFP4 products and the gated block, with the
elementwise error each fp32 / bf16 step of the kernels may add (torch, any
device). Half steps: bf16 2^-8, fp32 2^-24 relative.

An fp32 sum of K products on the matrix cores passes at most K/4 + 64
roundings on any chain (32 products and more enter per instruction, their
inner additions in groups; 64 covers the slices of a split sum), each half a
step of a partial sum that is at most sum |x||w|."""
import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24


def sum_err(absprod, K):
    return (K / 4 + 64) * U32 * absprod


def exact_values(codes, scales):
    """MXFP4 codes [N][K/2] and scale bytes [N][K/32] -> fp64 [N][K]."""
    mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=codes.device)
    pow2 = torch.tensor([2.0 ** (b - 127) for b in range(255)] + [float("nan")], dtype=torch.float64,
                        device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(codes.shape[0], -1).long()
    v = mags[c & 7] * torch.where(c >= 8, -1.0, 1.0).to(torch.float64)
    return v * pow2[scales.long()].repeat_interleave(32, dim=1)


def mxfp4_round(x):
    """x [R][K] -> (values fp64, code magnitudes' units fp64) after MXFP4 rounding, by search over the E2M1 values:
    the nearest, the even code on a tie."""
    v = x.double().reshape(x.shape[0], -1, 32)
    bad = ~torch.isfinite(v).all(dim=-1, keepdim=True)
    m = torch.where(bad, torch.ones_like(v), v).abs().amax(dim=-1, keepdim=True)
    X = torch.full_like(m, -127.0)
    for e in range(-126, 126):  # X = floor(log2 m) - 2
        X = torch.where(m >= 2.0 ** (e + 2), torch.full_like(X, float(e)), X)
    pow2 = torch.tensor([2.0 ** i for i in range(-127, 128)], dtype=torch.float64, device=x.device)
    unit = pow2[(X + 127).long()]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    a = v.abs() / unit
    best = torch.zeros_like(a)
    dist = a.clone()
    for c in range(1, 8):
        d = (a - grid[c]).abs()
        take = (d < dist) | ((d == dist) & (c % 2 == 0))
        best = torch.where(take, grid[c], best)
        dist = torch.where(take, d, dist)
    out = torch.where(bad, torch.full_like(v, float("nan")), torch.copysign(best, v) * unit)
    return out.reshape(x.shape)


def linear(x, W, out_half=U16):
    """x, W fp64 -> y, elementwise error bound of the kernels' y."""
    y = x @ W.t()
    A = x.abs() @ W.abs().t()
    return y, sum_err(A, x.shape[1]) * (1 + out_half) + out_half * y.abs()


def _act(g, u, L):
    gc, uc = torch.clamp(g, max=L), torch.clamp(u, -L, L)
    s = torch.sigmoid(gc)
    return gc, uc, s


def ffn(x, w13, w2, L, dy=None):
    """The block on fp64 copies: dict of y (and dx, dw13, dw2), each (value, bound)."""
    I = w2.shape[1]
    T, H = x.shape
    w1, w3 = w13[:I], w13[I:]
    g, u = x @ w1.t(), x @ w3.t()
    eg, eu = sum_err(x.abs() @ w1.abs().t(), H), sum_err(x.abs() @ w3.abs().t(), H)
    gc, uc, s = _act(g, u, L)
    silu = gc * s
    h = silu * uc
    fast = 2.0 ** -20  # exponential and reciprocal of the activation, a few units in the last place each
    eh = 1.1 * uc.abs() * eg + silu.abs() * eu + (U16 + fast) * h.abs()
    y = h @ w2.t()
    ey = eh @ w2.abs().t() + sum_err(h.abs() @ w2.abs().t(), I) + U16 * y.abs()
    res = {"y": (y, ey * (1 + U16))}
    if dy is None:
        return res
    dh = dy @ w2
    edh = sum_err(dy.abs() @ w2.abs(), H)
    d1 = s * (1 + gc * (1 - s))
    dg, du = dh * uc * d1, dh * silu
    sg, su = eg, eu  # g and u are saved in fp32
    edg = (uc * d1).abs() * edh + (dh * d1).abs() * su + 0.5 * (dh * uc).abs() * sg + (U16 + 4 * fast) * dg.abs()
    edu = silu.abs() * edh + 1.1 * dh.abs() * sg + (U16 + 4 * fast) * du.abs()
    # within the fp32 error of a border the mask may fall either way
    edg = torch.where((g - L).abs() <= 2 * eg, dg.abs() + edg, torch.where(g > L, torch.zeros_like(edg), edg))
    edu = torch.where((u.abs() - L).abs() <= 2 * eu, du.abs() + edu, torch.where(u.abs() > L, torch.zeros_like(edu), edu))
    dg = torch.where(g > L, torch.zeros_like(dg), dg)
    du = torch.where(u.abs() > L, torch.zeros_like(du), du)
    dgu, edgu = torch.cat((dg, du), 1), torch.cat((edg, edu), 1)
    dx = dgu @ w13
    dw13 = dgu.t() @ x
    dw2 = dy.t() @ h
    res["dx"] = (dx, edgu @ w13.abs() + sum_err(dgu.abs() @ w13.abs(), 2 * I) + 2 * U16 * dx.abs())
    res["dw13"] = (dw13, edgu.t() @ x.abs() + sum_err(dgu.abs().t() @ x.abs(), T) + 2 * U16 * dw13.abs())
    res["dw2"] = (dw2, dy.abs().t() @ eh + sum_err(dy.abs().t() @ h.abs(), T) + 2 * U16 * dw2.abs())
    return res


def check(got, ref, bound, what, l2=None):
    """Every element within its bound (a tiny absolute floor for bf16's smallest values), and the whole within l2."""
    got = got.double()
    assert got.shape == ref.shape, what
    d = (got - ref).abs()
    bad = ~(d <= bound + 1e-37)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} elements past their bound, worst {float((d / (bound + 1e-37)).max()):.3g}x"
    if l2 is not None and float(ref.norm()) > 0:
        rel = float(d.norm() / ref.norm())
        assert rel <= l2, f"{what}: relative L2 {rel:.3g} > {l2:.3g}"
