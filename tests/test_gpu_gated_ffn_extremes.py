"""GPU tests of the gated block at values far from the ordinary: gates past
2^24 under limits that let them through."""
import math

import pytest
import torch

from plain64 import U16, sum_err

pytestmark = pytest.mark.gpu
mx = pytest.importorskip("mxfp4_moe_expert_amd")
DEV = "cuda"


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("limit", [math.inf, 2.0 ** 40])
# dgu's product in one launch with dw2's, alone (need: dx only), and of a split K (its reduction's epilogue)
@pytest.mark.parametrize("T,H,I,need", [(48, 64, 96, (True, True, True)), (48, 64, 96, (True, True, False)),
                                        (20, 4096, 72, (True, True, True)), (300, 512, 1024, (True, True, True))])
def test_gradients_of_large_gates(T, H, I, need, limit):
    """silu' is 1 at every large g: s = 1 there, and nothing of g may be left over.

    Each token reads one column of w13 (x is a one there), so g and u are bf16 values without an error, and
    dw13 in fp32 holds the block's dg and du as it rounded them. dy and w2 are small integers: dh is exact.
    With silu' = s + t (1 - s), t = g s, in fp32: the exponential's argument, the exponential and the reciprocal put
    (|g| + 4) 2^-24 on s (1 - s), 1 - s is off by half a step of s, 2^-24, times |t|, and the two sums by a step:
    at |g| <= 32 below (1 + 32) 36 / 4 + 32 + 4 < 2^9 steps of 2^-24, 2^-15 in all. Above 64, s is 1 and silu' as well."""
    g_ = _gen(T + H)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    cols = (torch.arange(T, device=DEV) * 7) % H if H % 7 else torch.arange(T, device=DEV)
    x[torch.arange(T, device=DEV), cols] = 1.0
    low = torch.randint(-2, 5, (I, H), generator=g_, device=DEV)
    high = torch.randint(20, 37, (I, H), generator=g_, device=DEV)
    e = torch.where(torch.rand(I, H, generator=g_, device=DEV) < 0.5, low, high)
    sign = torch.randint(0, 2, (2 * I, H), generator=g_, device=DEV) * 2 - 1
    mant = 1 + torch.randint(0, 128, (2 * I, H), generator=g_, device=DEV) / 128
    w13 = mant * sign
    w13[:I] = torch.ldexp(w13[:I], e)
    w13 = w13.to(torch.bfloat16)  # mantissas of 8 bits: exact
    w13[0, cols[:4]] = torch.tensor([2.0 ** 24, 3e7, 1e9, 1e10], device=DEV).to(torch.bfloat16)
    w2 = torch.randint(-2, 3, (H, I), generator=g_, device=DEV).to(torch.bfloat16)
    dy = torch.randint(-3, 4, (T, H), generator=g_, device=DEV).to(torch.bfloat16)
    y, saved = mx.gated_ffn(x, w13, w2, limit=limit, save=True)
    g, u = w13[:I].double()[:, cols].t(), w13[I:].double()[:, cols].t()
    assert torch.equal(saved[0].double(), torch.cat((g, u), 1))
    assert int((g > 2.0 ** 24).sum()) > T * I // 8
    dx, dw13, dw2 = mx.gated_ffn_backward(dy, x, w13, w2, saved, limit=limit, need=need, dw_fp32=True)
    s = torch.sigmoid(g)
    d1 = torch.where(g > 64, torch.ones_like(g), s * (1 + g * (1 - s)))
    d1 = torch.where(g < -64, torch.zeros_like(g), d1)
    dh = dy.double() @ w2.double()
    dg, du = dh * u * d1, dh * g * s
    got_g, got_u = dw13[:I].double()[:, cols].t(), dw13[I:].double()[:, cols].t()
    eg = (dh * u).abs() * 2.0 ** -15 + U16 * dg.abs()
    eu = 2.0 ** -15 * (dh * g * s).abs() + U16 * du.abs()
    bad = ~((got_g - dg).abs() <= eg)
    assert not bool(bad.any()), (int(bad.sum()), g[bad][:4], (got_g / (dh * u))[bad][:4])
    assert bool(((got_u - du).abs() <= eu + 1e-30).all())
    w = w13.double()
    ref = dg @ w[:I] + du @ w[I:]
    absw = torch.cat((dg, du), 1).abs() @ w.abs()
    bound = eg @ w[:I].abs() + eu @ w[I:].abs() + sum_err(absw, 2 * I) + 2 * U16 * ref.abs()
    assert bool(((dx.double() - ref).abs() <= bound).all())


# streamed rows: h's two parts in one product's columns (up to 8 rows), as two products of one and of two token blocks,
# by blocks of 16, 8 and 4 waves; then tile products
@pytest.mark.parametrize("T,H,I", [(1, 64, 64), (5, 264, 1032), (8, 64, 136), (3, 5144, 72), (2, 10264, 72), (9, 64, 64),
                                   (16, 264, 1032), (10, 5144, 72), (9, 10272, 72), (17, 64, 64), (32, 264, 520),
                                   (18, 5144, 72), (40, 64, 64), (100, 264, 136)])
def test_infinite_down_weights(T, H, I):
    """An infinite w2[n][i] makes column n of y infinite with the sign of h[t][i], whatever the rounding of h to bf16
    leaves or however that is signed; every other column is as without it."""
    g_ = _gen(T + H + I)
    x = torch.randn(T, H, generator=g_, device=DEV).to(torch.bfloat16)
    w13 = (torch.randn(2 * I, H, generator=g_, device=DEV) * 1.3 / math.sqrt(H)).to(torch.bfloat16)
    w2 = (torch.randn(H, I, generator=g_, device=DEV) / math.sqrt(I)).to(torch.bfloat16)
    clean, (_, h) = mx.gated_ffn(x, w13, w2, save=True, out_fp32=True)
    places = [(0, 3, math.inf), (1, I - 1, -math.inf), (17, 40, -math.inf), (H - 1, I // 2, math.inf), (33, 0, math.inf)]
    bad = w2.clone()
    for n, i, v in places:
        bad[n, i] = v
    for fp32 in (True, False):
        y = mx.gated_ffn(x, w13, bad, out_fp32=fp32)
        for n, i, v in places:
            assert bool((h[:, i] != 0).all())
            want = torch.sign(h[:, i].float()) * v
            assert torch.equal(y[:, n].float(), want), (n, i, v, y[:, n][:8], want[:8])
        keep = torch.ones(H, dtype=torch.bool, device=DEV)
        keep[[n for n, _, _ in places]] = False
        assert torch.equal(y[:, keep], clean[:, keep].to(y.dtype))


@pytest.mark.parametrize("T", [1, 8, 9, 16, 17, 32, 50])
def test_products_past_the_largest_value(T):
    """h = 1029 and 1027 under weights of 3e38 and -3e38: both parts' products pass fp32's range (bf16 holds 1032 and
    1024: the rest, -3 and 3, has either sign), and y is infinite, not NaN."""
    H = I = 64
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[:, 0], x[:, 1], x[:, 2] = 1.0, 1.0, 1.0
    w13 = torch.zeros(2 * I, H, dtype=torch.bfloat16, device=DEV)
    w13[0, 0], w13[0, 1] = 1024.0, 5.0
    w13[1, 0], w13[1, 1] = 1024.0, 3.0
    w13[I:, 2] = 1.0
    w2 = torch.zeros(H, I, dtype=torch.bfloat16, device=DEV)
    w2[0, 0], w2[1, 0], w2[2, 1], w2[3, 1], w2[4, 0] = 3e38, -3e38, 3e38, -3e38, 1.0
    y = mx.gated_ffn(x, w13, w2, limit=math.inf, out_fp32=True)
    for n, v in ((0, math.inf), (1, -math.inf), (2, math.inf), (3, -math.inf)):
        assert bool((y[:, n] == v).all()), (n, y[:, n][:4])
    assert bool((y[:, 4] == (1029.0 if T <= 32 else 1032.0)).all())
    assert not bool(y[:, 5:].any())
