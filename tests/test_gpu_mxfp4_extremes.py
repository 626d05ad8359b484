"""GPU tests of the MXFP4 conversions and products at the ends of the E8M0
range: weights and activations below fp32's smallest normal value, and weights
of 2^128 and more."""
import math

import pytest
import torch

import plain64
from plain64 import U32, check

pytestmark = pytest.mark.gpu
mx = pytest.importorskip("mxfp4_moe_expert_amd")
DEV = "cuda"
K, N = 256, 272


def _inputs(seed, T, lo, hi, scale, cols=K):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(lo, hi, (N, K // 32), generator=g, device=DEV, dtype=torch.uint8)
    return codes, scales, (torch.randn(T, cols, generator=g, device=DEV) * scale).to(torch.bfloat16)


# every route: streamed, tiles on the codes, tiles on W expanded
@pytest.mark.parametrize("T", [3, 20, 100, 3000])
@pytest.mark.parametrize("lo,hi,scale", [(0, 6, 2.0 ** 100), (0, 2, 1.0), (245, 253, 2.0 ** -100), (248, 251, 2.0 ** -130)])
def test_products_at_the_ends_of_the_range(T, lo, hi, scale):
    codes, scales, x = _inputs(T, T, lo, hi, scale)
    W = plain64.exact_values(codes, scales)
    for act in ("bf16", "mxfp4"):
        xe = plain64.mxfp4_round(x) if act == "mxfp4" else x.double()
        check(mx.linear_mxfp4(x, codes, scales, act=act, out_fp32=True), *plain64.linear(xe, W, U32), act, l2=1e-5)
    _, _, dy = _inputs(T, T, lo, hi, scale, cols=N)
    check(mx.linear_mxfp4_dx(dy, codes, scales, out_fp32=True), *plain64.linear(dy.double(), W.t(), U32), "dx", l2=1e-5)


def test_values_past_fp32_decode_to_infinity():
    codes = torch.tensor([c | (((c + 1) & 15) << 4) for c in range(16)], dtype=torch.uint8, device=DEV).repeat(2, 1)
    scales = torch.tensor([[253], [254]], dtype=torch.uint8, device=DEV)
    want = plain64.exact_values(codes, scales)
    want = torch.where(want.abs() >= 2.0 ** 128, torch.sign(want) * math.inf, want)
    for dt in (torch.float32, torch.bfloat16):
        assert torch.equal(mx.dequantize_mxfp4(codes, scales, dtype=dt).double(), want)


@pytest.mark.parametrize("T", [3, 20, 100, 3000])
def test_weights_past_fp32(T):
    """As 16-bit operands they are infinite, and stay in their rows; multiplied as codes they are exact."""
    codes, scales, x = _inputs(T, T, 245, 250, 2.0 ** -100)
    clean = mx.linear_mxfp4(x, codes, scales, out_fp32=True)
    scales[7, 3] = 254
    codes[7, 48:64] = 0x77  # 6 and 6: 1.5 2^129
    y = mx.linear_mxfp4(x, codes, scales, out_fp32=True)
    assert not bool(torch.isfinite(y[:, 7]).any())
    keep = torch.arange(N, device=DEV) != 7
    assert torch.equal(y[:, keep], clean[:, keep])
    ref = plain64.linear(plain64.mxfp4_round(x), plain64.exact_values(codes, scales), U32)
    check(mx.linear_mxfp4(x, codes, scales, act="mxfp4", out_fp32=True), *ref, "mxfp4", l2=1e-5)
