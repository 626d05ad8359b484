"""GPU tests of the MXFP4 products and the gated block at sizes that reach the
kernel variants the other tests do not: every number of waves of the streaming
pass (it takes at most 32 rows; K and the number of weight rows decide the
rest), and every tile with K split and whole. Against 64 bits within the bounds
of tests/plain64.py."""
import math

import pytest
import torch

import plain64
from plain64 import U16, U32, check

pytestmark = pytest.mark.gpu
mx = pytest.importorskip("mxfp4_moe_expert_amd")
DEV = "cuda"


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _bf16(seed, *shape, scale=1.0):
    return (torch.randn(*shape, generator=_gen(seed), device=DEV) * scale).to(torch.bfloat16)


def _weight(seed, N, K, lo=117, hi=124):
    g = _gen(seed)
    return (torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8),
            torch.randint(lo, hi, (N, K // 32), generator=g, device=DEV, dtype=torch.uint8))


def _linear(T, K, N, act, **kw):
    print(f"[linear_mxfp4 {act} T={T} K={K} N={N}]", flush=True)
    codes, scales = _weight(K + N, N, K, **kw)
    x = _bf16(T, T, K)
    xe = plain64.mxfp4_round(x) if act == "mxfp4" else x.double()
    ref, bound = plain64.linear(xe, plain64.exact_values(codes, scales), U32)
    out = mx.linear_mxfp4(x, codes, scales, act=act, out_fp32=True)
    check(out, ref, bound, "fp32", l2=1e-5)
    assert torch.equal(mx.linear_mxfp4(x, codes, scales, act=act), out.to(torch.bfloat16))


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,K,N", [(1, 96, 5124), (3, 544, 6000), (16, 2080, 10240), (17, 96, 5137), (20, 2080, 6001),
                                   (32, 512, 10001), (1, 96, 10242), (3, 544, 12000), (20, 288, 12001)])
def test_linear_streamed_by_fewer_waves(T, K, N, act):
    _linear(T, K, N, act)


# the product on W's codes with 256-row tiles and K split; on W expanded, K split, with each tile
@pytest.mark.parametrize("T,K,N", [(541, 6976, 2624), (1163, 6496, 131), (2925, 6208, 129), (5339, 5600, 131),
                                   (4254, 13376, 130), (4159, 2656, 129)])
def test_linear_split_tiles(T, K, N):
    _linear(T, K, N, "bf16")


@pytest.mark.parametrize("T,K,N", [(204, 3648, 90), (710, 21632, 129), (4228, 24800, 130)])
def test_linear_mxfp4_rows_split_tiles(T, K, N):
    _linear(T, K, N, "mxfp4")


@pytest.mark.parametrize("T,K,N", [(200, 96, 931), (715, 160, 8234), (1217, 160, 28162), (8518, 160, 18923)])
def test_linear_dx_split_tiles(T, K, N):
    print(f"[linear_mxfp4_dx T={T} K={K} N={N}]", flush=True)
    codes, scales = _weight(K + N, N, K)
    dy = _bf16(T, T, N)
    ref, bound = plain64.linear(dy.double(), plain64.exact_values(codes, scales).t(), U32)
    out = mx.linear_mxfp4_dx(dy, codes, scales, out_fp32=True)
    check(out, ref, bound, "fp32", l2=1e-5)
    assert torch.equal(mx.linear_mxfp4_dx(dy, codes, scales), out.to(torch.bfloat16))


def _block(T, H, I):
    return (_bf16(T, T, H), _bf16(H, 2 * I, H, scale=1.3 / math.sqrt(H)), _bf16(I, H, I, scale=1 / math.sqrt(I)),
            _bf16(T + 1, T, H, scale=0.1))


# streamed by 8 and 4 waves a block, for gate and up (by I) and down (by H); then gate and down products of a split K
@pytest.mark.parametrize("T,H,I", [(4, 264, 6000), (17, 72, 2568), (18, 136, 3000), (4, 5512, 136), (12, 5512, 136),
                                   (18, 5512, 72), (3, 10400, 72), (9, 10272, 72), (72, 6688, 712), (2757, 11200, 72),
                                   (66, 1448, 6696), (4242, 72, 12328), (4163, 136, 12320)])
def test_ffn(T, H, I):
    print(f"[gated_ffn T={T} H={H} I={I}]", flush=True)
    x, w13, w2, _ = _block(T, H, I)
    ref = plain64.ffn(x.double(), w13.double(), w2.double(), 10.0)
    y = mx.gated_ffn(x, w13, w2)
    check(y, *ref["y"], "y", l2=2 * U16)
    y32, (gu, h) = mx.gated_ffn(x, w13, w2, save=True, out_fp32=True)
    assert torch.equal(y32.to(torch.bfloat16), y)
    g = torch.cat((x.double() @ w13[:I].double().t(), x.double() @ w13[I:].double().t()), 1)
    check(gu, g, plain64.sum_err(x.double().abs() @ w13.double().abs().t(), H), "gu")


# pairs of products by the tile they share; single products whole and of a split K by tile
@pytest.mark.parametrize("T,H,I", [(1, 1056, 13712), (486, 8, 7184), (66, 136, 15888), (65, 11104, 136), (11157, 72, 656),
                                   (10881, 72, 264), (11329, 72, 136), (65, 6664, 1424), (4299, 12472, 72),
                                   (1226, 136, 12128), (66, 1560, 3112), (11383, 72, 2072), (5664, 136, 376),
                                   (13351, 136, 2056)])
def test_ffn_backward(T, H, I):
    print(f"[gated_ffn_backward T={T} H={H} I={I}]", flush=True)
    x, w13, w2, dy = _block(T, H, I)
    ref = plain64.ffn(x.double(), w13.double(), w2.double(), 10.0, dy.double())
    y, saved = mx.gated_ffn(x, w13, w2, save=True)
    got = mx.gated_ffn_backward(dy, x, w13, w2, saved)
    for name, t in zip(("dx", "dw13", "dw2"), got):
        check(t, *ref[name], name, l2=2 * U16)
    for need in ((True, False, False), (False, True, False), (False, False, True)):
        part = mx.gated_ffn_backward(dy, x, w13, w2, saved, need=need)
        assert all((p is None) == (not n) and (p is None or torch.equal(p, t)) for n, p, t in zip(need, part, got))
