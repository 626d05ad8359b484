"""GPU tests of the dense products where their kernel or cut changes with the
size, and where offsets pass 32 bits: against 64-bit products within the
bounds of tests/plain64.py."""
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


def _weight(seed, N, K):
    g = _gen(seed)
    return (torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8),
            torch.randint(117, 124, (N, K // 32), generator=g, device=DEV, dtype=torch.uint8))


def _check_linear(T, K, N, act):
    print(f"[linear_mxfp4 {act} T={T} K={K} N={N}]", flush=True)
    codes, scales = _weight(K + N, N, K)
    x = _bf16(T, T, K)
    xe = plain64.mxfp4_round(x) if act == "mxfp4" else x.double()
    ref, bound = plain64.linear(xe, plain64.exact_values(codes, scales), U32)
    out = mx.linear_mxfp4(x, codes, scales, act=act, out_fp32=True)
    check(out, ref, bound, "fp32", l2=1e-5)
    assert torch.equal(mx.linear_mxfp4(x, codes, scales, act=act), out.to(torch.bfloat16))


# around the sizes where streaming ends and the tile product begins
@pytest.mark.parametrize("T,K", [(64, 2048), (65, 2048), (63, 2080), (64, 2080), (32, 4096), (33, 4096), (16, 8192),
                                 (17, 8192), (2, 65536), (3, 65536), (24, 4096), (25, 4096), (12, 8192), (13, 8192), (32, 3008),
                                 (33, 3008), (1, 65536)])
def test_linear_streamed_or_tiled(T, K):
    _check_linear(T, K, 272, "bf16")


@pytest.mark.parametrize("T,K", [(32, 1024), (33, 1024), (24, 4096), (25, 4096), (12, 8192), (13, 8192), (1, 65536),
                                 (2, 65536), (20, 4096), (21, 4096), (10, 8192), (11, 8192), (32, 2560), (33, 2560)])
def test_linear_mxfp4_rows_streamed_or_tiled(T, K):
    _check_linear(T, K, 272, "mxfp4")


# weights read as codes, then expanded first; tiles of 64, 128 and 256 rows; K split and whole
@pytest.mark.parametrize("T,K,N", [(80, 8192, 520), (160, 4096, 4096), (520, 2048, 2048), (900, 4096, 2048),
                                   (1400, 2048, 4096), (1900, 2048, 4096), (2600, 1056, 4096), (6000, 544, 2056)])
@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
def test_linear_cuts(T, K, N, act):
    _check_linear(T, K, N, act)


@pytest.mark.parametrize("T,H,I", [(42, 4096, 2048), (43, 4096, 2048), (32, 1024, 4096), (33, 1024, 4096),
                                   (64, 2048, 1024), (65, 2048, 1024), (500, 1024, 2048), (1500, 2048, 2048),
                                   (24, 4096, 2048), (25, 4096, 2048), (8, 1024, 4096), (9, 1024, 4096), (12, 1024, 4096),
                                   (32, 2048, 1024), (33, 2048, 1024)])
def test_ffn_streamed_or_tiled(T, H, I):
    print(f"[gated_ffn T={T} H={H} I={I}]", flush=True)
    x, w13 = _bf16(T, T, H), _bf16(H, 2 * I, H, scale=1.3 / math.sqrt(H))
    w2 = _bf16(I, H, I, scale=1 / math.sqrt(I))
    ref = plain64.ffn(x.double(), w13.double(), w2.double(), 10.0)
    check(mx.gated_ffn(x, w13, w2), *ref["y"], "y", l2=2 * U16)


@pytest.mark.parametrize("T,H,I", [(1, 4096, 2048), (1, 256, 128), (7, 264, 136), (16, 1024, 512), (17, 2048, 72),
                                   (33, 512, 1024), (64, 2048, 1024)])
def test_ffn_streamed_keeps_sixteen_bits_of_h(T, H, I):
    """Streamed rows (up to 32 here): h = hi + lo, each rounded by at most a half step of bf16 of what is left, 2^-16 of
    h together; with random signs the fp32 output is within that of its norm (beside 2^-20 of the activation, 1e-6 of
    the sums). More rows run as tile products with h in one bf16: a half step, 2^-8, of each of its values."""
    x, w13 = _bf16(T, T, H), _bf16(H, 2 * I, H, scale=1.3 / math.sqrt(H))
    w2 = _bf16(I, H, I, scale=1 / math.sqrt(I))
    y, bound = plain64.ffn(x.double(), w13.double(), w2.double(), 10.0)["y"]
    out = mx.gated_ffn(x, w13, w2, out_fp32=True)
    check(out, y, bound, "fp32", l2=2.0 ** -15 if T <= 32 else U16)
    saving, (_, h) = mx.gated_ffn(x, w13, w2, save=True, out_fp32=True)
    assert torch.equal(saving, out)
    I0 = w13[:I].double(), w13[I:].double()
    g, u = (x.double() @ w.t() for w in I0)
    h64 = torch.nn.functional.silu(g.clamp(max=10.0)) * u.clamp(-10.0, 10.0)
    assert float((h.double() - h64).norm() / h64.norm()) <= U16


def test_ffn_streamed_infinite_h():
    """h past bf16's largest value: the output keeps its infinities apart from NaN, as bf16 operands would."""
    H = I = 8
    x = torch.zeros(2, H, dtype=torch.bfloat16, device=DEV)
    x[0, 0], x[1, 1] = 3e38, 1.0
    w13 = torch.zeros(2 * I, H, dtype=torch.bfloat16, device=DEV)
    w13[:I, 0], w13[:I, 1], w13[I:, 0], w13[I:, 1] = 1.0, 1.0, 1.0, 1.0
    w2 = torch.ones(H, I, dtype=torch.bfloat16, device=DEV)
    y = mx.gated_ffn(x, w13, w2, limit=math.inf)
    assert bool((y[0] == math.inf).all())
    assert bool(torch.isfinite(y[1]).all())


# the backward's products two to a launch, with every tile, and one to a launch with K split
@pytest.mark.parametrize("T,H,I", [(2, 64, 4096), (70, 4096, 64), (400, 512, 512), (700, 1024, 1024),
                                   (1500, 2048, 1024), (2000, 1024, 4096), (3000, 4096, 2048), (5000, 256, 264)])
def test_ffn_backward_cuts(T, H, I):
    print(f"[gated_ffn_backward T={T} H={H} I={I}]", flush=True)
    x, w13 = _bf16(T, T, H), _bf16(H, 2 * I, H, scale=1.3 / math.sqrt(H))
    w2, dy = _bf16(I, H, I, scale=1 / math.sqrt(I)), _bf16(T + 1, T, H, scale=0.1)
    ref = plain64.ffn(x.double(), w13.double(), w2.double(), 10.0, dy.double())
    y, saved = mx.gated_ffn(x, w13, w2, save=True)
    for name, got in zip(("dx", "dw13", "dw2"), mx.gated_ffn_backward(dy, x, w13, w2, saved)):
        check(got, *ref[name], name, l2=2 * U16)


# ---------------------------------------------------------------- offsets past 32 bits

ROWS = torch.tensor([0, 1, 16383, 32767, 32768, 40000, 65534, 65535])


def test_linear_long_output():
    T, K, N = 65536, 64, 65536  # out: 2^32 values
    codes, scales = _weight(1, N, K)
    W = plain64.exact_values(codes, scales)
    x = _bf16(2, T, K)
    rows = ROWS.to(DEV)
    for act in ("bf16", "mxfp4"):
        xe = plain64.mxfp4_round(x[rows]) if act == "mxfp4" else x[rows].double()
        out = mx.linear_mxfp4(x, codes, scales, act=act)
        check(out[rows], *plain64.linear(xe, W), act)
        del out
    codes, scales = _weight(3, K, N)  # the gradient's long side: dx [T][65536]
    dy = _bf16(4, T, K)
    dx = mx.linear_mxfp4_dx(dy, codes, scales)
    check(dx[rows], *plain64.linear(dy[rows].double(), plain64.exact_values(codes, scales).t()), "dx")


def test_quantize_long_tensors():
    rows, K = 70000, 32768  # 2.3e9 values
    x = torch.empty(rows, K, dtype=torch.bfloat16, device=DEV)
    for i in range(0, rows, 10000):
        x[i:i + 10000] = _bf16(i, min(10000, rows - i), K)
    codes, scales = mx.quantize_mxfp4(x)
    pick = torch.tensor([0, 32767, 65535, 65536, 69999], device=DEV)
    part = mx.quantize_mxfp4(x[pick].contiguous())
    assert torch.equal(codes[pick], part[0]) and torch.equal(scales[pick], part[1])
    del x
    back = mx.dequantize_mxfp4(codes, scales)
    assert torch.equal(back[pick], mx.dequantize_mxfp4(*part))
    del back
    # few values, far apart: the last row starts at element 2.6e9
    wide = torch.zeros(40000 * 65544, dtype=torch.bfloat16, device=DEV).view(40000, 65544)
    wide[:, 8:72] = _bf16(5, 40000, 64)
    far = mx.quantize_mxfp4(wide[:, 8:72])
    near = mx.quantize_mxfp4(wide[:, 8:72].contiguous())
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])


def test_ffn_long_batch():
    T, H, I = 65536, 64, 16384  # g and u: 2^31 values
    x, w13 = _bf16(1, T, H), _bf16(2, 2 * I, H, scale=1.3 / math.sqrt(H))
    w2, dy = _bf16(3, H, I, scale=1 / math.sqrt(I)), _bf16(4, T, H, scale=0.1)
    y, saved = mx.gated_ffn(x, w13, w2, save=True)
    dx, dw13, dw2 = mx.gated_ffn_backward(dy, x, w13, w2, saved)
    rows = ROWS.to(DEV)
    ref = plain64.ffn(x[rows].double(), w13.double(), w2.double(), 10.0, dy[rows].double())
    check(y[rows], *ref["y"], "y", l2=2 * U16)
    check(dx[rows], *ref["dx"], "dx", l2=2 * U16)
    # the weights' gradients, column by column of the block: h and the gradients of g and u need that column only
    cols = torch.tensor([0, 17, 8191, 8192, 16383], device=DEV)
    w13c = w13.view(2, I, H)[:, cols].reshape(-1, H)
    ref = plain64.ffn(x.double(), w13c.double(), w2[:, cols].double(), 10.0, dy.double())
    check(dw13.view(2, I, H)[:, cols].reshape(-1, H), *ref["dw13"], "dw13", l2=2 * U16)
    check(dw2[:, cols], *ref["dw2"], "dw2", l2=2 * U16)


def test_every_path_captured_and_replayed():
    """Each kernel family captured into a graph of its own (its first launch at that size) and replayed with eager
    calls of the same between the replays."""
    calls = []
    for T, K, N, act in [(1, 256, 64, "bf16"), (100, 1024, 512, "bf16"), (700, 1024, 512, "bf16"),
                         (3000, 1024, 2048, "bf16"), (20, 512, 96, "mxfp4"), (300, 1024, 512, "mxfp4"),
                         (5000, 1024, 4096, "mxfp4")]:
        codes, scales = _weight(K, N, K)
        x = _bf16(T, T, K)
        calls.append(lambda x=x, c=codes, s=scales, act=act: (mx.linear_mxfp4(x, c, s, act=act),))
        if act == "bf16":
            dy = _bf16(T + 1, T, N)
            calls.append(lambda dy=dy, c=codes, s=scales: (mx.linear_mxfp4_dx(dy, c, s),))
    for T, H, I in [(2, 256, 128), (200, 512, 256), (1500, 512, 1024), (4000, 2048, 2048)]:
        x, w13 = _bf16(T, T, H), _bf16(H, 2 * I, H, scale=1.3 / math.sqrt(H))
        w2, dy = _bf16(I, H, I, scale=1 / math.sqrt(I)), _bf16(T + 1, T, H, scale=0.1)

        def step(x=x, w13=w13, w2=w2, dy=dy):
            y, saved = mx.gated_ffn(x, w13, w2, save=True)
            return (y,) + mx.gated_ffn_backward(dy, x, w13, w2, saved)

        calls.append(step)
    rows = _bf16(9, 70, 96)
    calls.append(lambda: mx.quantize_mxfp4(rows))
    torch.cuda.synchronize()
    graphs = []
    for call in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, out))
    for rep in range(3):
        for g, out in graphs:
            for t in out:
                t.zero_()
            g.replay()
        eager = [call() for call in calls]
        torch.cuda.synchronize()
        for i, ((_, out), ref) in enumerate(zip(graphs, eager)):
            assert all(torch.equal(a, b) for a, b in zip(out, ref)), (rep, i)
