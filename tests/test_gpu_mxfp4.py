"""GPU tests of the MXFP4 conversions and plain products: every code against
the CPU encoder and the 64-bit definition, products against 64-bit products
within the bounds of tests/plain64.py."""
import numpy as np
import pytest
import torch

import oracle
import plain64
import synth
from plain64 import U16, U32, check

pytestmark = pytest.mark.gpu
mx = pytest.importorskip("mxfp4_moe_expert_amd")
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}


def _rand(seed, *shape, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV) * scale


def _weight(seed, N, K):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(117, 124, (N, K // 32), generator=g, device=DEV, dtype=torch.uint8)
    return codes, scales


# ---------------------------------------------------------------- conversions

@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (7, 4096), (64, 2080), (1000, 160), (129, 8192)])
def test_quantize_codes_and_values(rows, K, dtype):
    x = (_rand(rows + K, rows, K) * torch.exp2(_rand(1, rows, 1, scale=4.0))).to(DT[dtype])
    codes, scales = mx.quantize_mxfp4(x)
    want = plain64.mxfp4_round(x)
    assert torch.equal(plain64.exact_values(codes, scales), want)
    c, s = synth.quant_mxfp4(x.float().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)  # signs of zeros among them
    assert torch.equal(mx.dequantize_mxfp4(codes, scales, dtype=torch.float32).double(), want)
    assert torch.equal(mx.dequantize_mxfp4(codes, scales).double(), want)


def test_quantize_ties_borders_and_extremes():
    """Every midpoint of the E2M1 grid and its fp32 neighbours, at the smallest, ordinary and largest exponents;
    groups of zeros, of subnormals, and with the largest finite values."""
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    vals = [v for m in mids for v in (m, np.nextafter(np.float32(m), np.float32(0)),
                                      np.nextafter(np.float32(m), np.float32(9)))] + [4.0, 6.0, 7.999999, 0.0, 1e-7]
    row = np.array((vals + [-v for v in vals])[:64], dtype=np.float32)
    row = np.pad(row, (0, 64 - len(row)), constant_values=4.0)
    row[0] = row[32] = 4.0  # the group maximum: exponent 2
    rows = [np.ldexp(row, e).astype(np.float32) for e in (-140, -128, -127, -126, -125, -60, 0, 60, 124, 125)]
    rows.append(np.zeros(64, np.float32))
    rows.append(-np.zeros(64, np.float32))
    rows.append(np.full(64, np.float32(1e-45)))
    rows.append(np.full(64, np.finfo(np.float32).max))
    x = torch.from_numpy(np.stack(rows)).to(DEV)
    codes, scales = mx.quantize_mxfp4(x)
    c, s = synth.quant_mxfp4(x.cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)
    assert torch.equal(mx.dequantize_mxfp4(codes, scales, dtype=torch.float32).double(), plain64.mxfp4_round(x))


@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_non_finite_groups(dtype):
    x = _rand(5, 4, 128).to(DT[dtype])
    x[0, 40] = float("nan")
    x[1, 0] = float("inf")
    x[2, 127] = float("-inf")
    codes, scales = mx.quantize_mxfp4(x)
    want = plain64.mxfp4_round(x)
    bad = torch.zeros(4, 4, dtype=torch.bool, device=DEV)
    bad[0, 1] = bad[1, 0] = bad[2, 3] = True
    assert torch.equal(scales == 255, bad)
    assert bool((codes.reshape(4, 4, 16)[bad] == 0).all())
    for dt in (torch.float32, torch.bfloat16):
        got = mx.dequantize_mxfp4(codes, scales, dtype=dt).double()
        assert torch.equal(torch.isnan(got), bad.repeat_interleave(32, dim=1))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


def test_dequantize_every_code_and_scale():
    """All 16 codes under all 256 scale bytes, in fp32 and bf16."""
    codes = torch.tensor([c | (((c + 1) & 15) << 4) for c in range(16)], dtype=torch.uint8, device=DEV).repeat(256, 1)
    scales = torch.arange(256, device=DEV).to(torch.uint8).reshape(256, 1)
    want = plain64.exact_values(codes, scales)
    over = want.abs() > torch.finfo(torch.float32).max  # 4 and 6 times 2^127: past fp32
    for dt in (torch.float32, torch.bfloat16):
        got = mx.dequantize_mxfp4(codes, scales, dtype=dt).double()
        keep = ~over & ~torch.isnan(want)
        assert torch.equal(got[keep], want[keep])
        assert bool(torch.isnan(got[torch.isnan(want)]).all())


def test_quantize_strided_rows_and_shapes():
    big = _rand(9, 50, 256).to(torch.bfloat16)
    view = big[3:40, 32:192]
    a, b = mx.quantize_mxfp4(view)
    c, d = mx.quantize_mxfp4(view.contiguous())
    assert torch.equal(a, c) and torch.equal(b, d)
    w = _rand(10, 3, 8, 64)
    a, b = mx.quantize_mxfp4(w)
    assert a.shape == (3, 8, 32) and b.shape == (3, 8, 2)
    c, d = mx.quantize_mxfp4(w.reshape(24, 64))
    assert torch.equal(a.reshape(24, 32), c)
    e = mx.quantize_mxfp4(torch.empty(0, 64, device=DEV))
    assert e[0].shape == (0, 32) and mx.dequantize_mxfp4(*e).shape == (0, 64)


def test_quantize_refusals_on_device():
    x = _rand(1, 8, 64)
    with pytest.raises(ValueError):
        mx.quantize_mxfp4(x[:, :48])
    with pytest.raises(ValueError):
        mx.quantize_mxfp4(x.t())
    with pytest.raises(TypeError):
        mx.quantize_mxfp4(x.double())
    with pytest.raises(mx.MoEError):
        mx.quantize_mxfp4(_rand(1, 8, 65)[:, :64])  # rows not 16-byte aligned
    c, s = mx.quantize_mxfp4(x)
    with pytest.raises(ValueError):
        mx.dequantize_mxfp4(c, s[:4])
    with pytest.raises(TypeError):
        mx.linear_mxfp4(x, c, s)                    # fp32 activations
    with pytest.raises(ValueError):
        mx.linear_mxfp4(x[:, :32].to(torch.bfloat16).contiguous(), c, s)
    with pytest.raises(mx.MoEError):
        mx.linear_mxfp4(torch.zeros(100, 64, dtype=torch.bfloat16, device=DEV), c, s, act="mxfp4",
                        ws=torch.empty(256, dtype=torch.uint8, device=DEV))


# ---------------------------------------------------------------- products

# The streaming pass ends at 32 rows, or earlier by size: 33 and 64 rows below run as tile products. Its variants by
# waves, and the tiles with K split, are in test_gpu_dense_variants.py.
SHAPES = [  # T, K, N: the streaming pass (1 .. 64), then every tile size and splits of K
    (1, 32, 1), (1, 4096, 1536), (1, 96, 17), (2, 8192, 256), (15, 2080, 100), (16, 4096, 4096), (17, 512, 12000),
    (32, 1024, 48), (33, 8192, 640), (64, 2048, 1000), (64, 288, 20000),
    (65, 32, 16), (65, 4096, 1536), (100, 2048, 4096), (129, 160, 130), (200, 8192, 256), (300, 4096, 4096),
    (257, 2080, 259), (513, 1024, 1023), (1000, 4096, 4096), (2048, 544, 2050), (4100, 1024, 4096),
]


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_linear_mxfp4(T, K, N, act):
    print(f"[linear_mxfp4 {act} T={T} K={K} N={N}]", flush=True)
    codes, scales = _weight(K + N, N, K)
    x = _rand(T, T, K).to(torch.bfloat16)
    W = plain64.exact_values(codes, scales)
    xe = plain64.mxfp4_round(x) if act == "mxfp4" else x.double()
    out32 = mx.linear_mxfp4(x, codes, scales, act=act, out_fp32=True)
    ref, bound = plain64.linear(xe, W, U32)
    check(out32, ref, bound, "fp32", l2=1e-5)  # random signs: far below the worst case of the bound
    out16 = mx.linear_mxfp4(x, codes, scales, act=act)
    assert torch.equal(out16, out32.to(torch.bfloat16))
    assert torch.equal(out32, mx.linear_mxfp4(x, codes, scales, act=act, out_fp32=True))  # repeatable


@pytest.mark.parametrize("T,K,N", [(1, 32, 1), (1, 4096, 1536), (5, 96, 7), (64, 2048, 1000), (100, 160, 4096),
                                   (129, 2080, 130), (300, 4096, 4096), (777, 1024, 513), (2048, 4096, 2048),
                                   (4100, 512, 1024)])
def test_linear_mxfp4_dx(T, K, N):
    print(f"[linear_mxfp4_dx T={T} K={K} N={N}]", flush=True)
    codes, scales = _weight(K + N, N, K)
    dy = _rand(T, T, N).to(torch.bfloat16)
    W = plain64.exact_values(codes, scales)
    ref, bound = plain64.linear(dy.double(), W.t(), U32)
    out32 = mx.linear_mxfp4_dx(dy, codes, scales, out_fp32=True)
    check(out32, ref, bound, "fp32", l2=1e-5)
    assert torch.equal(mx.linear_mxfp4_dx(dy, codes, scales), out32.to(torch.bfloat16))


def test_linear_dx_is_the_gradient_of_the_product():
    """<linear(x), dy> = <x, linear_dx(dy)> for x, dy of small integers (every sum exact in fp32), and central
    differences of the product (exact for a linear map) along random directions."""
    T, K, N = 70, 96, 40
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.full((N, K // 32), 127, dtype=torch.uint8, device=DEV)
    x, v = (torch.randint(-3, 4, (T, K), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    dy = torch.randint(-3, 4, (T, N), generator=g, device=DEV).to(torch.bfloat16)
    dx = mx.linear_mxfp4_dx(dy, codes, scales, out_fp32=True).double()
    f = [(mx.linear_mxfp4(x + s * v, codes, scales, out_fp32=True).double() * dy.double()).sum() for s in (1, -1)]
    assert float((f[0] - f[1]) / 2) == float((dx * v.double()).sum())


@pytest.mark.parametrize("T", [3, 100])
@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
def test_linear_non_finite_stay_in_their_rows_and_columns(T, act):
    K, N = 288, 70
    codes, scales = _weight(1, N, K)
    x = _rand(2, T, K).to(torch.bfloat16)
    clean = mx.linear_mxfp4(x, codes, scales, act=act)
    x2 = x.clone()
    x2[1, 5] = float("nan")
    x2[2, 287] = float("inf")
    got = mx.linear_mxfp4(x2, codes, scales, act=act)
    assert bool(torch.isnan(got[1]).all())
    assert not bool(torch.isfinite(got[2]).any())
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(got[keep], clean[keep])
    s2 = scales.clone()
    s2[7, 8] = 255
    got = mx.linear_mxfp4(x, codes, s2, act=act)
    assert bool(torch.isnan(got[:, 7]).all())
    cols = [n for n in range(N) if n != 7]
    assert torch.equal(got[:, cols], clean[:, cols])


@pytest.mark.parametrize("T,K,N", [(5, 96, 19), (100, 160, 131), (300, 4096, 1000)])
@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
def test_linear_writes_its_output_only(T, K, N, act):
    """Outputs inside a larger buffer, workspace of exactly the stated size inside another filled with NaN patterns:
    nothing around either changes, and stale workspace contents do not reach the result."""
    codes, scales = _weight(1, N, K)
    x = _rand(2, T, K).to(torch.bfloat16)
    ref = mx.linear_mxfp4(x, codes, scales, act=act)
    buf = torch.full((T * N + 256,), 7.0, dtype=torch.bfloat16, device=DEV)
    need = mx.lib().moe_linear_mxfp4_workspace_size(T, K, N, mx._ACTS[act])
    wsb = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=DEV)
    off = (-wsb.data_ptr()) % 256
    ws = wsb[off:off + need]
    out = buf[:T * N].view(T, N)
    mx.linear_mxfp4(x, codes, scales, act=act, out=out, ws=ws)
    assert torch.equal(out, ref)
    assert bool((buf[T * N:] == 7.0).all())
    assert bool((wsb[off + need:] == 0xFF).all()) and bool((wsb[:off] == 0xFF).all())


def test_linear_empty_batch():
    codes, scales = _weight(1, 16, 64)
    assert mx.linear_mxfp4(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), codes, scales).shape == (0, 16)
    assert mx.linear_mxfp4_dx(torch.empty(0, 16, dtype=torch.bfloat16, device=DEV), codes, scales).shape == (0, 64)


def test_linear_on_two_streams_and_in_graphs():
    """Calls on two streams at once, and two captured graphs replayed with eager calls between: every result equals
    the eager one (the scratch of a call is its own)."""
    T, K, N = 200, 2048, 1024
    codes, scales = _weight(1, N, K)
    xs = [_rand(10 + i, T, K).to(torch.bfloat16) for i in range(4)]
    dys = [_rand(20 + i, T, N).to(torch.bfloat16) for i in range(4)]

    def step(i):
        return (mx.linear_mxfp4(xs[i], codes, scales), mx.linear_mxfp4(xs[i], codes, scales, act="mxfp4"),
                mx.linear_mxfp4_dx(dys[i], codes, scales), mx.linear_mxfp4(xs[i][:9].contiguous(), codes, scales))

    ref = [step(i) for i in range(4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None] * 4
    for i in range(4):
        with torch.cuda.stream(streams[i % 2]):
            got[i] = step(i)
    torch.cuda.synchronize()
    for i in range(4):
        assert all(torch.equal(a, b) for a, b in zip(got[i], ref[i])), i
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(i))
        graphs.append(g)
    for rep in range(3):
        for i in range(2):
            for o in outs[i]:
                o.zero_()
        for g in graphs:
            g.replay()
        eager = step(2)
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], ref[i])), (rep, i)
        assert all(torch.equal(a, b) for a, b in zip(eager, ref[2])), rep
        xs[2].add_(0)  # eager work between replays


# ---------------------------------------------------------------- together, as a user has them

def test_encoded_weights_run_in_the_layer():
    """fp32 expert weights encoded here go into the layer's expert pass: equal to the pass on the CPU encoder's
    bytes, and one expert's own products through linear_mxfp4 give the same block (the pass rounds h to bf16)."""
    H, I, E, k, T = 256, 128, 16, 6, 24
    cfg = mx.config(hidden_size=H, n_routed_experts=E, top_k=k, moe_intermediate=I)
    w13 = _rand(1, E, 2 * I, H, scale=0.05)
    w2 = _rand(2, E, H, I, scale=0.05)
    x = _rand(3, T, H).to(torch.bfloat16)
    c13, s13 = mx.quantize_mxfp4(w13)
    c2, s2 = mx.quantize_mxfp4(w2)
    hc, hs = synth.quant_mxfp4(w13.reshape(-1, H).cpu().numpy())
    assert np.array_equal(c13.cpu().numpy().reshape(hc.shape), hc) and np.array_equal(s13.cpu().numpy().reshape(hs.shape), hs)
    ids = torch.arange(k, dtype=torch.int32, device=DEV).repeat(T, 1)
    w = torch.full((T, k), 1.0 / k, dtype=torch.float32, device=DEV)
    off, slots, _ = mx.permute(cfg, ids)
    got = mx.expert_ffn(cfg, x, off, slots, w, c13, s13, c2, s2)
    ref = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for e in range(k):
        gu = mx.linear_mxfp4(x, c13[e], s13[e], out_fp32=True)
        g, u = gu[:, :I].double(), gu[:, I:].double()
        h = (torch.nn.functional.silu(g.clamp(max=10)) * u.clamp(-10, 10)).to(torch.bfloat16)
        ref += mx.linear_mxfp4(h, c2[e], s2[e], out_fp32=True).double() / k
    rel = float((got.double() - ref).norm() / ref.norm())
    assert rel <= 2 * U16, rel  # both round h to bf16: a value near a tie may fall either way
