"""GPU tests of the int8 conversions and the int8 x int8 product against 64-bit forms. Codes and scales have to be those
of the definition, bit for bit; the sum of a product is exact, so its fp32 value passes three roundings (the sum as fp32,
and the two scales) and a bf16 one a fourth."""
import numpy as np
import pytest
import torch

from plain64 import U16, U32, check

pytestmark = pytest.mark.gpu
mx = pytest.importorskip("mxfp4_moe_expert_amd")
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rand(seed, *shape, scale=1.0):
    return torch.randn(*shape, generator=_gen(seed), device=DEV) * scale


def _codes(seed, rows, K, low=-127):
    return torch.randint(low, 128, (rows, K), generator=_gen(seed), device=DEV, dtype=torch.int8)


def encode(x):
    """Codes and scales of x [R][K] in 64 bits (the quotient of two fp32 values, rounded in 64 bits, lies on a border
    between two codes only if it does exactly: the border is 2^-33 of it away at the least)."""
    v = x.double()
    bad = ~torch.isfinite(v).all(dim=1)
    m = torch.where(bad.unsqueeze(1), torch.zeros_like(v), v).abs().amax(dim=1)
    s = (m / 127).float().clamp(min=2.0 ** -126)
    s = torch.where(m == 0, torch.ones_like(s), s)
    q = torch.round(torch.where(bad.unsqueeze(1), torch.zeros_like(v), v) / s.double().unsqueeze(1))
    return q.to(torch.int8), torch.where(bad, torch.full_like(s, float("nan")), s)


def same(a, b):
    return torch.equal(torch.nan_to_num(a, nan=-7.0), torch.nan_to_num(b, nan=-7.0))


# ---------------------------------------------------------------- conversions

# K on both sides of every change of the kernel (16-byte pieces per row: 64, 128, 256, 512, 1024, 2048), in 8 and 4 values
KS = [16, 48, 512, 528, 1024, 1040, 2048, 2064, 4096, 4112, 8192, 8208, 16384, 16400, 65536]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("K", KS)
def test_quantize_and_back(K, dtype):
    rows = 7 if K > 4096 else 37
    x = (_rand(K, rows, K) * torch.exp2(_rand(1, rows, 1, scale=4.0).clamp(-9, 9))).to(DT[dtype])
    codes, scales = mx.quantize_int8(x)
    q, s = encode(x)
    assert torch.equal(codes, q) and torch.equal(scales, s)
    v = q.double() * s.double().unsqueeze(1)
    assert torch.equal(mx.dequantize_int8(codes, scales, dtype=torch.float32), v.float())
    # the product of code and scale is rounded to fp32, then to bf16
    assert torch.equal(mx.dequantize_int8(codes, scales), v.float().to(torch.bfloat16))


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 1000])
def test_quantize_row_counts(rows):
    for K in (32, 2048):
        x = _rand(rows, rows, K).to(torch.bfloat16)
        codes, scales = mx.quantize_int8(x)
        q, s = encode(x)
        assert torch.equal(codes, q) and torch.equal(scales, s)


def test_quantize_borders_between_codes():
    """Rows whose scale is a power of two hold exact borders n + 1/2 and their fp32 neighbours; rows of ordinary scales
    hold the fp32 values around every border of theirs."""
    n = np.arange(127, dtype=np.float32) + np.float32(0.5)
    around = np.concatenate([n, np.nextafter(n, np.float32(0)), np.nextafter(n, np.float32(999))])
    base = np.concatenate([around, -around, np.zeros(16 * 48 - 2 * len(around) - 1, np.float32), [np.float32(127)]])
    rows = [np.ldexp(base, e).astype(np.float32) for e in (-126, -125, -60, 0, 60, 120)]
    for m in (1.0, 3.3, 0.7123, 1e-30, 3e38, 1.7e-38, 5e-39):
        s = np.float32(max(np.float32(m) / np.float32(127), 2.0 ** -126))
        with np.errstate(over="ignore", under="ignore"):
            near = [np.float32(np.float64(s) * float(k)) for k in n]
        near = np.array(near, np.float32)
        row = np.concatenate([near, np.nextafter(near, np.float32(0)), np.nextafter(near, np.float32(np.inf))])
        row = np.concatenate([row, -row])
        row = np.where(np.abs(row) > np.float32(m), np.float32(0), row)
        rows.append(np.concatenate([row, np.zeros(16 * 48 - len(row) - 1, np.float32), [np.float32(m)]]))
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).to(DEV)
    codes, scales = mx.quantize_int8(x)
    q, s = encode(x)
    assert torch.equal(scales, s)
    assert torch.equal(codes, q)
    assert int(codes.abs().max()) == 127


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("K", [32, 2048, 32768])
def test_quantize_zeros_and_non_finite_rows(K, dtype):
    x = _rand(3, 6, K).to(DT[dtype])
    x[0] = 0.0
    x[1] = -0.0
    x[2, K - 1] = float("inf")
    x[3, 0] = float("-inf")
    x[4, K // 2] = float("nan")
    codes, scales = mx.quantize_int8(x)
    q, s = encode(x)
    assert torch.equal(codes, q) and same(scales, s)
    assert scales[0] == 1 and scales[1] == 1 and bool(scales[2:5].isnan().all()) and not codes[:5].any()
    back = mx.dequantize_int8(codes, scales, dtype=torch.float32)
    assert bool(back[2:5].isnan().all()) and bool(torch.isfinite(back[5]).all())


def test_quantize_tiny_rows():
    x = torch.tensor([2.0 ** -149, -(2.0 ** -130), 2.0 ** -126, 0.0] * 8, device=DEV).repeat(3, 1)
    x[1] *= 2.0 ** -10
    x[2] *= 64.0
    codes, scales = mx.quantize_int8(x)
    q, s = encode(x)
    assert torch.equal(codes, q) and torch.equal(scales, s)


def test_more_rows_than_one_launch_takes():
    """2^29 + 40 rows of 16 values at eight threads each are more than 2^32 threads."""
    rows, K = 2 ** 29 + 40, 16
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, 2 ** 28 - 1, 2 ** 28, 2 ** 28 + 1, 2 ** 29 - 1, 2 ** 29, rows - 1], device=DEV)
    x[at] = _rand(17, at.numel(), K).bfloat16()
    codes, scales = mx.quantize_int8(x)
    want, ws = encode(x[at])
    assert torch.equal(codes[at], want) and torch.equal(scales[at], ws)
    assert int(torch.count_nonzero(codes)) == int(torch.count_nonzero(want))
    assert int(torch.count_nonzero(scales != 1)) == at.numel()
    mx.dequantize_int8(codes, scales, out=x)
    assert torch.equal(x[at], (want.float() * ws[:, None]).bfloat16())
    assert int(torch.count_nonzero(x)) == int(torch.count_nonzero(want))


def test_quantize_strided_rows_shapes_and_outputs():
    whole = _rand(5, 40, 256).to(torch.bfloat16)
    part = whole[:, 64:160]
    codes, scales = mx.quantize_int8(part)
    q, s = encode(part)
    assert torch.equal(codes, q) and torch.equal(scales, s)
    c3, s3 = mx.quantize_int8(whole.view(4, 10, 256))
    assert c3.shape == (4, 10, 256) and s3.shape == (4, 10)
    c1, s1 = mx.quantize_int8(whole[0])
    assert c1.shape == (256,) and s1.shape == () and torch.equal(c1, c3[0, 0])
    out = (torch.full((40, 256), 99, dtype=torch.int8, device=DEV), torch.zeros(41, device=DEV)[1:])
    assert mx.quantize_int8(whole, out=out)[0] is out[0]             # scales at any multiple of 4 bytes
    assert torch.equal(out[0], c3.view(40, 256)) and torch.equal(out[1], s3.view(40))
    assert torch.equal(mx.dequantize_int8(*out), mx.dequantize_int8(c3, s3).view(40, 256))
    e = mx.quantize_int8(whole[:0])
    assert e[0].shape == (0, 256) and e[1].shape == (0,)
    assert mx.dequantize_int8(*e).shape == (0, 256)


# ---------------------------------------------------------------- the product

def product(xq, xs, q, s, half):
    y = (xq.double() @ q.double().t()) * xs.double().unsqueeze(1) * s.double()
    return y, (3 * U32 * (1 + half) + half) * y.abs()


# rows: one, the sizes around those where kernel, tile or cut change, many; K and N: odd multiples of 16, any N
LINEAR = [(3, 8192, 12000), (5, 4096, 300), (6, 4112, 6000), (8, 1040, 12304), (1, 16, 1), (1, 4096, 1536), (2, 1040, 17), (7, 272, 100), (8, 4096, 256), (9, 8192, 48), (16, 2048, 1000),
          (17, 2064, 33), (31, 528, 4096), (32, 4096, 512), (33, 8192, 4096), (48, 144, 130), (64, 4096, 4096),
          (65, 65536, 64), (100, 4112, 127), (129, 1024, 257), (300, 4096, 768), (513, 1296, 2000), (1000, 4096, 4096),
          (4097, 512, 640)]


@pytest.mark.parametrize("T,K,N", LINEAR)
def test_linear_from_bf16(T, K, N):
    x = _rand(T, T, K).to(torch.bfloat16)
    x[:, ::31] *= 6
    q, s = _codes(K, N, K), _rand(N, N).abs() * 0.01 + 1e-4
    xq, xs = encode(x)
    y, b = product(xq, xs, q, s, 0.0)
    check(mx.linear_w8a8(x, q, s, out_fp32=True), y, b, "fp32")
    y, b = product(xq, xs, q, s, U16)
    check(mx.linear_w8a8(x, q, s), y, b, "bf16")


@pytest.mark.parametrize("T,K,N", LINEAR)
def test_linear_from_codes(T, K, N):
    xq, xs = _codes(T, T, K, low=-128), _rand(1, T).abs() + 1e-3
    q, s = _codes(K, N, K, low=-128), _rand(N, N) * 0.01
    y, b = product(xq, xs, q, s, 0.0)
    check(mx.linear_w8a8(xq, q, s, x_scale=xs, out_fp32=True), y, b, "fp32")


def test_linear_largest_sums():
    """65536 products of 128 x 128, either sign: 2^30, the largest the format reaches."""
    for T in (1, 20, 70):
        xq = torch.full((T, 65536), -128, dtype=torch.int8, device=DEV)
        q = torch.full((24, 65536), -128, dtype=torch.int8, device=DEV)
        q[12:] = 127
        one = torch.ones(24, device=DEV)
        y = mx.linear_w8a8(xq, q, one, x_scale=torch.ones(T, device=DEV), out_fp32=True)
        assert bool((y[:, :12] == 2.0 ** 30).all()) and bool((y[:, 12:] == -128.0 * 127 * 65536).all())


@pytest.mark.parametrize("T,K,N", [(3, 65536, 65536), (70, 65536, 65536), (65536, 65536, 40)])
def test_linear_operands_past_32_bits(T, K, N):
    """Operands of 4 GB and more: rows at both ends, in the middle and on both sides of 2^31 and 2^32 bytes."""
    x, q, s = _rand(T, T, K).to(torch.bfloat16), _codes(N, N, K), _rand(1, N).abs() + 1e-3
    t = torch.tensor(sorted({0, T // 4, max(T // 2 - 1, 0), T // 2, T - 1}), device=DEV)
    n = torch.tensor(sorted({0, N // 4, N // 2 - 1, N // 2, N - 2, N - 1}), device=DEV)
    got = mx.linear_w8a8(x, q, s, out_fp32=True)[t][:, n]
    xq, xs = encode(x[t])
    y, b = product(xq, xs, q[n], s[n], 0.0)
    check(got, y, b, "fp32")


@pytest.mark.parametrize("T", [1, 6, 20, 90, 600])
def test_linear_rows_do_not_depend_on_each_other(T):
    """A row's result is the same bits alone and among others; non-finite rows and channels stay by themselves."""
    K, N = 1536, 320
    x, q, s = _rand(T, T, K).to(torch.bfloat16), _codes(1, N, K), _rand(2, N).abs()
    y = mx.linear_w8a8(x, q, s)
    for t in {0, T // 2, T - 1}:
        assert torch.equal(mx.linear_w8a8(x[t:t + 1], q, s)[0], y[t]), t
    x2, s2 = x.clone(), s.clone()
    x2[T // 2, 5] = float("inf")
    s2[7] = float("nan")
    z = mx.linear_w8a8(x2, q, s2)
    assert bool(z[T // 2].isnan().all()) and bool(z[:, 7].isnan().all())
    rows = [t for t in range(T) if t != T // 2]
    cols = [n for n in range(N) if n != 7]
    assert torch.equal(z[rows][:, cols], y[rows][:, cols])


@pytest.mark.parametrize("T,N", [(1, 33), (20, 33), (90, 129), (600, 1000)])
def test_linear_writes_its_output_only_and_takes_offset_scales(T, N):
    K = 272
    x, q = _rand(T, T, K).to(torch.bfloat16), _codes(1, N, K)
    s = _rand(2, N + 3).abs()[3:]                                     # starts at 12 bytes
    buf = torch.full((T * N + 64,), 7.0, device=DEV, dtype=torch.bfloat16)
    out = buf[32:32 + T * N].view(T, N)
    need = mx.lib().moe_linear_w8a8_workspace_size(T, K, N, 0)
    ws = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device=DEV)
    mx.linear_w8a8(x, q, s, out=out, ws=ws[:need])
    assert torch.equal(out, mx.linear_w8a8(x, q, s.clone()))
    assert bool((buf[:32] == 7).all()) and bool((buf[32 + T * N:] == 7).all()) and bool((ws[need:] == 0xAB).all())
    assert mx.linear_w8a8(x[:0], q, s).shape == (0, N)


def test_linear_refusals_on_device():
    x, q, s = _rand(0, 4, 64).to(torch.bfloat16), _codes(0, 16, 64), _rand(0, 16).abs()
    for bad in (lambda: mx.linear_w8a8(x[:, :48], q, s), lambda: mx.linear_w8a8(x, q, s[:8]),
                lambda: mx.linear_w8a8(x, q[:, ::2], s), lambda: mx.linear_w8a8(x[0], q, s),
                lambda: mx.linear_w8a8(x.t(), q, s), lambda: mx.linear_w8a8(x, q, s.cpu()),
                lambda: mx.linear_w8a8(q, q, s, x_scale=s[:3]), lambda: mx.quantize_int8(x[:, :40].contiguous()),
                lambda: mx.quantize_int8(x.t())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: mx.linear_w8a8(x.float(), q, s), lambda: mx.linear_w8a8(x, q.float(), s),
                lambda: mx.linear_w8a8(x, q, s, x_scale=s[:4])):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(mx.MoEError, match="x: not 16-byte"):
        mx.linear_w8a8(_rand(0, 4 * 64 + 4).to(torch.bfloat16)[4:].view(4, 64), q, s)
    with pytest.raises(mx.MoEError):
        mx.linear_w8a8(_rand(0, 90, 64).to(torch.bfloat16), q, s, ws=torch.empty(256, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("T", [1, 20, 90, 700])
def test_linear_on_two_streams_and_in_graphs(T):
    K, N = 2048, 520
    q, s = _codes(1, N, K), _rand(2, N).abs()
    xs = [_rand(10 + i, T, K).to(torch.bfloat16) for i in range(4)]
    want = [mx.linear_w8a8(x, q, s) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i, x in enumerate(xs):
        with torch.cuda.stream(streams[i % 2]):
            got.append(mx.linear_w8a8(x, q, s))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    held, graphs, outs = [x.clone() for x in xs[:2]], [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mx.linear_w8a8(held[i], q, s))
        graphs.append(g)
    for r in range(3):
        for i in range(2):
            held[i].copy_(xs[(r + i) % 4])
            graphs[i].replay()
        eager = mx.linear_w8a8(xs[3], q, s)
        torch.cuda.synchronize()
        assert torch.equal(eager, want[3])
        for i in range(2):
            assert torch.equal(outs[i], want[(r + i) % 4]), (r, i)


def test_linear_agrees_with_the_16_bit_activations_product():
    """Weights of linear_w8a16 as they are; the two differ by what 8 bits leave of the activations: at most half a scale
    per value, as a bound over the row's products, and both outputs' rounding."""
    T, K, N = 70, 1024, 512
    x, q, s = _rand(1, T, K).to(torch.bfloat16), _codes(2, N, K), _rand(3, N).abs() * 0.01 + 1e-3
    a, b = mx.linear_w8a8(x, q, s, out_fp32=True).double(), mx.linear_w8a16(x, q, s, out_fp32=True).double()
    _, xs = encode(x)
    lim = 0.5 * xs.double().unsqueeze(1) * (q.double().abs().sum(dim=1) * s.double()) * (1 + 2.0 ** -20)
    lim = lim + (K / 4 + 64) * U32 * ((x.double().abs() @ q.double().abs().t()) * s.double())
    assert bool(((a - b).abs() <= lim).all())
