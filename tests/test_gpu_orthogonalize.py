"""GPU tests of the Newton-Schulz update against the same steps in 64 bits. How far the result may be off is what its
roundings alone bring about: the steps in 64 bits with the values rounded to fp16 where the kernels round them (X to two
values, its first one in the last step; A; b A + c A A), by half as much again for the fp32 sums and for roundings that
fall the other way, and a bf16 output's half step."""
import pytest
import torch

pytestmark = pytest.mark.gpu
mx = pytest.importorskip("mxfp4_moe_expert_amd")
DEV = "cuda"
COEF = (3.4445, -4.7750, 2.0315)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def gradient(seed, R, C, kind="plain", B=None):
    g = _gen(seed)
    shape = (R, C) if B is None else (B, R, C)
    noise = torch.randn(*shape, generator=g, device=DEV)
    if kind == "plain":
        return noise * 1e-3
    r = max(1, min(R, C) // 8)
    lead = () if B is None else (B,)
    left = torch.randn(*lead, R, r, generator=g, device=DEV) * torch.logspace(0, -1.5, r, device=DEV)
    return 1e-3 * (left @ torch.randn(*lead, r, C, generator=g, device=DEV) + 0.03 * noise)


def steps64(G, steps=5, coef=COEF, eps=1e-7, rounded=False):
    a, b, c = coef

    def half(v):
        return (v * 256).to(torch.float16).double() / 256 if rounded else v

    def plain_half(v):
        return v.to(torch.float16).double() if rounded else v

    X = G.double()
    flip = X.shape[0] > X.shape[1]
    X = X.t().contiguous() if flip else X
    X = X / (X.norm() + eps)
    for i in range(steps):
        h = half(X)
        A = plain_half(h @ h.t())
        P = plain_half(b * A + c * (A @ A))
        X = a * (h if rounded and i + 1 == steps else X) + P @ h
    return X.t() if flip else X


def hold(got, G, steps=5, coef=COEF, eps=1e-7):
    want = steps64(G, steps, coef, eps)
    sim = steps64(G, steps, coef, eps, rounded=True)
    n = float(want.norm())
    e_sim, e = float((sim - want).norm()) / n, float((got.double() - want).norm()) / n
    # where few values are rounded, single roundings show: one of each kind and step, as large as they come
    few = 2.0 ** -9 if min(G.shape) < 16 else 0.0
    assert e <= 1.5 * e_sim + few + 2.0 ** -8, f"{e:.3g} off, {e_sim:.3g} by rounding"
    assert e <= 1e-2
    return e


# m x n on both sides of every change of way: tile rows (32, 64, 128, 256), what one block holds (32 x 1024, 64 x 512,
# 128 x 256), panels of 64; above 256 tile products, K split or whole
SIZES = [(32, 1024), (1025, 31), (33, 512), (513, 64), (65, 256), (257, 128), (128, 1000), (129, 64), (200, 3000), (256, 257),
         (1, 1), (1, 9), (9, 1), (2, 3), (7, 8), (8, 8), (16, 5), (17, 33), (33, 17), (64, 64), (100, 300), (300, 100),
         (127, 129), (129, 128), (256, 256), (257, 520), (520, 257), (64, 2050), (2050, 72), (256, 4096), (1001, 600),
         (1024, 1024), (1000, 2000), (2048, 640)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,C", SIZES)
def test_against_64_bits(R, C, dtype):
    for kind in ("plain", "strong"):
        G = gradient(R + C, R, C, kind).to(dtype)
        hold(mx.orthogonalize(G), G)


def test_fp16_input_steps_and_coefficients():
    G = (gradient(1, 130, 70) * 100).to(torch.float16)
    for steps in (1, 2, 3, 8):
        hold(mx.orthogonalize(G, steps=steps), G, steps=steps)
    cubic = (1.5, -0.5, 0.0)
    hold(mx.orthogonalize(G, steps=12, coefficients=cubic), G, steps=12, coef=cubic)
    hold(mx.orthogonalize(G, eps=10.0), G, eps=10.0)


def test_singular_values_end_near_one():
    G = gradient(3, 300, 520)
    s = torch.linalg.svdvals(mx.orthogonalize(G).double())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.25


@pytest.mark.parametrize("R,C", [(40, 100), (1000, 72), (150, 1300), (513, 513)])
def test_stack(R, C):
    """A stack is its matrices one by one, and a matrix's bits do not depend on the others'."""
    G = gradient(5, R, C, "strong", B=5) * torch.tensor([1.0, 1e-4, 1e5, 3.0, 1.0], device=DEV).view(5, 1, 1)
    got = mx.orthogonalize(G.view(5, 1, R, C))
    assert got.shape == (5, 1, R, C) and got.dtype == torch.bfloat16
    for i in range(5):
        hold(got[i, 0], G[i])
        hold(mx.orthogonalize(G[i]), G[i])
        others = gradient(50 + i, R, C, B=5)
        others[i] = G[i]
        assert torch.equal(mx.orthogonalize(others)[i], got[i, 0])


@pytest.mark.parametrize("B,R,C", [(1500, 200, 1104), (300, 700, 600)])
def test_stack_in_parts(B, R, C):
    """More matrices than the workspace holds at a time."""
    G = gradient(6, R, C, B=B).to(torch.bfloat16)
    size = mx.lib().moe_orthogonalize_workspace_size
    assert size(4 * B, R, C) < 1.5 * size(B, R, C)
    got = mx.orthogonalize(G)
    for i in list(range(0, B, B // 12)) + [B - 2, B - 1]:
        hold(got[i], G[i])


def test_stack_past_32_bits():
    """Nine matrices of 512 MB, each worked on by itself: the last starts 2^32 bytes in, and has the bits it has alone."""
    g = torch.zeros(9, 16384, 16384, dtype=torch.bfloat16, device=DEV)
    g[8] = torch.randn(16384, 16384, generator=_gen(3), device=DEV)
    out = mx.orthogonalize(g, steps=1)
    assert torch.equal(out[8], mx.orthogonalize(g[8], steps=1)) and bool(out[8].isfinite().all())
    assert int(torch.count_nonzero(out[:8])) == 0 and int(torch.count_nonzero(out[8])) > 2 ** 27


def test_scales_at_the_ends_of_the_range():
    G = gradient(7, 100, 60)
    base = mx.orthogonalize(G, eps=0.0)
    for p in (-90, -60, 60, 120):                                   # powers of two that lose no bit: the same X
        assert torch.equal(G * 2.0 ** p / 2.0 ** p, G)
        assert torch.equal(mx.orthogonalize(G * 2.0 ** p, eps=0.0), base), p
    tiny = G * 2.0 ** -120                                          # subnormal values among them
    hold(mx.orthogonalize(tiny, eps=0.0), tiny, eps=0.0)
    hold(mx.orthogonalize(tiny, eps=float(tiny.double().norm())), tiny, eps=float(tiny.double().norm()))


def test_zeros_non_finite_and_single_values():
    G = gradient(8, 64, 96, B=5)
    G[1] = 0.0
    G[2, 5, 7] = float("inf")
    G[3, 60, 1] = float("nan")
    got = mx.orthogonalize(G)
    assert not got[1].any()
    assert bool(got[2].isnan().all()) and bool(got[3].isnan().all())
    hold(got[0], G[0])
    hold(got[4], G[4])
    one = torch.zeros(40, 50, device=DEV)
    one[3, 4] = -2e-3
    got = mx.orthogonalize(one)
    hold(got, one)
    assert int((got != 0).sum()) == 1


def test_rank_deficient_and_tied_directions():
    G = gradient(9, 200, 8) @ gradient(10, 8, 300)                  # rank 8
    hold(mx.orthogonalize(G), G)
    eye = torch.eye(72, 130, device=DEV)                            # every singular value the same
    hold(mx.orthogonalize(eye), eye)


def test_empty_stack_outputs_and_workspace():
    assert mx.orthogonalize(torch.empty(0, 8, 9, device=DEV)).shape == (0, 8, 9)
    for R, C in ((33, 50), (50, 33), (64, 128), (200, 700), (700, 200), (300, 290)):
        G = gradient(11, R, C)
        need = mx.lib().moe_orthogonalize_workspace_size(1, R, C)
        ws = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device=DEV)
        buf = torch.full((R * C + 32,), 7.0, dtype=torch.bfloat16, device=DEV)
        out = buf[16:16 + R * C].view(R, C)
        assert mx.orthogonalize(G, out=out, ws=ws[:need]) is out
        assert bool((buf[:16] == 7).all()) and bool((buf[16 + R * C:] == 7).all()) and bool((ws[need:] == 0xAB).all())
        assert torch.equal(out, mx.orthogonalize(G))


def test_refusals_on_device():
    G = gradient(12, 16, 24)
    for bad in (lambda: mx.orthogonalize(G[0]), lambda: mx.orthogonalize(G.t()), lambda: mx.orthogonalize(G[:, :0]),
                lambda: mx.orthogonalize(G, out=torch.empty(24, 16, dtype=torch.bfloat16, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: mx.orthogonalize(G, out=torch.empty_like(G)), lambda: mx.orthogonalize(G.double())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: mx.orthogonalize(torch.zeros(1, 16392, device=DEV)), lambda: mx.orthogonalize(G, steps=0),
                lambda: mx.orthogonalize(G, eps=-1.0), lambda: mx.orthogonalize(G, coefficients=(1.0, float("nan"), 0.0)),
                lambda: mx.orthogonalize(gradient(12, 300, 280), ws=torch.empty(256, dtype=torch.uint8, device=DEV))):
        with pytest.raises(mx.MoEError):
            bad()
    with pytest.raises(mx.MoEError, match="out: not 16-byte"):
        mx.orthogonalize(G, out=torch.empty(16 * 24 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(16, 24))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,C", [(16, 24), (7, 5), (50, 33)])
def test_input_at_any_element(R, C, dtype):
    G = gradient(13, R, C).to(dtype)
    want = mx.orthogonalize(G)
    for skip in (1, 2, 3, 5):
        buf = torch.full((R * C + 16,), float("nan"), dtype=dtype, device=DEV)
        at = buf[skip:skip + R * C].view(R, C)
        at.copy_(G)
        assert torch.equal(mx.orthogonalize(at), want), skip


@pytest.mark.parametrize("R,C", [(60, 100), (1200, 160), (260, 390)])
def test_on_two_streams_and_in_graphs(R, C):
    Gs = [gradient(20 + i, R, C, "strong") for i in range(4)]
    want = [mx.orthogonalize(G) for G in Gs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i, G in enumerate(Gs):
        with torch.cuda.stream(streams[i % 2]):
            got.append(mx.orthogonalize(G))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    held, graphs, outs = [G.clone() for G in Gs[:2]], [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mx.orthogonalize(held[i]))
        graphs.append(g)
    for r in range(3):
        for i in range(2):
            held[i].copy_(Gs[(r + i) % 4])
            graphs[i].replay()
        eager = mx.orthogonalize(Gs[3])
        torch.cuda.synchronize()
        assert torch.equal(eager, want[3])
        for i in range(2):
            assert torch.equal(outs[i], want[(r + i) % 4]), (r, i)
