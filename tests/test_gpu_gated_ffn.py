"""GPU tests of the gated block with bf16 weights and its gradients, against
the 64-bit form and bounds of tests/plain64.py, and against differences."""
import math

import numpy as np
import pytest
import torch

import plain64
from plain64 import U16, check

pytestmark = pytest.mark.gpu
mx = pytest.importorskip("mxfp4_moe_expert_amd")
DEV = "cuda"


def _inputs(seed, T, H, I, scale=None):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g, device=DEV)

    sc = scale if scale is not None else 1.3 / math.sqrt(H)
    return (r(T, H).to(torch.bfloat16), (r(2 * I, H) * sc).to(torch.bfloat16),
            (r(H, I) / math.sqrt(I)).to(torch.bfloat16), (r(T, H) * 0.1).to(torch.bfloat16))


def _ref(x, w13, w2, L, dy=None):
    return plain64.ffn(x.double(), w13.double(), w2.double(), L, None if dy is None else dy.double())


# Relative L2 of the whole: independent roundings of at most a half step each, so no more than the sum of the half
# steps on the way: y and dw2: h and the output; dx and dw13: dg / du and the output.
L2_OUT, L2_GRAD = 2 * U16, 2 * U16

# The streaming pass ends at 32 rows, or earlier by size: 33 and 64 rows below run as tile products. Its variants by
# waves, and the tiles with K split, are in test_gpu_dense_variants.py.
SHAPES = [  # T, H, I: the streaming pass (1 .. 64), then every tile size, splits and ragged edges
    (1, 8, 8), (1, 4096, 2048), (2, 264, 136), (16, 1024, 512), (17, 2048, 72), (33, 512, 1024), (64, 4096, 512),
    (65, 8, 8), (65, 1024, 264), (100, 4096, 2048), (129, 264, 520), (300, 4096, 2048), (777, 2048, 1024),
    (1000, 200, 4096), (2100, 1032, 2048),
]


@pytest.mark.parametrize("T,H,I", SHAPES)
def test_forward(T, H, I):
    print(f"[gated_ffn T={T} H={H} I={I}]", flush=True)
    x, w13, w2, _ = _inputs(T + H, T, H, I)
    y = mx.gated_ffn(x, w13, w2)
    check(y, *_ref(x, w13, w2, 10.0)["y"], "y", l2=L2_OUT)
    y2, (gu, h) = mx.gated_ffn(x, w13, w2, save=True, out_fp32=True)
    assert torch.equal(y2.to(torch.bfloat16), y)
    g, u = x.double() @ w13[:I].double().t(), x.double() @ w13[I:].double().t()
    eg = plain64.sum_err(x.double().abs() @ w13.double().abs().t(), H)
    assert gu.dtype == torch.float32 and h.dtype == torch.bfloat16
    check(gu, torch.cat((g, u), 1), eg, "gu")
    assert torch.equal(y, mx.gated_ffn(x, w13, w2))  # repeatable


@pytest.mark.parametrize("T,H,I", [(1, 8, 8), (1, 1024, 512), (3, 264, 136), (64, 512, 1024), (65, 1024, 264),
                                   (129, 264, 520), (300, 2048, 1024), (777, 2048, 1024), (1000, 200, 2048),
                                   (2100, 1032, 1024), (1024, 4096, 2048)])
def test_gradients(T, H, I):
    print(f"[gated_ffn_backward T={T} H={H} I={I}]", flush=True)
    x, w13, w2, dy = _inputs(T + H, T, H, I)
    y, saved = mx.gated_ffn(x, w13, w2, save=True)
    got = dict(zip(("dx", "dw13", "dw2"), mx.gated_ffn_backward(dy, x, w13, w2, saved)))
    ref = _ref(x, w13, w2, 10.0, dy)
    for name in got:
        check(got[name], *ref[name], name, l2=L2_GRAD)
    f32 = mx.gated_ffn_backward(dy, x, w13, w2, saved, dw_fp32=True)
    assert torch.equal(f32[1].to(torch.bfloat16), got["dw13"]) and torch.equal(f32[2].to(torch.bfloat16), got["dw2"])
    for need in ((True, False, False), (False, True, False), (False, False, True)):
        part = mx.gated_ffn_backward(dy, x, w13, w2, saved, need=need)
        for n, p, name in zip(need, part, got):
            assert (p is None) == (not n)
            if n:
                assert torch.equal(p, got[name]), name


@pytest.mark.parametrize("T", [5, 150])
@pytest.mark.parametrize("limit", [0.5, 1.0, 0.7001, math.inf])
def test_clamp_borders(T, limit):
    """Limits that many values pass (and one that bf16 does not hold): no gradient through a clamp that acted."""
    H, I = 128, 256
    x, w13, w2, dy = _inputs(T, T, H, I)
    L = float(np.float32(limit))
    y, saved = mx.gated_ffn(x, w13, w2, limit=limit, save=True)
    ref = _ref(x, w13, w2, L, dy)
    check(y, *ref["y"], "y", l2=L2_OUT)
    g = x.double() @ w13[:I].double().t()
    if limit < 2:
        assert int((g > L).sum()) > 100
    eg = plain64.sum_err(x.double().abs() @ w13[:I].double().abs().t(), H)
    sure = (g - L).abs() > 2 * eg
    assert torch.equal((saved[0][:, :I].double() > L)[sure], (g > L)[sure])  # the side of the border is kept
    for name, t in zip(("dx", "dw13", "dw2"), mx.gated_ffn_backward(dy, x, w13, w2, saved, limit=limit)):
        check(t, *ref[name], name, l2=L2_GRAD)


@pytest.mark.parametrize("T", [1, 100])
def test_saved_values_at_the_border(T):
    """g and u exactly at, just above and just below the limit, by less than a bf16 step: only the one past it stops
    the gradient (a value at the limit passes it)."""
    H, I, L = 8, 8, 10.0
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[:, 0], x[:, 1] = 1.0, 1.0 / 64
    w13 = torch.zeros(2 * I, H, dtype=torch.bfloat16, device=DEV)
    # columns 0..2: g = 10, 10 + 1/64, 10 - 1/64 (bf16 steps by 1/16 there), u = 1; 3..6: the same for u = +-10..
    for i, (gv, ge, uv, ue) in enumerate([(10, 0, 1, 0), (10, 1, 1, 0), (10, -1, 1, 0), (1, 0, 10, 0), (1, 0, 10, 1),
                                          (1, 0, -10, -1), (1, 0, -10, 1), (1, 0, 1, 0)]):
        w13[i, 0], w13[i, 1] = gv, ge
        w13[I + i, 0], w13[I + i, 1] = uv, ue
    w2 = torch.eye(8, dtype=torch.bfloat16, device=DEV)
    dy = torch.ones(T, H, dtype=torch.bfloat16, device=DEV)
    y, saved = mx.gated_ffn(x, w13, w2, limit=L, save=True)
    gu = saved[0].float()
    assert (gu[0, :3] > L).tolist() == [False, True, False]
    assert (gu[0, I + 3:I + 7].abs() > L).tolist() == [False, True, True, False]
    dx, dw13, dw2 = mx.gated_ffn_backward(dy, x, w13, w2, saved, limit=L, dw_fp32=True)
    live = (dw13[:, 0] != 0).tolist()
    assert live[:3] == [True, False, True] and live[I + 3:I + 7] == [True, False, False, True]
    check(y, *_ref(x, w13, w2, L)["y"], "y")


@pytest.mark.parametrize("T", [2, 90])
def test_gradients_against_differences(T):
    """Central differences of the kernel's own fp32 output along random directions. A step keeps bf16 inputs exact
    (values and steps on one coarse grid); the two outputs each carry the block's rounding of h (2^-8 of a term,
    independent from term to term), so the quotient may be off by about 2^-8 |dy| |h| |w2| / step, summed over
    independent terms: 6 deviations are allowed, plus the curvature term step^2 / 6 |f'''|."""
    H, I = 64, 32
    g = torch.Generator(device=DEV)
    g.manual_seed(7)

    def grid(*s, step):  # multiples of step, at most 64 steps
        return (torch.randint(-48, 49, s, generator=g, device=DEV) * step).to(torch.bfloat16)

    x, w13, w2 = grid(T, H, step=1 / 32), grid(2 * I, H, step=1 / 128), grid(H, I, step=1 / 64)
    dy = grid(T, H, step=1 / 32)
    y, saved = mx.gated_ffn(x, w13, w2, save=True, out_fp32=True)
    grads = mx.gated_ffn_backward(dy, x, w13, w2, saved, dw_fp32=True)
    h = plain64.ffn(x.double(), w13.double(), w2.double(), 10.0)
    hv = saved[1].double().abs()
    for name, t, grad, step in (("x", x, grads[0], 1 / 4), ("w13", w13, grads[1], 1 / 32), ("w2", w2, grads[2], 1 / 8)):
        v = (torch.randint(0, 2, t.shape, generator=g, device=DEV) * 2 - 1).to(torch.bfloat16) * step
        vals, exact = [], []
        for sgn in (1, -1):
            args = {"x": x, "w13": w13, "w2": w2}
            moved = t + sgn * v
            assert torch.equal(moved.double(), t.double() + sgn * v.double())
            args[name] = moved
            yy = mx.gated_ffn(args["x"], args["w13"], args["w2"], out_fp32=True)
            vals.append((yy.double() * dy.double()).sum())
            exact.append((plain64.ffn(args["x"].double(), args["w13"].double(), args["w2"].double(), 10.0)["y"][0]
                          * dy.double()).sum())
        num = float(vals[0] - vals[1]) / 2
        curve = abs(float(exact[0] - exact[1]) / 2 - float((plain64.ffn(
            x.double(), w13.double(), w2.double(), 10.0, dy.double())["d" + name][0] * v.double()).sum()))
        ana = float((grad.double() * v.double()).sum())
        # deviations: h's rounding in both outputs, and the gradient's own roundings (2 half steps of each element)
        dh = (dy.double() @ w2.double()).abs()
        dev = U16 * float((dh * (hv + 1)).norm()) + 2 * U16 * float((grad.double() * v.double()).norm())
        assert abs(num - ana) <= curve + 6 * dev, (name, num, ana, curve, dev)
    assert h["y"][0].shape == y.shape


@pytest.mark.parametrize("T", [4, 80])
def test_non_finite_inputs_stay_in_their_rows(T):
    H, I = 72, 40
    x, w13, w2, dy = _inputs(1, T, H, I)
    y, saved = mx.gated_ffn(x, w13, w2, save=True)
    dx = mx.gated_ffn_backward(dy, x, w13, w2, saved)[0]
    x2 = x.clone()
    x2[2, 3] = float("nan")
    y2, saved2 = mx.gated_ffn(x2, w13, w2, save=True)
    dx2 = mx.gated_ffn_backward(dy, x2, w13, w2, saved2)[0]
    keep = [t for t in range(T) if t != 2]
    assert bool(torch.isnan(y2[2]).all()) and bool(torch.isnan(dx2[2]).all())
    assert torch.equal(y2[keep], y[keep]) and torch.equal(dx2[keep], dx[keep])


def test_large_pre_activations():
    """g of both signs far past the exponential's range: silu is 0 or the clamp, nothing overflows."""
    H, I, T = 64, 64, 70
    x, w13, w2, dy = _inputs(3, T, H, I, scale=60.0)
    y, saved = mx.gated_ffn(x, w13, w2, save=True)
    ref = _ref(x, w13, w2, 10.0, dy)
    check(y, *ref["y"], "y", l2=L2_OUT)
    for name, t in zip(("dx", "dw13", "dw2"), mx.gated_ffn_backward(dy, x, w13, w2, saved)):
        assert bool(torch.isfinite(t).all())
        check(t, *ref[name], name)


def test_empty_batch():
    x, w13, w2, _ = _inputs(1, 4, 64, 40)
    e = x[:0]
    y, saved = mx.gated_ffn(e, w13, w2, save=True)
    assert y.shape == (0, 64)
    dx, dw13, dw2 = mx.gated_ffn_backward(e, e, w13, w2, saved)
    assert dx.shape == (0, 64) and not bool(dw13.any()) and not bool(dw2.any())


def test_refusals_on_device():
    x, w13, w2, dy = _inputs(1, 4, 64, 40)
    with pytest.raises(mx.MoEError):
        mx.gated_ffn(x, w13, w2, limit=0.0)
    with pytest.raises(mx.MoEError):
        mx.gated_ffn(x, w13, w2, limit=float("nan"))
    with pytest.raises(ValueError):
        mx.gated_ffn(x, w13[:-2], w2)
    with pytest.raises(TypeError):
        mx.gated_ffn(x.float(), w13, w2)
    with pytest.raises(ValueError):
        mx.gated_ffn(x, w13, w2.t().contiguous().t())
    with pytest.raises(mx.MoEError):
        mx.gated_ffn(x[:, :60].contiguous(), w13[:, :60].contiguous(), w2[:60].contiguous())  # H % 8
    with pytest.raises(mx.MoEError):
        mx.gated_ffn(x, w13, w2, ws=torch.empty(0, dtype=torch.uint8, device=DEV))
    y, saved = mx.gated_ffn(x, w13, w2, save=True)
    with pytest.raises(ValueError):
        mx.gated_ffn_backward(dy[:2], x, w13, w2, saved)
    with pytest.raises(TypeError):
        mx.gated_ffn_backward(dy, x, w13, w2, (saved[1], saved[0]))


@pytest.mark.parametrize("T,H,I", [(5, 72, 40), (100, 264, 136), (300, 1024, 520)])
def test_stated_workspace_is_enough(T, H, I):
    """Workspaces of exactly the stated size, filled with NaN patterns, guarded on both sides."""
    x, w13, w2, dy = _inputs(1, T, H, I)
    y, saved = mx.gated_ffn(x, w13, w2, save=True)
    grads = mx.gated_ffn_backward(dy, x, w13, w2, saved)
    L = mx.lib()

    def guarded(need):
        b = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=DEV)
        o = (-b.data_ptr()) % 256
        return b, o, b[o:o + need]

    n1, n2 = L.moe_gated_ffn_workspace_size(T, H, I), L.moe_gated_ffn_backward_workspace_size(T, H, I)
    b1, o1, ws1 = guarded(n1)
    b2, o2, ws2 = guarded(n2)
    assert torch.equal(mx.gated_ffn(x, w13, w2, ws=ws1), y)
    for a, b in zip(mx.gated_ffn_backward(dy, x, w13, w2, saved, ws=ws2), grads):
        assert torch.equal(a, b)
    for b, o, n in ((b1, o1, n1), (b2, o2, n2)):
        assert bool((b[:o] == 0xFF).all()) and bool((b[o + n:] == 0xFF).all())


def test_training_step_on_streams_and_in_graphs():
    """A captured training step replayed with eager steps between, and steps on two streams at once."""
    T, H, I = 130, 512, 264
    sets = [_inputs(i, T, H, I) for i in range(3)]

    def step(i):
        x, w13, w2, dy = sets[i]
        y, saved = mx.gated_ffn(x, w13, w2, save=True)
        return (y,) + mx.gated_ffn_backward(dy, x, w13, w2, saved)

    ref = [step(i) for i in range(3)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            got.append(step(i))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], ref[i])), i
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(i))
        graphs.append(g)
    for rep in range(3):
        for o in outs[0] + outs[1]:
            o.zero_()
        for g in graphs:
            g.replay()
        eager = step(2)
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], ref[i])), (rep, i)
        assert all(torch.equal(a, b) for a, b in zip(eager, ref[2])), rep


def test_train_encode_serve():
    """The operators as used together: a step of the bf16 block, its updated weights encoded to MXFP4, and the
    encoded block served through linear_mxfp4, against the 64-bit block on the encoded values."""
    T, H, I = 96, 256, 128
    x, w13, w2, dy = _inputs(11, T, H, I)
    y, saved = mx.gated_ffn(x, w13, w2, save=True)
    dx, dw13, dw2 = mx.gated_ffn_backward(dy, x, w13, w2, saved, dw_fp32=True)
    m13, m2 = w13.float() - 0.1 * dw13, w2.float() - 0.1 * dw2
    c13, s13 = mx.quantize_mxfp4(m13)
    c2, s2 = mx.quantize_mxfp4(m2)
    q13, q2 = mx.dequantize_mxfp4(c13, s13), mx.dequantize_mxfp4(c2, s2)
    dense = mx.gated_ffn(x, q13, q2)
    check(dense, *_ref(x, q13, q2, 10.0)["y"], "dense on the encoded values", l2=L2_OUT)
    gu = mx.linear_mxfp4(x, c13, s13, out_fp32=True)
    h = (torch.nn.functional.silu(gu[:, :I].clamp(max=10.0)) * gu[:, I:].clamp(-10.0, 10.0)).to(torch.bfloat16)
    served = mx.linear_mxfp4(h, c2, s2)
    check(served, *_ref(x, q13, q2, 10.0)["y"], "served", l2=L2_OUT)
