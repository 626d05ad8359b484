"""Host-side checks of the MXFP4 and gated-block entry points (no GPU): every
refusal is returned before anything is launched, and empty calls succeed."""
import math

import pytest
import torch

mx = pytest.importorskip("mxfp4_moe_expert_amd")

P = 0x100000        # never dereferenced: every call below fails a host check
ODD = 0x100008      # not 16-byte aligned
OK, EINVAL, EUNSUP, EWS = mx.MOE_OK, mx.MOE_EINVAL, mx.MOE_EUNSUPPORTED, mx.MOE_EWORKSPACE


def test_quantize_refusals():
    f = mx.lib().moe_mxfp4_quantize
    assert f(4, 64, 0, None, 64, P, P, None) == EINVAL
    assert f(4, 64, 0, P, 64, None, P, None) == EINVAL
    assert f(4, 64, 0, P, 64, P, None, None) == EINVAL
    assert f(-1, 64, 0, P, 64, P, P, None) == EINVAL
    assert f(4, 0, 0, P, 64, P, P, None) == EINVAL
    assert f(4, 64, 0, P, 32, P, P, None) == EINVAL      # rows overlap
    assert f(4, 64, 0, P, 68, P, P, None) == EINVAL      # rows not 16-byte aligned
    assert f(4, 64, 1, P, 66, P, P, None) == EINVAL
    assert f(4, 64, 0, ODD, 64, P, P, None) == EINVAL
    assert f(4, 64, 3, P, 64, P, P, None) == EUNSUP      # dtype
    assert f(4, 48, 0, P, 48, P, P, None) == EUNSUP      # K % 32
    assert f(4, 65568, 0, P, 65568, P, P, None) == EUNSUP
    assert f(1 << 40, 64, 0, P, 64, P, P, None) == EUNSUP
    assert f(0, 64, 0, None, 64, None, None, None) == OK


def test_dequantize_refusals():
    f = mx.lib().moe_mxfp4_dequantize
    assert f(4, 64, None, P, 0, P, None) == EINVAL
    assert f(4, 64, P, None, 0, P, None) == EINVAL
    assert f(4, 64, P, P, 0, None, None) == EINVAL
    assert f(4, 64, P, P, 0, ODD, None) == EINVAL
    assert f(4, 64, P, P, 2, P, None) == EUNSUP          # binary16 does not hold every value
    assert f(4, 40, P, P, 0, P, None) == EUNSUP
    assert f(0, 64, None, None, 0, None, None) == OK


def test_linear_refusals():
    L = mx.lib()
    size, f = L.moe_linear_mxfp4_workspace_size, L.moe_linear_mxfp4
    for T, K, N, act in ((-1, 64, 16, 0), (65537, 64, 16, 0), (8, 48, 16, 0), (8, 65568, 16, 0), (8, 64, 0, 0),
                         (8, 64, 65537, 0), (8, 64, 16, 2)):
        assert size(T, K, N, act) == 0, (T, K, N, act)
    assert 0 < size(1, 4096, 4096, 0) <= 256                        # streamed: nothing to keep
    assert size(8192, 4096, 4096, 0) >= 4096 * 4096 * 2             # the weights in bf16
    assert 65 * 4096 // 2 < size(65, 4096, 4096, 1) < 4096 * 4096 * 2
    assert f(8, 64, 16, P, P, P, 2, P, 0, None, 0, None) == EUNSUP
    assert f(8, 48, 16, P, P, P, 0, P, 0, None, 0, None) == EUNSUP
    assert f(-1, 64, 16, P, P, P, 0, P, 0, None, 0, None) == EINVAL
    for i in (3, 4, 5, 7):
        for v in (None, ODD):
            args = [8, 64, 16, P, P, P, 0, P, 0, None, 0, None]
            args[i] = v
            assert f(*args) == EINVAL, (i, v)
    need = size(100, 64, 16, 1)
    assert f(100, 64, 16, P, P, P, 1, P, 0, None, need, None) == EINVAL
    assert f(100, 64, 16, P, P, P, 1, P, 0, P + 16, need, None) == EINVAL
    assert f(100, 64, 16, P, P, P, 1, P, 0, P, need - 1, None) == EWS
    assert f(0, 64, 16, None, None, None, 0, None, 0, None, 0, None) == OK


def test_linear_dx_refusals():
    L = mx.lib()
    size, f = L.moe_linear_mxfp4_dx_workspace_size, L.moe_linear_mxfp4_dx
    assert size(8, 48, 16) == 0 and size(8, 64, 0) == 0
    need = size(8, 64, 17)
    assert need >= 17 * 64 * 2 + 8 * 24 * 2                          # W in bf16, dy in padded rows
    for i in (3, 4, 5, 6):
        args = [8, 64, 17, P, P, P, P, 0, P, need, None]
        args[i] = None
        assert f(*args) == EINVAL, i
    assert f(8, 64, 17, P, P, P, P, 0, P, need - 1, None) == EWS
    assert f(8, 64, 17, P, P, P, P, 0, None, need, None) == EINVAL
    assert f(0, 64, 17, None, None, None, None, 0, None, 0, None) == OK


def test_gated_ffn_refusals():
    L = mx.lib()
    size, f = L.moe_gated_ffn_workspace_size, L.moe_gated_ffn
    for T, H, I in ((-1, 64, 64), (65537, 64, 64), (8, 60, 64), (8, 64, 60), (8, 16392, 64), (8, 64, 16392), (8, 0, 64)):
        assert size(T, H, I) == 0, (T, H, I)
    need = size(8, 64, 64)
    good = [8, 64, 64, 10.0, P, P, P, None, None, P, 0, P, need, None]

    def call(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    for lim in (0.0, -1.0, math.nan):
        assert call(a3=lim) == EINVAL, lim
    for i in (4, 5, 6, 9, 11):
        assert call(**{f"a{i}": None}) == EINVAL, i
        assert call(**{f"a{i}": ODD}) == EINVAL, i
    assert call(a7=P) == EINVAL and call(a8=P) == EINVAL            # saved tensors: both or none
    assert call(a12=need - 1) == EWS
    assert call(a1=60) == EUNSUP
    assert f(0, 64, 64, 10.0, None, None, None, None, None, None, 0, None, 0, None) == OK


def test_gated_ffn_backward_refusals():
    L = mx.lib()
    size, f = L.moe_gated_ffn_backward_workspace_size, L.moe_gated_ffn_backward
    assert size(8, 60, 64) == 0 and size(0, 64, 64) > 0
    need = size(8, 64, 64)
    good = [8, 64, 64, 10.0, P, P, P, P, P, P, P, P, P, 0, P, need, None]

    def call(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    for i in (4, 5, 6, 7, 8, 9, 14):
        assert call(**{f"a{i}": None}) == EINVAL, i
    for i in (4, 5, 6, 7, 8, 9, 10, 11, 12, 14):
        assert call(**{f"a{i}": ODD}) == EINVAL, i
    assert call(a3=math.nan) == EINVAL
    assert call(a15=need - 1) == EWS
    assert call(a2=60) == EUNSUP
    assert f(0, 64, 64, 10.0, None, None, None, None, None, None, None, None, None, 0, None, 0, None) == OK


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(16, 2, dtype=torch.uint8)
    with pytest.raises(ValueError):
        mx.quantize_mxfp4(x)
    with pytest.raises(TypeError):
        mx.quantize_mxfp4([1.0])
    with pytest.raises(TypeError):
        mx.dequantize_mxfp4(c, s, dtype=torch.float16)
    with pytest.raises(ValueError):
        mx.dequantize_mxfp4(c, s)
    with pytest.raises(ValueError):
        mx.linear_mxfp4(x, c, s)
    with pytest.raises(ValueError):
        mx.linear_mxfp4(x, c, s, act="fp8")
    with pytest.raises(ValueError):
        mx.linear_mxfp4_dx(x, c, s)
    w = torch.zeros(32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mx.gated_ffn(x, w, torch.zeros(64, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        mx.gated_ffn_backward(x, x, w, torch.zeros(64, 16, dtype=torch.bfloat16), (x, x))


def test_plain_forms_agree_with_differences():
    """The gradients of the 64-bit form used as the kernels' reference, against central differences of its own
    forward value in every input (error of the differences: eps^2 times third derivatives, 1e-5 here)."""
    import plain64

    torch.manual_seed(0)
    T, H, I, L = 3, 16, 8, 1.0
    x, w13, w2 = (torch.randn(T, H, dtype=torch.float64), torch.randn(2 * I, H, dtype=torch.float64) * 0.4,
                  torch.randn(H, I, dtype=torch.float64))
    dy = torch.randn(T, H, dtype=torch.float64)
    g = (x @ w13.t())
    assert (g > L).any() and (g.abs()[:, I:] > L).any() and ((g.abs() - L).abs() > 1e-3).all()
    res = plain64.ffn(x, w13, w2, L, dy)
    eps = 1e-5
    for name, t in (("dx", x), ("dw13", w13), ("dw2", w2)):
        num = torch.zeros_like(t)
        for i in range(t.numel()):
            v = t.view(-1)[i].item()
            vals = []
            for sgn in (1, -1):
                t.view(-1)[i] = v + sgn * eps
                vals.append((plain64.ffn(x, w13, w2, L)["y"][0] * dy).sum().item())
            t.view(-1)[i] = v
            num.view(-1)[i] = (vals[0] - vals[1]) / (2 * eps)
        assert torch.allclose(num, res[name][0], rtol=1e-6, atol=1e-7), name
