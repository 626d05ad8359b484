"""Host-side checks of the int8 entry points (no GPU): every refusal is returned before anything is launched, and empty
calls succeed."""
import pytest
import torch

mx = pytest.importorskip("mxfp4_moe_expert_amd")

P = 0x100000        # never dereferenced: every call below fails a host check
ODD = 0x100008      # not 16-byte aligned
BYTE = 0x100002     # not 4-byte aligned
OK, EINVAL, EUNSUP, EWS = mx.MOE_OK, mx.MOE_EINVAL, mx.MOE_EUNSUPPORTED, mx.MOE_EWORKSPACE


def test_quantize_refusals():
    f = mx.lib().moe_int8_quantize
    for i in (3, 5, 6):
        args = [4, 64, 0, P, 64, P, P, None]
        args[i] = None
        assert f(*args) == EINVAL, i
    assert f(-1, 64, 0, P, 64, P, P, None) == EINVAL
    assert f(4, 0, 0, P, 64, P, P, None) == EINVAL
    assert f(4, 64, 0, P, 48, P, P, None) == EINVAL      # rows overlap
    assert f(4, 64, 0, P, 68, P, P, None) == EINVAL      # rows not 16-byte aligned
    assert f(4, 64, 1, P, 66, P, P, None) == EINVAL
    assert f(4, 64, 0, ODD, 64, P, P, None) == EINVAL
    assert f(4, 64, 0, P, 64, ODD, P, None) == EINVAL
    assert f(4, 64, 0, P, 64, P, BYTE, None) == EINVAL
    assert f(4, 64, 3, P, 64, P, P, None) == EUNSUP      # dtype
    assert f(4, 40, 0, P, 40, P, P, None) == EUNSUP      # K % 16
    assert f(4, 65552, 0, P, 65552, P, P, None) == EUNSUP
    assert f(1 << 40, 64, 0, P, 64, P, P, None) == EUNSUP
    assert f(0, 64, 0, None, 64, None, None, None) == OK


def test_dequantize_refusals():
    f = mx.lib().moe_int8_dequantize
    assert f(4, 64, None, P, 0, P, None) == EINVAL
    assert f(4, 64, P, None, 0, P, None) == EINVAL
    assert f(4, 64, P, P, 0, None, None) == EINVAL
    assert f(4, 64, P, P, 0, ODD, None) == EINVAL
    assert f(4, 64, P, BYTE, 0, P, None) == EINVAL
    assert f(4, 64, P, P, 2, P, None) == EUNSUP
    assert f(4, 40, P, P, 0, P, None) == EUNSUP
    assert f(0, 64, None, None, 0, None, None) == OK


def test_linear_refusals():
    L = mx.lib()
    size, f = L.moe_linear_w8a8_workspace_size, L.moe_linear_w8a8
    for T, K, N in ((-1, 64, 16), (65537, 64, 16), (8, 40, 16), (8, 65552, 16), (8, 64, 0), (8, 64, 65537)):
        for encoded in (0, 1):
            assert size(T, K, N, encoded) == 0, (T, K, N)
    assert size(1000, 4096, 64, 0) >= 1000 * 4096 + 4000             # codes and scales of the activations
    assert f(8, 40, 16, P, None, None, P, P, P, 0, P, 1 << 20, None) == EUNSUP
    assert f(-1, 64, 16, P, None, None, P, P, P, 0, P, 1 << 20, None) == EINVAL
    # one of x and (codes, scales), whole
    for x, c, s in ((None, None, None), (P, P, P), (P, None, P), (None, P, None), (None, None, P)):
        assert f(100, 64, 16, x, c, s, P, P, P, 0, P, 1 << 20, None) == EINVAL, (x, c, s)
    for i, bad in ((3, ODD), (6, None), (6, ODD), (7, None), (7, BYTE), (8, None), (8, ODD)):
        args = [100, 64, 16, P, None, None, P, P, P, 0, P, 1 << 20, None]
        args[i] = bad
        assert f(*args) == EINVAL, (i, bad)
    for i, bad in ((4, ODD), (5, BYTE)):
        args = [100, 64, 16, None, P, P, P, P, P, 0, P, 1 << 20, None]
        args[i] = bad
        assert f(*args) == EINVAL, (i, bad)
    need = size(100, 64, 16, 0)
    assert f(100, 64, 16, P, None, None, P, P, P, 0, None, need, None) == EINVAL
    assert f(100, 64, 16, P, None, None, P, P, P, 0, P + 16, need, None) == EINVAL
    assert f(100, 64, 16, P, None, None, P, P, P, 0, P, need - 1, None) == EWS
    assert f(0, 64, 16, None, None, None, None, None, None, 0, None, 0, None) == OK


def test_binding_refuses_host_tensors_and_wrong_types():
    x, q, s = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(16, 64, dtype=torch.int8), torch.zeros(16)
    with pytest.raises(ValueError):
        mx.quantize_int8(x)
    with pytest.raises(TypeError):
        mx.quantize_int8([1.0])
    with pytest.raises(TypeError):
        mx.dequantize_int8(q, s, dtype=torch.float16)
    with pytest.raises(ValueError):
        mx.dequantize_int8(q, s)
    with pytest.raises(ValueError):
        mx.linear_w8a8(x, q, s)
    with pytest.raises(ValueError):
        mx.linear_w8a8(q, q, s, x_scale=s)
