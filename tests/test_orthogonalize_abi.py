"""Host-side checks of the orthogonalised update's entry points (no GPU): every refusal is returned before anything is
launched."""
import math

import pytest
import torch

mx = pytest.importorskip("mxfp4_moe_expert_amd")

P = 0x100000        # never dereferenced: every call below fails a host check
ODD = 0x100008      # not 16-byte aligned
OK, EINVAL, EUNSUP, EWS = mx.MOE_OK, mx.MOE_EINVAL, mx.MOE_EUNSUPPORTED, mx.MOE_EWORKSPACE


def test_refusals():
    L = mx.lib()
    size, f = L.moe_orthogonalize_workspace_size, L.moe_orthogonalize
    for B, R, C in ((-1, 8, 8), (65536, 8, 8), (1, 0, 8), (1, 8, 0), (1, 16385, 8), (1, 8, 16385)):
        assert size(B, R, C) == 0, (B, R, C)
    need = size(2, 1001, 640)
    assert need >= 2 * 2 * (3 * 1008 * 640 + 2 * 640 * 640)
    assert size(9, 60, 100) == 256                                   # none used
    assert size(1, 256, 4096) >= 4 * 256 * 4096                      # X in 32 bits
    assert size(65535, 256, 512) < 3 << 30                           # a stack is worked on in parts
    good = [2, 1001, 640, 0, P, 5, 3.4, -4.7, 2.0, 1e-7, P, P, need, None]

    def call(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    for i in (4, 10, 11):
        assert call(**{f"a{i}": None}) == EINVAL, i
    assert call(a10=ODD) == EINVAL and call(a11=ODD) == EINVAL
    assert call(a4=P + 1) == EINVAL and call(a3=1, a4=P + 2) == EINVAL
    assert call(a11=P + 16) == EINVAL
    for i, v in ((0, -1), (1, 0), (2, -3), (5, 0), (9, -1.0), (9, math.nan), (6, math.inf), (7, math.nan), (8, -math.inf)):
        assert call(**{f"a{i}": v}) == EINVAL, (i, v)
    for i, v in ((0, 65536), (1, 16385), (2, 20000), (3, 3), (5, 65)):
        assert call(**{f"a{i}": v}) == EUNSUP, (i, v)
    assert call(a12=need - 1) == EWS
    assert call(a0=0, a4=None, a10=None, a11=None) == OK


def test_binding_refuses_host_tensors_and_wrong_types():
    with pytest.raises(ValueError):
        mx.orthogonalize(torch.zeros(8, 8))
    with pytest.raises(TypeError):
        mx.orthogonalize([[1.0]])
