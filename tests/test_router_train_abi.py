"""Host-side checks of the router's training entry points (no GPU), and the 64-bit form used as their reference against
differences of its own values."""
import pytest
import torch

mx = pytest.importorskip("mxfp4_moe_expert_amd")

P = 0x100000        # never dereferenced: every call below fails a host check
ODD = 0x100008      # not 16-byte aligned
BYTE = 0x100002     # not 4-byte aligned
OK, EINVAL, EUNSUP, EWS = mx.MOE_OK, mx.MOE_EINVAL, mx.MOE_EUNSUPPORTED, mx.MOE_EWORKSPACE


def test_balance_loss_refusals():
    L = mx.lib()
    size, f = L.moe_balance_workspace_size, L.moe_balance_loss
    for T, E, S in ((-1, 8, 1), (65537, 8, 1), (8, 0, 1), (8, 257, 1), (8, 8, 0), (8, 8, 65537)):
        assert size(T, E, S) == 0
    need = size(5000, 64, 3)
    good = [5000, 64, 6, 3, P, P, P, 1e-3, P, P, P, P, need, None]

    def call(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    for i in (4, 5, 6, 8, 9, 10, 11):
        assert call(**{f"a{i}": None}) == EINVAL, i
        assert call(**{f"a{i}": BYTE}) == EINVAL, i
    assert call(a4=ODD) == EINVAL and call(a11=P + 16) == EINVAL
    assert call(a12=need - 1) == EWS
    assert size(64, 256, 1) == 256                                  # none used
    assert call(a0=-1) == EINVAL and call(a1=0) == EINVAL and call(a2=0) == EINVAL and call(a3=0) == EINVAL
    assert call(a0=65537) == EUNSUP and call(a1=257) == EUNSUP and call(a2=9) == EUNSUP and call(a3=65537) == EUNSUP


def test_route_backward_refusals():
    f = mx.lib().moe_route_backward
    good = [100, 64, 6, 3, P, P, P, P, P, P, 1.5, P, None]

    def call(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    for i in (4, 5, 6, 11):
        assert call(**{f"a{i}": None}) == EINVAL, i
    for i in (4, 5, 6, 7, 8, 9, 11):
        assert call(**{f"a{i}": BYTE}) == EINVAL, i
    assert call(a4=ODD) == EINVAL and call(a11=ODD) == EINVAL
    assert call(a7=None, a9=None) == EINVAL                         # nothing to compute
    assert call(a0=-1) == EINVAL and call(a2=9) == EUNSUP and call(a1=257) == EUNSUP
    assert call(a0=0, a4=None, a5=None, a11=None) == OK


def test_route_logits_refusals():
    import ctypes

    cfg = mx.config(hidden_size=256, n_routed_experts=16, moe_intermediate=128)
    need = mx.workspace_size(cfg, 8)
    good = [ctypes.byref(cfg), 8, P, P, P, None, P, P, P, P, need, None]
    for i in (2, 3, 4, 6, 7, 9):
        a = list(good)
        a[i] = None
        assert mx.lib().moe_route_logits(*a) == EINVAL, i
    a = list(good)
    a[8] = ODD
    assert mx.lib().moe_route_logits(*a) == EINVAL


def test_binding_refuses_host_tensors_and_wrong_shapes():
    z, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        mx.balance_loss(z, ids)
    with pytest.raises(ValueError):
        mx.route_backward(z, ids, dw=torch.zeros(4, 2))


@pytest.mark.parametrize("with_dw", [False, True])
def test_plain_form_agrees_with_differences(with_dw):
    """Central differences of the 64-bit loss (and of <w, dw>) in every logit: eps^2 times third derivatives, 1e-8 here."""
    import train64

    torch.manual_seed(0)
    T, E, k = 7, 6, 2
    z = torch.randn(T, E, dtype=torch.float64) * 2
    ids = torch.stack([torch.randperm(E)[:k] for _ in range(T)]).to(torch.int32)
    ids[3, 1] = ids[3, 0]                                           # the same expert twice
    off = [0, 3, 3, 6]                                              # an empty sequence; the last token in none
    dw = torch.randn(T, k, dtype=torch.float64) if with_dw else None

    def value(z):
        r = train64.router(z, ids, off, alpha=0.7)
        v = 1.3 * r["loss"]
        if with_dw:
            s = r["s"][:6].gather(1, ids[:6].long())
            v = v + (2.5 * s / s.sum(1, keepdim=True) * dw[:6]).sum()
        return v

    got = train64.router(z, ids, off, alpha=0.7, scale=2.5, dloss=1.3, dw=dw)["dz"]
    eps = 1e-5
    for t in range(T):
        for e in range(E):
            d = torch.zeros_like(z)
            d[t, e] = eps
            num = (value(z + d) - value(z - d)) / (2 * eps)
            assert abs(num - got[t, e]) <= 1e-7 * (1 + abs(num)), (t, e)
