"""GPU tests of the router's training operators against the 64-bit forms of tests/train64.py: the balance loss, the counts
and the gradient of the logits, over group sizes, ragged and empty sequences, padding and values at the edges."""
import pytest
import torch

import train64
from plain64 import check

pytestmark = pytest.mark.gpu
mx = pytest.importorskip("mxfp4_moe_expert_amd")
DEV = "cuda"


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _batch(seed, T, E, k, spread=1.5):
    g = _gen(seed)
    z = torch.randn(T, E, generator=g, device=DEV) * spread + torch.randn(E, generator=g, device=DEV)
    key = z + 0.3 * torch.randn(T, E, generator=g, device=DEV)
    ids = torch.topk(key, min(k, E), dim=1).indices
    if k > E:  # more slots than experts: some stand twice
        ids = torch.cat((ids, torch.randint(0, E, (T, k - E), generator=g, device=DEV)), dim=1)
    return z, ids.to(torch.int32), torch.randn(T, k, generator=g, device=DEV)


def _offsets(seed, T, S, pad=0):
    g = torch.Generator()
    g.manual_seed(seed)
    cut = torch.sort(torch.randint(0, T - pad + 1, (S - 1,), generator=g)).values
    return torch.cat((torch.zeros(1), cut, torch.tensor([float(T - pad)]))).to(torch.int32).to(DEV)


def _hold(z, ids, off, dw, alpha=0.01, scale=1.5, dloss=None):
    loss, counts, saved = mx.balance_loss(z, ids, off, alpha=alpha)
    borders = None if off is None else off.tolist()
    d = 1.0 if dloss is None else float(dloss)
    for bal, w in ((True, None), (True, dw), (False, dw)):
        r = train64.router(z.double(), ids, borders, alpha=alpha, scale=scale, dloss=d, dw=w, balance=bal)
        if bal:
            assert abs(float(loss) - float(r["loss"])) <= float(r["eloss"]) + 1e-37
            assert torch.equal(counts, r["counts"])
            got = mx.route_backward(z, ids, dw=w, saved=saved, scale=scale, dloss=dloss)
            check(got, r["dz"], r["edz"], f"dz, dw {w is not None}")
        elif borders is None:
            got = mx.route_backward(z, ids, dw=w, scale=scale)
            check(got, r["dz"], r["edz"], "dz of the weights alone")
    return loss, counts, saved


# experts: both sides of every group size (32, 64, 128), not multiples of four, one, the most; tokens: one, those around
# the runs' borders and counts
@pytest.mark.parametrize("E,k", [(1, 1), (2, 3), (5, 2), (8, 8), (31, 3), (32, 6), (33, 4), (64, 6), (65, 1), (100, 7),
                                 (128, 8), (130, 6), (192, 6), (255, 5), (256, 6)])
@pytest.mark.parametrize("T", [1, 2, 31, 33, 129, 1000])
def test_one_sequence(T, E, k):
    z, ids, dw = _batch(T + E, T, E, k)
    _hold(z, ids, None, dw)


@pytest.mark.parametrize("T,E,S,pad", [(64, 256, 2, 0), (256, 256, 8, 1), (257, 256, 8, 1), (256, 256, 9, 1),
                                       (2048, 32, 5, 7), (2049, 32, 5, 7), (1500, 8, 1025, 2), (64, 60, 9, 3), (777, 64, 5, 30), (4097, 256, 7, 82),
                                       (8193, 128, 33, 0), (300, 16, 299, 1), (33, 256, 200, 5), (8200, 255, 3, 8199)])
def test_ragged_sequences_and_padding(T, E, S, pad):
    z, ids, dw = _batch(T, T, E, 6)
    _hold(z, ids, _offsets(S, T, S, pad), dw, dloss=torch.full((1,), -2.5, device=DEV))


def test_largest_batch():
    z, ids, dw = _batch(1, 65536, 256, 6)
    _hold(z, ids, _offsets(5, 65536, 16, 100), dw)


def test_sequences_behind_an_offset_and_all_empty():
    z, ids, dw = _batch(2, 100, 32, 4)
    off = torch.tensor([10, 10, 40, 40, 90], dtype=torch.int32, device=DEV)
    _, _, saved = _hold(z, ids, off, dw)
    dz = mx.route_backward(z, ids, dw=dw, saved=saved)
    assert not dz[:10].any() and not dz[90:].any() and bool(dz[10:90].abs().sum(1).gt(0).all())
    for off in ([0, 0], [100, 100, 100], [7, 7, 7, 7]):
        off = torch.tensor(off, dtype=torch.int32, device=DEV)
        loss, counts, saved = mx.balance_loss(z, ids, off, alpha=1.0)
        assert float(loss) == 0.0 and not counts.any()
        assert not mx.route_backward(z, ids, dw=dw, saved=saved).any()


def test_empty_batch():
    z, ids = torch.empty(0, 64, device=DEV), torch.empty(0, 6, dtype=torch.int32, device=DEV)
    loss, counts, saved = mx.balance_loss(z, ids)
    assert float(loss) == 0.0 and counts.shape == (64,) and not counts.any()
    assert mx.route_backward(z, ids, saved=saved).shape == (0, 64)


@pytest.mark.parametrize("E", [32, 100, 256])
def test_logits_at_the_edges(E):
    """Masked experts (-inf, the type's lowest value), logits far on either side, rows with one live expert and with none."""
    z, ids, dw = _batch(9, 70, E, 4)
    z[:, 3] = float("-inf")
    z[:, 7] = torch.finfo(torch.float32).min
    z[5] *= 20.0
    z[6] = -90.0
    z[7] = 60.0
    z[8, ::2] = -160.0
    z[9] = float("-inf")
    z[9, 11] = 0.5
    z[10] = float("-inf")
    z[11] = torch.finfo(torch.float32).min
    z[12] = torch.linspace(-17.5, -16.5, E, device=DEV)
    r = train64.router(z.double(), ids, None, alpha=0.3, scale=1.5, dw=dw)
    loss, counts, saved = mx.balance_loss(z, ids, alpha=0.3)
    assert abs(float(loss) - float(r["loss"])) <= float(r["eloss"])
    got = mx.route_backward(z, ids, dw=dw, saved=saved)
    assert bool(torch.isfinite(got).all())
    masked = z <= torch.finfo(torch.float32).min
    assert int(masked.sum()) > 130 and not got[masked].any()
    ok = torch.ones(70, dtype=torch.bool, device=DEV)
    ok[10:12] = False  # 0 by definition; the 64-bit form agrees but has no bound to speak of
    check(got[ok], r["dz"][ok], r["edz"][ok], "dz")


@pytest.mark.parametrize("T,E", [(6, 8), (700, 8), (700, 256)])
def test_scores_below_the_normal_range_have_no_shares(T, E):
    """exp(-100 / 2) is normal; 256 exp(-97) is not, and its inverse would be infinite."""
    z, ids, dw = _batch(31, T, E, 6)
    low, none = z.clone(), z.clone()
    low[1], none[1] = -194.0, float("-inf")
    low[3], none[3] = -100.0, -100.0
    a, b = mx.balance_loss(low, ids, alpha=0.01), mx.balance_loss(none, ids, alpha=0.01)
    assert bool(torch.isfinite(a[0])) and float(a[0]) == float(b[0])
    d = mx.route_backward(low, ids, dw, a[2])
    assert bool(torch.isfinite(d).all()) and bool((d[1] == 0).all())
    assert torch.equal(d, mx.route_backward(none, ids, dw, b[2]))


def test_nan_logits_stay_in_their_row():
    z, ids, dw = _batch(9, 70, 64, 4)
    _, _, saved = mx.balance_loss(z, ids)
    a = mx.route_backward(z, ids, dw=dw, saved=saved)
    z2 = z.clone()
    z2[30, 5] = float("nan")
    loss, counts, saved2 = mx.balance_loss(z2, ids)
    assert bool(loss.isnan()) and int(counts.sum()) == 70 * 4
    b = mx.route_backward(z2, ids, dw=dw, saved=saved2)
    assert bool(b[30].isnan().any())
    assert torch.equal(torch.cat((a[:30], a[31:])), torch.cat((b[:30], b[31:])))


def test_ids_and_offsets_out_of_range_are_flagged():
    z, ids, dw = _batch(4, 200, 64, 6)
    mx.device_flags(clear=True)
    want = train64.router(z.double(), ids, None, alpha=1.0)
    bad = ids.clone()
    bad[3, 2], bad[77, 0], bad[199, 5] = -1, 64, 2 ** 31 - 1
    r = train64.router(z.double(), bad, None, alpha=1.0, scale=1.5, dw=dw)
    loss, counts, saved = mx.balance_loss(z, bad, alpha=1.0)
    assert mx.device_flags(clear=True) == {"expert_id"}
    assert torch.equal(counts, r["counts"]) and int(counts.sum()) == int(want["counts"].sum()) - 3
    check(mx.route_backward(z, bad, dw=dw, saved=saved), r["dz"], r["edz"], "dz")
    assert mx.device_flags(clear=True) == {"expert_id"}
    for off in ([0, 150, 100, 200], [0, 300], [-5, 200], [200, 0], [150, 20, 170, -3, 4000]):
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        loss, counts, saved = mx.balance_loss(z, ids, o)
        assert bool(loss.isnan()), off
        mx.route_backward(z, ids, dw=dw, saved=saved)
        assert mx.device_flags(clear=True) == {"sequence"}, off


def test_results_do_not_depend_on_timing():
    z, ids, dw = _batch(3, 20000, 256, 6)
    off = _offsets(8, 20000, 40)
    first = None
    for _ in range(4):
        loss, counts, saved = mx.balance_loss(z, ids, off)
        d = mx.route_backward(z, ids, dw=dw, saved=saved)
        got = (loss, counts, saved[0][:40 * 256 + 1], d)
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(got, first))
        first = tuple(t.clone() for t in got)


def test_gradient_against_differences_of_the_loss():
    """Along the gradient v, loss(z + h v) - loss(z - h v) = 2 h |v|^2 up to h^3 third derivatives and the losses' own
    errors; h moves the largest logit by 0.02, where the third-order part is below (0.02)^2 of the whole."""
    z, ids, _ = _batch(6, 300, 64, 6)
    off = torch.tensor([0, 100, 300], dtype=torch.int32, device=DEV)
    _, _, saved = mx.balance_loss(z, ids, off, alpha=1.0)
    v = mx.route_backward(z, ids, saved=saved).double()
    h = 0.02 / float(v.abs().max())
    zp, zm = (z.double() + h * v).float(), (z.double() - h * v).float()
    lp, lm = (float(mx.balance_loss(t, ids, off, alpha=1.0)[0]) for t in (zp, zm))
    moved = float(((zp.double() - zm.double()) * v).sum())
    noise = sum(float(train64.router(t.double(), ids, [0, 100, 300], alpha=1.0)["eloss"]) for t in (zp, zm))
    assert abs((lp - lm) - moved) <= 1e-3 * moved + noise


def test_workspace_is_enough_and_outputs_alone_are_written():
    for T, E, S in ((1, 3, 1), (100, 37, 4), (100, 37, 9), (3000, 256, 6)):
        z, ids, dw = _batch(T, T, E, 3)
        off = _offsets(S, T, S) if S > 1 else None
        want = mx.balance_loss(z, ids, off)
        need = mx.lib().moe_balance_workspace_size(T, E, S)
        ws = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device=DEV)
        got = mx.balance_loss(z, ids, off, ws=ws[:need])
        assert bool((ws[need:] == 0xAB).all())
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        buf = torch.full((T * E + 32,), 7.0, device=DEV)
        out = buf[16:16 + T * E].view(T, E)
        assert mx.route_backward(z, ids, dw=dw, saved=got[2], out=out) is out
        assert bool((buf[:16] == 7).all()) and bool((buf[16 + T * E:] == 7).all())
        assert torch.equal(out, mx.route_backward(z, ids, dw=dw, saved=want[2]))


def test_refusals_on_device():
    z, ids, dw = _batch(0, 8, 64, 6)
    off = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    saved = mx.balance_loss(z, ids, off)[2]
    for bad in (lambda: mx.balance_loss(z[:4], ids), lambda: mx.balance_loss(z.t(), ids),
                lambda: mx.balance_loss(z, ids, off[:1]), lambda: mx.balance_loss(z, ids, off.view(1, 2)),
                lambda: mx.balance_loss(z, ids, off.cpu()), lambda: mx.route_backward(z, ids),
                lambda: mx.route_backward(z, ids, dw=dw[:, :5]), lambda: mx.route_backward(z, ids, dw=dw[:4]),
                lambda: mx.route_backward(z, ids, saved=(saved[0][:-1],) + saved[1:]),
                lambda: mx.route_backward(z[:, :32].contiguous(), ids, saved=saved),
                lambda: mx.route_backward(z, ids, saved=saved, dloss=torch.ones(2, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: mx.balance_loss(z.double(), ids), lambda: mx.balance_loss(z, ids.long()),
                lambda: mx.balance_loss(z, ids, off.long()), lambda: mx.route_backward(z, ids, dw=dw.half())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(mx.MoEError):
        mx.balance_loss(torch.zeros(4, 300, device=DEV), ids[:4])
    with pytest.raises(mx.MoEError):
        mx.balance_loss(z, torch.zeros(8, 9, dtype=torch.int32, device=DEV))
    with pytest.raises(mx.MoEError, match="logits: not 16-byte"):
        mx.balance_loss(torch.zeros(8 * 64 + 1, device=DEV)[1:].view(8, 64), ids)


def test_on_two_streams_and_in_graphs():
    T, E = 900, 128
    off = torch.tensor([0, 200, 200, 850], dtype=torch.int32, device=DEV)
    batches = [_batch(20 + i, T, E, 6) for i in range(4)]

    def step(z, ids, dw):
        loss, counts, saved = mx.balance_loss(z, ids, off, alpha=0.1)
        return loss, counts, mx.route_backward(z, ids, dw=dw, saved=saved)

    want = [step(*b) for b in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i, b in enumerate(batches):
        with torch.cuda.stream(streams[i % 2]):
            got.append(step(*b))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    held = [[t.clone() for t in b] for b in batches[:2]]
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*held[i]))
        graphs.append(g)
    for r in range(3):
        for i in range(2):
            for dst, src in zip(held[i], batches[(r + i) % 4]):
                dst.copy_(src)
            graphs[i].replay()
        eager = step(*batches[3])
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(eager, want[3]))
        for i in range(2):
            assert all(torch.equal(u, v) for u, v in zip(outs[i], want[(r + i) % 4])), (r, i)


@pytest.mark.parametrize("T", [1, 5, 64, 65, 300])
@pytest.mark.parametrize("E", [16, 100, 256])
def test_route_returns_its_logits(T, E):
    """The logits are the fp32 sums the scores come from: ids and weights as without them, weights recomputed from them,
    and the products in 64 bits within the sum's error (H products, the router splitting gate_w into bf16 parts)."""
    H, k = 512, 4
    cfg = mx.config(hidden_size=H, n_routed_experts=E, top_k=k, moe_intermediate=128)
    g = _gen(T + E)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    gw = torch.randn(E, H, generator=g, device=DEV) * 0.05
    bias, lo = torch.randn(E, generator=g, device=DEV) * 0.1, torch.randn(E, generator=g, device=DEV) * 0.1
    for offset in (None, lo):
        ids, w, z = mx.route(cfg, x, gw, bias, logit_offset=offset, return_logits=True)
        ids0, w0 = mx.route(cfg, x, gw, bias, logit_offset=offset)
        assert torch.equal(ids, ids0) and torch.equal(w, w0)
        ref = x.double() @ gw.double().t() + (0 if offset is None else lo.double())
        absum = x.double().abs() @ gw.double().abs().t() + 1
        assert bool(((z.double() - ref).abs() <= (H + 64) * 2.0 ** -24 * absum).all())
        s, _ = train64.scores(z.double())
        sj = s.gather(1, ids.long())
        assert torch.allclose(w.double(), 1.5 * sj / sj.sum(1, keepdim=True), rtol=1e-5, atol=0)
