"""The training operators in one run, as they are used: a frozen int8 projection, the router with its balance loss, the
gated block and its gradients, the router's gradient, and the orthogonalised update of every matrix. Each operator's result
is held to the 64-bit form on the inputs that it had (its roundings do not reach the next one's reference), and the whole
run is captured and replayed."""
import pytest
import torch

import plain64
import train64
from test_gpu_int8 import encode, product
from test_gpu_orthogonalize import hold

pytestmark = pytest.mark.gpu
mx = pytest.importorskip("mxfp4_moe_expert_amd")
DEV = "cuda"
T, K, H, I, E, TOPK, ALPHA = 300, 512, 256, 128, 32, 4, 1e-2
OFFSETS = [0, 120, 120, 290]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def weights(seed):
    g = _gen(seed)

    def randn(*s):
        return torch.randn(*s, generator=g, device=DEV)

    q, scale = mx.quantize_int8(randn(H, K) * 0.05)                 # the frozen projection
    return {"q": q, "scale": scale, "gate": randn(E, H) * 0.05, "bias": randn(E) * 0.01,
            "w13": (randn(2 * I, H) * 0.06).to(torch.bfloat16), "w2": (randn(H, I) * 0.06).to(torch.bfloat16),
            "off": torch.tensor(OFFSETS, dtype=torch.int32, device=DEV)}


def batch(seed):
    g = _gen(seed)
    return (torch.randn(T, K, generator=g, device=DEV).to(torch.bfloat16),
            (torch.randn(T, H, generator=g, device=DEV) * 0.1).to(torch.bfloat16),
            torch.randn(T, TOPK, generator=g, device=DEV) * 1e-3)


def step(cfg, w, x, dy, dtopk, ws):
    h = mx.linear_w8a8(x, w["q"], w["scale"])
    ids, tw, logits = mx.route(cfg, h, w["gate"], w["bias"], ws=ws, return_logits=True)
    loss, counts, aux = mx.balance_loss(logits, ids, w["off"], alpha=ALPHA)
    y, saved = mx.gated_ffn(h, w["w13"], w["w2"], save=True)
    dh, dw13, dw2 = mx.gated_ffn_backward(dy, h, w["w13"], w["w2"], saved)
    dlogits = mx.route_backward(logits, ids, dw=dtopk, saved=aux, scale=cfg.routed_scaling_factor)
    dgate = dlogits.t().contiguous() @ h.float()
    o13 = mx.orthogonalize(dw13.view(2, I, H))
    o2 = mx.orthogonalize(dw2)
    ogate = mx.orthogonalize(dgate)
    return {"h": h, "ids": ids, "tw": tw, "logits": logits, "loss": loss, "counts": counts, "y": y, "dh": dh, "dw13": dw13,
            "dw2": dw2, "dlogits": dlogits, "dgate": dgate, "o13": o13, "o2": o2, "ogate": ogate}


def config():
    return mx.config(hidden_size=H, n_routed_experts=E, top_k=TOPK, moe_intermediate=I)


def test_every_operator_on_the_inputs_it_had():
    cfg, w, (x, dy, dtopk) = config(), weights(1), batch(2)
    r = step(cfg, w, x, dy, dtopk, mx.Workspace(DEV))
    y, b = product(*encode(x), w["q"], w["scale"], plain64.U16)
    plain64.check(r["h"], y, b, "projection")
    h = r["h"].double()
    z = h @ w["gate"].double().t()
    assert bool(((r["logits"].double() - z).abs() <= (H + 64) * 2.0 ** -24 * (h.abs() @ w["gate"].double().abs().t() + 1)).all())
    ref = train64.router(r["logits"].double(), r["ids"], OFFSETS, alpha=ALPHA, scale=cfg.routed_scaling_factor, dw=dtopk)
    assert abs(float(r["loss"]) - float(ref["loss"])) <= float(ref["eloss"])
    assert torch.equal(r["counts"], ref["counts"])
    assert int(r["counts"].sum()) == (OFFSETS[-1] - OFFSETS[0]) * TOPK
    plain64.check(r["dlogits"], ref["dz"], ref["edz"], "dlogits")
    block = plain64.ffn(h, w["w13"].double(), w["w2"].double(), 10.0, dy.double())
    for name in ("y", "dw13", "dw2"):
        plain64.check(r[name], *block[name], name)
    plain64.check(r["dh"], *block["dx"], "dh")
    for i in range(2):
        hold(r["o13"][i], r["dw13"].view(2, I, H)[i])
    hold(r["o2"], r["dw2"])
    hold(r["ogate"], r["dgate"])


def test_the_update_follows_its_gradient():
    """<dw, update> is the sum of singular values times theirs, and each
    of those lies above 0.6 of a singular value that is not tiny."""
    cfg, w, (x, dy, dtopk) = config(), weights(3), batch(4)
    r = step(cfg, w, x, dy, dtopk, mx.Workspace(DEV))
    for g, o in ((r["dw13"].view(2, I, H)[0], r["o13"][0]), (r["dw2"], r["o2"])):
        s = torch.linalg.svdvals(g.double())
        along = float((g.double() * o.double()).sum())
        assert along >= 0.6 * float(s[s > 0.02 * s.norm()].sum())
        assert along <= 1.25 * float(s.sum())


def test_captured_and_replayed():
    cfg, w, ws = config(), weights(5), mx.Workspace(DEV)
    batches = [batch(10 + i) for i in range(3)]
    want = [{k: v.clone() for k, v in step(cfg, w, *b, ws).items()} for b in batches]
    torch.cuda.synchronize()
    held = [t.clone() for t in batches[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cfg, w, *held, ws)
    for i in (1, 2, 0, 1):
        for dst, src in zip(held, batches[i]):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for name in want[i]:
            if name not in ("dgate", "ogate"):                       # a library product's, which may be cut otherwise
                assert torch.equal(out[name], want[i][name]), (i, name)
        hold(out["ogate"], out["dgate"])
        eager = step(cfg, w, *batches[2], ws)
        torch.cuda.synchronize()
        assert torch.equal(eager["o13"], want[2]["o13"]) and torch.equal(eager["dlogits"], want[2]["dlogits"])
