"""Cases of the int8 x int8 products, the router's training operators and the orthogonalised update, for timing and
comparison.

Each case is one call (or the calls of one training step) of an operator on inputs made from a seed. `run` computes it
either through the library (`own` true) or in plain torch operations in 32 bits (`own` false); `exact` gives the same
outputs in 64 bits from the operators' definitions, written apart from both.

Operators:
  quantize  x [rows][K] -> int8 codes and one fp32 scale per row (symmetric), and back to the values they stand for
  linear    y = x W^T with W in int8 and a scale per output channel, x rounded to int8 with a scale per token
  router    the balance loss of a routed batch, its per-expert counts, and the gradient of the router's logits from
            that loss and (dw true) from the routing weights
  ortho     Newton-Schulz orthogonalisation of a stack of gradient matrices
"""
import torch

own = False

ALPHA = 1e-3         # weight of the balance loss
SCALE = 1.5          # the layer's routed_scaling_factor
STEPS = 5            # Newton-Schulz steps, and their coefficients
COEF = (3.4445, -4.7750, 2.0315)
EPS = 1e-7

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decode batch's activations on their way into an int8 product: launch latency
        {"name": "quantize_int8_tokens_64x4096", "op": "quantize", "rows": 64, "K": 4096, "dtype": "bf16"},
        # fp32 master weights of a stack of projections rewritten into the int8 storage format: bandwidth
        {"name": "quantize_int8_weights_16384x4096", "op": "quantize", "rows": 16384, "K": 4096, "dtype": "f32"},
        # one token through the fused query / key-value down projection: the smallest product
        {"name": "linear_w8a8_t1_4096_1536", "op": "linear", "T": 1, "K": 4096, "N": 1536},
        # an odd decode batch through the attention output projection: weight bytes
        {"name": "linear_w8a8_t33_8192_4096", "op": "linear", "T": 33, "K": 8192, "N": 4096},
        # a prompt of ordinary length, not a multiple of any tile
        {"name": "linear_w8a8_t1000_4096_4096", "op": "linear", "T": 1000, "K": 4096, "N": 4096},
        # a full prefill batch
        {"name": "linear_w8a8_t8192_4096_4096", "op": "linear", "T": 8192, "K": 4096, "N": 4096},
        # the router's loss and gradient over a small batch of one sequence: latency
        {"name": "router_balance_t64_e256", "op": "router", "T": 64, "E": 256, "k": 6, "S": 1, "dw": False},
        # a training batch of ragged sequences, one of them empty, with the routing weights' gradient; padding at the end
        {"name": "router_train_t4097_e256_s7", "op": "router", "T": 4097, "E": 256, "k": 6, "S": 7, "dw": True},
        # the largest batch of the layer
        {"name": "router_balance_t65536_e256_s16", "op": "router", "T": 65536, "E": 256, "k": 6, "S": 16, "dw": False},
        # the router's own weight gradient: a wide matrix
        {"name": "ortho_gate_256x4096", "op": "ortho", "B": 1, "R": 256, "C": 4096, "dtype": "f32"},
        # a few narrow experts' matrices of odd sizes, taller than wide
        {"name": "ortho_odd_3x1001x600", "op": "ortho", "B": 3, "R": 1001, "C": 600, "dtype": "bf16"},
        # gate and up matrices of the gated block at the layer's sizes
        {"name": "ortho_w13_2x2048x4096", "op": "ortho", "B": 2, "R": 2048, "C": 4096, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], uniform over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "linear", "router", "router", "router", "ortho", "ortho", "ortho"])
    if op == "quantize":
        K = 16 * _log_int(rng, 4, 512)
        return {"op": op, "rows": _log_int(rng, 1, 16384), "K": K, "dtype": rng.choice(["bf16", "f32", "f16"])}
    if op == "linear":
        T, K = _log_int(rng, 1, 8192), 16 * _log_int(rng, 8, 512)
        # output features: mostly multiples of 16, as projections have; sometimes any number
        N = 16 * _log_int(rng, 8, 512)
        if rng.random() < 0.25:
            N += rng.randrange(1, 16)
        while T * K * N > 8192 * 4096 * 4096:
            T = max(1, T // 2)
        return {"op": op, "T": T, "K": K, "N": N}
    if op == "router":
        # experts: mostly multiples of 8, as layers have; sometimes any number
        E = 8 * _log_int(rng, 1, 32)
        if rng.random() < 0.25 and E < 256:
            E += rng.randrange(1, 8)
        return {"op": op, "T": _log_int(rng, 1, 65536), "E": E, "k": rng.randrange(1, 9) if E >= 8 else 1,
                "S": _log_int(rng, 1, 64), "dw": rng.random() < 0.5}
    B, R, C = _log_int(rng, 1, 8), _log_int(rng, 16, 4096), _log_int(rng, 16, 4096)
    if rng.random() < 0.5:
        R, C = max(16, R // 16 * 16), max(16, C // 16 * 16)
    while B * min(R, C) ** 2 * (max(R, C) + min(R, C) / 3) > 2 * 2048 ** 2 * (4096 + 2048 / 3):
        R, C = max(1, R * 3 // 4), max(1, C * 3 // 4)
    return {"op": op, "B": B, "R": R, "C": C, "dtype": rng.choice(["bf16", "f32"])}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _tokens(g, T, K):
    """Activations: N(0, 1) with a few channels eight times as large, as hidden states have them."""
    x = _randn(g, T, K)
    x[:, torch.randint(0, K, (max(1, K // 128),), generator=g, device="cuda")] *= 8.0
    return x


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op == "quantize":
        x = _tokens(g, case["rows"], case["K"])
        if case["dtype"] == "f32":
            x *= 0.02  # master weights
        st["x"] = x.to(_DTYPES[case["dtype"]])
    elif op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        w = _randn(g, N, K) * 0.02
        st["q"], st["scale"] = _plain_quantize(w)
        st["x"] = _tokens(g, T, K).to(torch.bfloat16)
    elif op == "router":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        # the logits of unit activations, some experts preferred; the chosen experts have the largest score + bias
        st["logits"] = 1.28 * _randn(g, T, E) + 0.7 * _randn(g, E)
        score = torch.nn.functional.softplus(st["logits"]).sqrt()
        st["ids"] = torch.topk(score + 0.1 * _randn(g, E), k, dim=1).indices.to(torch.int32)
        # S ragged sequences, about one in eight empty; with several, a few tokens of padding behind the last
        cut = torch.rand(S, generator=g, device="cuda")
        part = cut * (torch.rand(S, generator=g, device="cuda") > 0.125)
        part[torch.randint(0, S, (1,), generator=g, device="cuda")] = 1.0
        live = T if S == 1 else max(1, T - T // 50)
        ends = (part.double().cumsum(0) / part.double().sum() * live).round().to(torch.int32)
        st["offsets"] = torch.cat((torch.zeros(1, dtype=torch.int32, device="cuda"), ends))
        st["dw"] = _randn(g, T, k) * 1e-6 if case["dw"] else None
    else:
        B, R, C = case["B"], case["R"], case["C"]
        rank = max(1, min(R, C) // 8)
        # a gradient: some strong directions of falling size over a floor of noise
        left = _randn(g, B, R, rank) * torch.logspace(0, -1.5, rank, device="cuda")
        st["g"] = (1e-3 * (left @ _randn(g, B, rank, C) + 0.3 * _randn(g, B, R, C))).to(_DTYPES[case["dtype"]])
    return st


# ---------------------------------------------------------------- plain forms (32 bits)

def _plain_quantize(x):
    """x [R][K] -> codes [R][K] int8, scales [R] fp32: the row's largest magnitude over 127 (1 for a row of zeros), each
    value over it rounded to the nearest whole number, ties to even; a row with a value that is not finite: scale NaN.
    The quotients are taken in 64 bits: in 32 some land on the border between two codes that lie beside it."""
    v = x.to(torch.float32)
    top = v.abs().amax(dim=1)
    finite = torch.isfinite(v).all(dim=1)
    # division by a tensor: by a plain number torch multiplies with the rounded reciprocal
    s = torch.clamp(top / torch.full_like(top, 127.0), min=2.0 ** -126)
    s = torch.where(top == 0, torch.ones_like(s), s)
    s = torch.where(finite, s, torch.full_like(s, float("nan")))
    q = torch.round(v.double() / s.unsqueeze(1).double())
    q = torch.where(finite.unsqueeze(1), q, torch.zeros_like(q))
    return q.clamp(-127, 127).to(torch.int8), s


def _plain_router(st):
    case = st["case"]
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    z, ids, off = st["logits"], st["ids"].long(), st["offsets"].long()
    dev = z.device
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(off, t, right=True) - 1            # S: behind the last sequence
    live = seq < S
    seq = seq.clamp(max=S - 1)
    lengths = (off[1:] - off[:-1]).float()
    soft = torch.clamp(z, min=0.0) + torch.log1p(torch.exp(-z.abs()))
    s = torch.sqrt(soft)
    total = s.sum(dim=1, keepdim=True)
    p = s / total
    slot = (seq.unsqueeze(1) * E + ids).reshape(-1)
    c = torch.zeros(S * E, device=dev).index_add_(0, slot, live.unsqueeze(1).expand(T, k).reshape(-1).float()).view(S, E)
    member = (seq.unsqueeze(0) == torch.arange(S, device=dev).unsqueeze(1)) & live.unsqueeze(0)
    mean_p = (member.float() @ p) / lengths.clamp(min=1).unsqueeze(1)
    f = c * (E / k) / lengths.clamp(min=1).unsqueeze(1)
    nonempty = (lengths > 0).sum().clamp(min=1).float()
    loss = ALPHA * (f * mean_p).sum() / nonempty
    fr = f[seq]
    lead = torch.where(live, ALPHA / nonempty / lengths.clamp(min=1)[seq], torch.zeros_like(total[:, 0])).unsqueeze(1)
    ds = lead * (fr - (fr * p).sum(dim=1, keepdim=True)) / total
    if st["dw"] is not None:
        sj = torch.gather(s, 1, ids)
        norm = sj.sum(dim=1, keepdim=True)
        dsj = SCALE / norm * (st["dw"] - (st["dw"] * sj).sum(dim=1, keepdim=True) / norm)
        ds = ds + torch.zeros_like(ds).scatter_add_(1, ids, torch.where(live.unsqueeze(1), dsj, torch.zeros_like(dsj)))
    sig = 1.0 / (1.0 + torch.exp(-z))
    return loss, c.sum(dim=0).to(torch.int32), ds * sig / (2.0 * s)


def _plain_ortho(g):
    a, b, c = COEF
    x = g.to(torch.float32)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / ((x * x).sum(dim=(1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2).contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return (x.transpose(1, 2) if tall else x).to(torch.bfloat16).contiguous()


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        q, s = _plain_quantize(st["x"])
        return (q.float() * s.unsqueeze(1)).to(_out_dtype(case))
    if op == "linear":
        xq, xs = _plain_quantize(st["x"])
        y = xq.float() @ st["q"].float().t()
        return (y * xs.unsqueeze(1) * st["scale"].unsqueeze(0)).to(torch.bfloat16)
    if op == "router":
        return _plain_router(st)
    return _plain_ortho(st["g"])


def _out_dtype(case):
    """The values of the codes come back in fp32 for fp32 inputs, else in bf16."""
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


# ---------------------------------------------------------------- one pass

def run(st):
    if not own:
        return _plain(st)
    import mxfp4_moe_expert_amd as mx

    case = st["case"]
    op = case["op"]
    if op == "quantize":
        q, s = mx.quantize_int8(st["x"])
        return mx.dequantize_int8(q, s, dtype=_out_dtype(case))
    if op == "linear":
        return mx.linear_w8a8(st["x"], st["q"], st["scale"])
    if op == "router":
        loss, counts, saved = mx.balance_loss(st["logits"], st["ids"], st["offsets"], alpha=ALPHA)
        dlogits = mx.route_backward(st["logits"], st["ids"], dw=st["dw"], saved=saved, scale=SCALE)
        return loss, counts, dlogits
    return mx.orthogonalize(st["g"], steps=STEPS, coefficients=COEF, eps=EPS)


def work(case):
    op = case["op"]
    if op == "quantize":
        n, rows = case["rows"] * case["K"], case["rows"]
        size = 4 if case["dtype"] == "f32" else 2
        # x in, codes and scales out and in again, values out; two operations a value each way
        return {"bytes": n * size + 2 * (n + 4 * rows) + n * size, "flops": 4 * n}
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": N * K + 4 * N + 2 * T * (K + N), "flops": 2 * T * K * N}
    if op == "router":
        T, E, k = case["T"], case["E"], case["k"]
        # logits, ids (and the weights' gradient) in, the logits' gradient out; about 20 operations a logit
        return {"bytes": 2 * 4 * T * E + 4 * T * k * (2 if case["dw"] else 1), "flops": 20 * T * E}
    B, m, n = case["B"], min(case["R"], case["C"]), max(case["R"], case["C"])
    size = 4 if case["dtype"] == "f32" else 2
    # half of the two symmetric products, and the third whole
    return {"bytes": B * m * n * (size + 2), "flops": STEPS * B * (m * m * n + m * m * m + 2 * m * m * n)}


# ---------------------------------------------------------------- 64 bits, from the definitions

def _exact_int8(x):
    """Codes and scales of x [R][K] as 64-bit numbers; a scale is the fp32 value that is stored."""
    v = x.double()
    top = v.abs().max(dim=1, keepdim=True).values
    s = torch.where(top > 0, (top / 127).clamp(min=2.0 ** -126), torch.ones_like(top)).float().double()
    return torch.round(v / s), s


def _exact_router(st):
    case = st["case"]
    E, k = case["E"], case["k"]
    z, ids, dw = st["logits"].double(), st["ids"].long(), st["dw"]
    s = torch.where(z > 30, z, torch.log1p(torch.exp(z.clamp(max=30)))).sqrt()
    slope = torch.sigmoid(z) / (2 * s)
    off = st["offsets"].tolist()
    runs = [(b, e) for b, e in zip(off, off[1:]) if e > b]
    grad = torch.zeros_like(z)
    counts = torch.zeros(E, dtype=torch.int64, device=z.device)
    loss = torch.zeros((), dtype=torch.float64, device=z.device)
    for b, e in runs:
        n = e - b
        c = torch.bincount(ids[b:e].reshape(-1), minlength=E)
        counts += c
        f = c.double() * E / (k * n)
        total = s[b:e].sum(dim=1, keepdim=True)
        share = s[b:e] / total
        loss = loss + ALPHA / len(runs) * torch.dot(f, share.mean(dim=0))
        # d share_j / d s_i = (delta_ij - share_j) / total
        grad[b:e] = ALPHA / len(runs) / n * (f - (share @ f).unsqueeze(1)) / total
        if dw is not None:
            w = dw[b:e].double()
            chosen = s[b:e].gather(1, ids[b:e])
            norm = chosen.sum(dim=1, keepdim=True)
            grad[b:e].scatter_add_(1, ids[b:e], SCALE * (w * norm - (w * chosen).sum(dim=1, keepdim=True)) / norm ** 2)
    return loss, counts.to(torch.int32), grad * slope


def _exact_ortho(g):
    a, b, c = COEF
    out = []
    for m in g.double():
        flip = m.shape[0] > m.shape[1]
        y = m.t().contiguous() if flip else m
        y = y / (torch.linalg.vector_norm(y) + EPS)
        for _ in range(STEPS):
            q = torch.mm(y, y.t())
            y = a * y + torch.mm(q, b * y + c * torch.mm(q, y))
        out.append(y.t() if flip else y)
    return torch.stack(out)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        q, s = _exact_int8(st["x"])
        return q * s
    if op == "linear":
        q, s = _exact_int8(st["x"])
        return (q @ st["q"].double().t()) * s * st["scale"].double()
    if op == "router":
        return _exact_router(st)
    return _exact_ortho(st["g"])
