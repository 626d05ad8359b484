"""Plain 64-bit forms of the router's training operators, with the elementwise error the fp32 steps of the kernels may add
(torch, any device).

Errors, in half steps of fp32 (2^-24), each relative to its value: the exponent of h = exp(-|z| / 2) passes two roundings,
|z| together, and the hardware's exponential adds 2; e = h^2 has 2 |z| + 5; log1p(e) of at most that and 5 more, and so
does softplus; its root half of that and 2: a score has at most |z| + 8. Sums of a row add 8 and the reciprocal 2."""
import torch

U32 = 2.0 ** -24


def scores(z):
    soft = torch.where(z > 0, z, torch.zeros_like(z)) + torch.log1p(torch.exp(-z.abs()))
    s = soft.sqrt()
    slope = torch.where(z < -40, torch.exp(z / 2) / 2, torch.sigmoid(z) / (2 * s))
    return torch.where(z < -40, torch.exp(z / 2), s), slope


def router(z, ids, offsets=None, alpha=1.0, scale=1.0, dloss=1.0, dw=None, balance=True):
    """Logits z fp64 [T][E], ids [T][k], offsets: list of S + 1 borders -> dict of loss, counts [E], f (list of rows, empty
    sequences None), dz, and the bounds eloss, edz."""
    T, E = z.shape
    k = ids.shape[1]
    off = [0, T] if offsets is None else list(offsets)
    runs = [(b, e) for b, e in zip(off, off[1:]) if e > b]
    s, slope = scores(z)
    total = s.sum(1, keepdim=True)
    inv = torch.where(total > 0, 1 / total, torch.zeros_like(total))
    p = s * inv
    far = torch.where(z > -400, z, torch.zeros_like(z)).abs().amax(1, keepdim=True)  # below: scores under 2^-288
    units = far + 8                                                 # of every score of the row
    dev = z.device
    counts = torch.zeros(E, dtype=torch.int64, device=dev)
    loss = torch.zeros((), dtype=torch.float64, device=dev)
    eloss = torch.zeros((), dtype=torch.float64, device=dev)
    ds, eds = torch.zeros_like(z), torch.zeros_like(z)
    for b, e in runs:
        n, Q = e - b, len(runs)
        one = torch.zeros(E, dtype=torch.int64, device=dev)
        flat = ids[b:e].reshape(-1).long()
        flat = flat[(flat >= 0) & (flat < E)]
        one.index_add_(0, flat, torch.ones_like(flat))
        counts += one
        f = one.double() * E / (k * n)
        P = p[b:e].mean(0)
        loss = loss + alpha / Q * (f * P).sum()
        # shares: two scores and 10; their sum: at most 512 additions on a chain; 16 for the rest
        eloss = eloss + abs(alpha) / Q * (f * ((2 * units[b:e] + 10 + 528) * p[b:e]).mean(0)).sum() * U32
        if balance:
            g = dloss * alpha / (Q * n) * f
            dot = (g * p[b:e]).sum(1, keepdim=True)
            ds[b:e] += (g - dot) * inv[b:e]
            eds[b:e] += (g.abs() + dot.abs()) * inv[b:e] * (4 * units[b:e] + 40) * U32
        if dw is not None:
            i = ids[b:e].long()
            ok = (i >= 0) & (i < E)
            i = i.clamp(0, E - 1)
            w = torch.where(ok, dw[b:e].double(), 0.0)
            sj = torch.where(ok, s[b:e].gather(1, i), 0.0)
            N = sj.sum(1, keepdim=True)
            Ni = torch.where(N > 0, 1 / N, torch.zeros_like(N))
            dsj = torch.where(ok, scale * Ni * (w - (w * sj).sum(1, keepdim=True) * Ni), 0.0)
            edj = torch.where(ok, abs(scale) * Ni * (w.abs() + (w.abs() * sj).sum(1, keepdim=True) * Ni), 0.0)
            ds[b:e] = ds[b:e].scatter_add(1, i, dsj)
            eds[b:e] = eds[b:e].scatter_add(1, i, edj * (4 * units[b:e] + 40) * U32)
    # the slope: sigmoid 2 |z| + 10, the root's reciprocal half of softplus's and 2
    edz = (eds + ds.abs() * (4 * units + 20) * U32) * slope
    return {"loss": loss, "counts": counts.to(torch.int32), "dz": ds * slope, "eloss": eloss, "edz": edz, "s": s, "p": p}
