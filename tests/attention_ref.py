"""Attention and its gradients from the definitions in 64 bits, with the error that the kernels may make.

The kernels' roundings, relative to the value (bfloat16 has 8 significant bits, float32 24): scores are float32
sums of exact products, so a probability is off by a factor of at most 1 + eps, eps = 2^-23 (the sum's terms'
magnitudes * D + what the exponential takes, |s|, |lse| and a few roundings more); probabilities and ds are
rounded to bfloat16 (2^-8) as operands, outputs to bfloat16 (2^-8)."""
import math

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24


def spans(offsets, T, B):
    """[begin, end) of every sequence."""
    if offsets is None:
        n = T // B
        return [(b * n, b * n + n) for b in range(B)]
    o = offsets.tolist()
    return [(max(0, min(T, o[i])), max(0, min(T, o[i + 1]))) for i in range(len(o) - 1)]


def visible(lq, lk, causal, window, device):
    """[lq, lk] truth values."""
    at = torch.arange(lq, device=device)[:, None] + (lk - lq)
    key = torch.arange(lk, device=device)[None, :]
    if not causal:
        return torch.ones(lq, lk, dtype=torch.bool, device=device)
    see = key <= at
    return see & (key > at - window) if window else see


def heads(q, k, v, dout=None, offsets_q=None, offsets_k=None, batch=1, causal=True, window=0, scale=None):
    """Sequence by sequence, head by head: the rows' and keys' ranges, head, key head and the matrices in 64 bits."""
    Hq, D = q.shape[1], q.shape[2]
    G = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    batch = batch if offsets_q is None else offsets_q.numel() - 1
    for (a, b), (c, d) in zip(spans(offsets_q, q.shape[0], batch), spans(offsets_k, k.shape[0], batch)):
        if b <= a:
            b = a
        if d <= c:
            d = c
        see = visible(b - a, d - c, causal, window, q.device)
        for h in range(Hq):
            Q, K, V = q[a:b, h].double(), k[c:d, h // G].double(), v[c:d, h // G].double()
            s = torch.where(see, Q @ K.t() * scale, torch.full((), -math.inf, dtype=torch.float64, device=q.device))
            lse = torch.logsumexp(s, 1) if d > c else torch.full((b - a,), -math.inf, dtype=torch.float64, device=q.device)
            p = torch.exp(s - torch.where(lse > -math.inf, lse, torch.zeros_like(lse))[:, None])
            p = torch.where(see, p, torch.zeros_like(p))
            size = (Q.abs() @ K.abs().t() * scale).amax(1) if d > c else torch.zeros(b - a, dtype=torch.float64, device=q.device)
            deep = torch.where(lse > -math.inf, lse.abs(), torch.zeros_like(lse))
            eps = 2 * U32 * ((D + 8) * size + 4 * deep + 16)          # of each row's probabilities
            yield (a, b), (c, d), h, h // G, scale, Q, K, V, p, lse, eps, None if dout is None else dout[a:b, h].double()


def forward(q, k, v, **kw):
    """out and lse in 64 bits, what each may be off by before a rounding of the output, and the rows of sequences."""
    Tq, Hq, D = q.shape
    z = dict(dtype=torch.float64, device=q.device)
    out, lse, e_out, e_lse = torch.zeros(Tq, Hq, D, **z), torch.zeros(Hq, Tq, **z), torch.zeros(Tq, Hq, D, **z), torch.zeros(Hq, Tq, **z)
    rows = torch.zeros(Tq, dtype=torch.bool, device=q.device)
    for (a, b), (c, d), h, g, _, Q, K, V, p, z_, eps, _ in heads(q, k, v, **kw):
        rows[a:b] = True
        out[a:b, h], lse[h, a:b] = p @ V, z_
        n = d - c
        # each probability's rounding and error, the sum's and the products' float32 sums over n keys
        e_out[a:b, h] = (p @ V.abs()) * (U16 + 3 * eps[:, None] + 4 * U32 * (n + 64))
        e_lse[h, a:b] = eps + 2 * U32 * (n + 64) + 4 * U32 * torch.where(z_ > -math.inf, z_.abs(), torch.zeros_like(z_))
    return out, lse, e_out, e_lse, rows


def backward(q, k, v, dout, **kw):
    """dq, dk, dv in 64 bits and what each may be off by, the rounding of the outputs included."""
    z = dict(dtype=torch.float64, device=q.device)
    dq, dk, dv = (torch.zeros(t.shape, **z) for t in (q, k, v))
    eq, ek, ev = (torch.zeros(t.shape, **z) for t in (q, k, v))
    for (a, b), (c, d), h, g, scale, Q, K, V, p, _, eps, dO in heads(q, k, v, dout, **kw):
        o = p @ V
        delta = (dO * o).sum(1, keepdim=True)
        ds = p * (dO @ V.t() - delta)
        mag = (dO.abs() @ V.abs().t()) * 2 * U32 * (V.shape[1] + 8)
        e_delta = (dO.abs() * o.abs()).sum(1, keepdim=True) * (U16 + 2 * U32 * (V.shape[1] + 8))
        e_ds = ds.abs() * (U16 + 2 * eps[:, None]) + p * (mag + e_delta) * (1 + 2 * U16)
        n, m = d - c, b - a
        dq[a:b, h] += scale * ds @ K
        eq[a:b, h] += scale * (e_ds + 4 * U32 * (n + 64) * ds.abs()) @ K.abs()
        dk[c:d, g] += scale * ds.t() @ Q
        ek[c:d, g] += scale * (e_ds + 4 * U32 * (8 * m + 64) * ds.abs()).t() @ Q.abs()
        dv[c:d, g] += p.t() @ dO
        ev[c:d, g] += (p * (U16 + 2 * eps[:, None] + 4 * U32 * (8 * m + 64))).t() @ dO.abs()
    return [(x, e + U16 * (x.abs() + e)) for x, e in ((dq, eq), (dk, ek), (dv, ev))]
