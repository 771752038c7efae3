"""Cases of the router and of attention in a block of experts, for measuring them.

Two families, as a transformer block trained (and served) with FP8 linear layers uses them:
  attention   between the QKV layer and the projection: rows grouped over shared key/value heads, sequences
              packed one behind the other, causal or not, with a window or without; the output leaves as
              bfloat16 and as the projection's FP8 input; its backward recomputes the probabilities;
  route       in front of the sort by expert: the choice of experts from the router's logits, their weights,
              the experts' counts and the balance loss; its backward.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, one rounding at the
end), or, with ``own`` set, by the framework's calls.  ``exact`` gives the same outputs from the
definitions in 64 bits.  FP8 codes are returned as the values they stand for.
"""
import math

import torch

own = False

E4M3 = 0
FP8_MAX = 448.0
TAIL = 5              # rows behind the last sequence of a ragged batch: in no sequence, never written


# ------------------------------------------------------------------------------------- cases

def _attn(name, op, batch, q, k, heads, kv_heads, dim, causal=True, window=0, ragged=False, fp8=False):
    return dict(name=name, op=op, batch=batch, q=q, k=k, heads=heads, kv_heads=kv_heads, dim=dim, causal=causal,
                window=window, ragged=ragged, fp8=fp8)


def _route(name, op, tokens, experts, top, bf16=False, normalise=True, padded=False):
    return dict(name=name, op=op, tokens=tokens, experts=experts, top=top, bf16=bf16, normalise=normalise, padded=padded)


def listed():
    return [
        # serving: one new token for each of 16 sequences of up to 4096 tokens, a 4096-wide model's heads
        _attn("attn-decode", "attn_fwd", 16, 1, 4096, 32, 8, 128, ragged=True, fp8=True),
        # serving: 256 further tokens of each of two long prompts
        _attn("attn-chunk", "attn_fwd", 2, 256, 8192, 32, 8, 128, fp8=True),
        # training: 8192 tokens of the same model in sequences of 2048, the projection's input as FP8
        _attn("attn-train", "attn_fwd", 4, 0, 2048, 32, 8, 128, fp8=True),
        # an image or video transformer: every token sees its whole sample, odd head size, ragged samples
        _attn("attn-odd", "attn_fwd", 7, 0, 1001, 16, 16, 72, causal=False, ragged=True),
        # backward of the training case
        _attn("attn-train-bwd", "attn_bwd", 4, 0, 2048, 32, 8, 128),
        # backward over one long document
        _attn("attn-long-bwd", "attn_bwd", 1, 0, 8192, 32, 8, 128),
        # backward of a small model on packed ragged documents with a window
        _attn("attn-odd-bwd", "attn_bwd", 9, 0, 701, 12, 4, 64, window=256, ragged=True),
        # serving: 16 tokens to 4 of 64 experts
        _route("route-decode", "route_fwd", 16, 64, 4),
        # training: 8192 tokens to 4 of 64 experts, logits in float32
        _route("route-train", "route_fwd", 8192, 64, 4),
        # training: a larger batch to 8 of 256 experts, logits in bfloat16 as a layer leaves them
        _route("route-large", "route_fwd", 32768, 256, 8, bf16=True),
        # backward of the training case
        _route("route-train-bwd", "route_bwd", 8192, 64, 4),
        # backward of an odd layer: weights as the softmax leaves them, some rows padding
        _route("route-odd-bwd", "route_bwd", 5000, 40, 6, bf16=True, normalise=False, padded=True),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "route_fwd", "route_bwd"])
    if op in ("route_fwd", "route_bwd"):
        experts = _log(rng, 4, 512)
        return dict(op=op, tokens=_log(rng, 1, min(65536, (1 << 23) // experts)), experts=experts,
                    top=rng.randint(1, min(8, experts)), bf16=rng.random() < 0.5, normalise=rng.random() < 0.6,
                    padded=rng.random() < 0.4)
    kv_heads = rng.choice([1, 2, 4, 8, rng.randint(1, 12)])
    heads = kv_heads * rng.choice([1, 2, 4, 8, rng.randint(1, 7)])
    dim = rng.choice([64, 128, 128, 8 * rng.randint(2, 16)])
    c = dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, causal=rng.random() < 0.7, ragged=rng.random() < 0.6,
             window=0, fp8=op == "attn_fwd" and rng.random() < 0.5)
    # as much as one sequence of 8192 tokens with 32 heads of 128, at most
    most = int(math.sqrt(8192 * 8192 * 32 * 128 / (heads * dim)))
    if op == "attn_fwd" and rng.random() < 0.4:          # new tokens behind those that are there already
        c["batch"], c["q"] = _log(rng, 1, 32), rng.choice([1, 1, _log(rng, 2, 256)])
        c["k"] = max(c["q"], _log(rng, 16, min(8192, most)))
    else:
        c["k"], c["q"] = _log(rng, 1, min(8192, most)), 0
        c["batch"] = _log(rng, 1, max(1, min(32, 8192 // c["k"])))
    if c["causal"] and rng.random() < 0.3:
        c["window"] = _log(rng, 1, 1024)
    return c


def _lengths(c):
    """Each sequence's new tokens and keys: equal, or spread between a quarter of the longest and the longest."""
    B, L = c["batch"], c["k"]
    if not c["ragged"]:
        return [c["q"] or L] * B, [L] * B
    k = [max(1, L - (L * 3 // 4) * ((i * 7919 + 13) % 101) // 100) for i in range(B)]
    return [min(c["q"], n) if c["q"] else n for n in k], k


def _pairs(c):
    """Pairs of a row and a key that it may see, of one head."""
    n = 0
    for lq, lk in zip(*_lengths(c)):
        if not c["causal"]:
            n += lq * lk
            continue
        first = lk - lq + 1                              # keys that the first new token sees
        n += sum(min(m, c["window"]) for m in range(first, lk + 1)) if c["window"] else (first + lk) * lq // 2
    return n


def work(c):
    if c["op"] in ("attn_fwd", "attn_bwd"):
        lq, lk = _lengths(c)
        rows, keys = sum(lq) * c["heads"], sum(lk) * c["kv_heads"]
        if c["op"] == "attn_fwd":
            return {"bytes": 2 * c["dim"] * (2 * rows + 2 * keys) + rows * (4 + c["dim"] * c["fp8"]),
                    "flops": 4 * c["dim"] * c["heads"] * _pairs(c)}
        return {"bytes": 2 * c["dim"] * (4 * rows + 4 * keys) + 4 * rows, "flops": 10 * c["dim"] * c["heads"] * _pairs(c)}
    T, E, k = c["tokens"], c["experts"], c["top"]
    size = 2 if c["bf16"] else 4
    if c["op"] == "route_fwd":
        return {"bytes": T * (E * size + 8 * k + 4) + 8 * E, "flops": 6 * T * E}
    return {"bytes": T * (2 * E * size + 12 * k + 4) + 4 * E, "flops": 8 * T * E}


# ------------------------------------------------------------------------------------ inputs

def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 6271 + 29)


def _normal(g, *shape, sd=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * sd).to(torch.bfloat16)


def _offsets(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def prepare(c, seed):
    g = _rng(seed)
    f32, bf = dict(device="cuda", dtype=torch.float32), dict(device="cuda", dtype=torch.bfloat16)
    u8, i32 = dict(device="cuda", dtype=torch.uint8), dict(device="cuda", dtype=torch.int32)
    s = dict(c)
    if c["op"] in ("attn_fwd", "attn_bwd"):
        lq, lk = _lengths(c)
        Hq, Hkv, D = c["heads"], c["kv_heads"], c["dim"]
        tail = TAIL if c["ragged"] else 0
        Tq, Tk = sum(lq) + tail, sum(lk) + tail
        s["lengths"] = (lq, lk)
        s["offsets_q"], s["offsets_k"] = (_offsets(lq), _offsets(lk)) if c["ragged"] else (None, None)
        if c["q"]:                                       # new tokens' queries; keys and values of all tokens
            s["q"], kv = _normal(g, Tq, Hq, D, sd=1.4), _normal(g, Tk, 2 * Hkv, D, sd=1.4)
            s["k"], s["v"] = kv[:, :Hkv], kv[:, Hkv:]
        else:                                            # one QKV layer's output: [tokens, q heads, k heads, v heads]
            qkv = _normal(g, Tk, Hq + 2 * Hkv, D, sd=1.4)
            s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["out"], s["lse"] = torch.zeros(Tq, Hq, D, **bf), torch.zeros(Hq, Tq, **f32)
        if c["fp8"]:
            s["out8"] = torch.zeros(Tq, Hq * D, **u8)
            s["scale"], s["sinv"], s["amax"] = torch.full((1,), 448.0 / 6.0, **f32), torch.zeros(1, **f32), torch.zeros(1, **f32)
        if c["op"] == "attn_bwd":
            s["dout"] = _normal(g, Tq, Hq, D, sd=0.02)
            s["dqkv"] = torch.zeros(Tk, Hq + 2 * Hkv, D, **bf)      # the QKV layer's output gradient
            plain = _attention_forward(s)
            s["out"], s["lse"] = plain[0].to(torch.bfloat16), plain[1]
        if own:
            import fp8_delayed_scaling_amd as F
            size = F.fp8_attention_workspace_bytes if c["op"] == "attn_fwd" else F.fp8_attention_bwd_workspace_bytes
            s["workspace"] = torch.empty(size(Tq, Tk, c["batch"], Hq, Hkv, D), **u8)
        return s
    T, E, k = c["tokens"], c["experts"], c["top"]
    popular = torch.randn(E, device="cuda", generator=g) * 0.5
    logits = torch.randn(T, E, device="cuda", generator=g) * 1.5 + popular
    if c["padded"]:                                      # padding tokens choose nothing
        logits = torch.where(torch.rand(T, 1, device="cuda", generator=g) < 0.02, torch.full_like(logits, -math.inf), logits)
    s["logits"] = logits.to(torch.bfloat16) if c["bf16"] else logits
    if c["op"] == "route_fwd":
        s["chosen"], s["weights"], s["lse"] = torch.zeros(T, k, **i32), torch.zeros(T, k, **f32), torch.zeros(T, **f32)
        s["counts"], s["prob_sum"], s["loss"] = torch.zeros(E + 1, **i32), torch.zeros(E, **f32), torch.zeros(1, **f32)
        if own:
            import fp8_delayed_scaling_amd as F
            s["workspace"] = torch.empty(F.fp8_moe_route_workspace_bytes(T, E), **u8)
        return s
    r = _route_forward(s)
    s["chosen"], s["weights"], s["lse"], s["counts"] = r["chosen"], r["weights"], r["lse"], r["counts"]
    s["dweights"] = torch.randn(T, k, device="cuda", generator=g) * 0.1
    s["dloss"] = torch.full((1,), 0.01, **f32)
    s["dlogits"] = torch.empty_like(s["logits"])
    return s


# -------------------------------------------------------------------------------- plain forms

def _visible(c, lq, lk):
    """Which of ``lk`` keys each of the last ``lq`` tokens sees, as a truth value [lq, lk] (None: all of them)."""
    if not c["causal"]:
        return None
    ahead = torch.arange(lk, device="cuda")[None, :] - torch.arange(lk - lq, lk, device="cuda")[:, None]
    seen = ahead <= 0
    return seen & (ahead > -c["window"]) if c["window"] else seen


def _parts(s):
    """The sequences' rows: (first query row, first key row, new tokens, keys, sequences taken together)."""
    lq, lk = s["lengths"]
    if s["ragged"]:
        q0 = k0 = 0
        for a, b in zip(lq, lk):
            yield q0, k0, a, b, 1
            q0, k0 = q0 + a, k0 + b
        return
    B, a, b = len(lq), lq[0], lk[0]
    together = max(1, min(B, (1 << 29) // (a * b * s["heads"])))
    for first in range(0, B, together):
        yield first * a, first * b, a, b, min(together, B - first)


def _by_head(t, first, rows, n, kv_heads):
    """Rows of ``n`` sequences as float32 [n * kv_heads, rows * group, D], the group's heads one behind the other."""
    H, D = t.shape[1], t.shape[2]
    group = H // kv_heads
    x = t[first:first + n * rows].float().view(n, rows, kv_heads, group, D)
    return x.permute(0, 2, 3, 1, 4).reshape(n * kv_heads, group * rows, D)


def _to_rows(x, n, rows, kv_heads):
    """The way back from ``_by_head``: [n * rows, heads, D]."""
    group = x.shape[1] // rows
    return x.view(n, kv_heads, group, rows, -1).permute(0, 3, 1, 2, 4).reshape(n * rows, kv_heads * group, -1)


def _probabilities(s, q, k, lq, lk):
    """The probabilities [heads, rows, keys] and the logarithms of their sums."""
    x = torch.matmul(q, k.transpose(1, 2).contiguous()) * s["dim"] ** -0.5
    seen = _visible(s, lq, lk)
    if seen is not None:
        x = torch.where(seen.repeat(q.shape[1] // lq, 1), x, torch.full((), -math.inf, device="cuda"))
    top = x.max(2, keepdim=True).values
    p = torch.exp(x - top)
    total = p.sum(2, keepdim=True)
    return p / total, (top + torch.log(total)).squeeze(2)


def _heads_at_once(s, lq, lk):
    return max(1, (1 << 30) // (lq * lk * (s["heads"] // s["kv_heads"])))


def _attention_forward(s):
    Tq, Hq, D = s["q"].shape
    Hkv = s["kv_heads"]
    out, lse = torch.zeros(Tq, Hq, D, device="cuda"), torch.zeros(Hq, Tq, device="cuda")
    for q0, k0, lq, lk, n in _parts(s):
        q, k, v = _by_head(s["q"], q0, lq, n, Hkv), _by_head(s["k"], k0, lk, n, Hkv), _by_head(s["v"], k0, lk, n, Hkv)
        o, sums = [], []
        step = _heads_at_once(s, lq, lk)
        for h in range(0, q.shape[0], step):
            p, row = _probabilities(s, q[h:h + step], k[h:h + step], lq, lk)
            o.append(torch.matmul(p, v[h:h + step]))
            sums.append(row)
        o = o[0] if len(o) == 1 else torch.cat(o)
        sums = sums[0] if len(sums) == 1 else torch.cat(sums)
        out[q0:q0 + n * lq] = _to_rows(o, n, lq, Hkv)
        lse[:, q0:q0 + n * lq] = _to_rows(sums[:, :, None], n, lq, Hkv)[:, :, 0].t()
    return out, lse


def _attention_backward(s):
    Tq, Hq, D = s["q"].shape
    Tk, Hkv = s["k"].shape[:2]
    dq, dk, dv = torch.zeros(Tq, Hq, D, device="cuda"), torch.zeros(Tk, Hkv, D, device="cuda"), torch.zeros(Tk, Hkv, D, device="cuda")
    scale = D ** -0.5
    for q0, k0, lq, lk, n in _parts(s):
        q, k, v = _by_head(s["q"], q0, lq, n, Hkv), _by_head(s["k"], k0, lk, n, Hkv), _by_head(s["v"], k0, lk, n, Hkv)
        do = _by_head(s["dout"], q0, lq, n, Hkv)
        gq, gk, gv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        step = _heads_at_once(s, lq, lk)
        for h in range(0, q.shape[0], step):
            at = slice(h, h + step)
            p = _probabilities(s, q[at], k[at], lq, lk)[0]
            gv[at] = torch.matmul(p.transpose(1, 2).contiguous(), do[at])
            dp = torch.matmul(do[at], v[at].transpose(1, 2).contiguous())
            ds = p * (dp - (p * dp).sum(2, keepdim=True)) * scale
            gq[at] = torch.matmul(ds, k[at])
            gk[at] = torch.matmul(ds.transpose(1, 2).contiguous(), q[at])
        dq[q0:q0 + n * lq] = _to_rows(gq, n, lq, Hkv)
        dk[k0:k0 + n * lk] = _to_rows(gk, n, lk, Hkv)
        dv[k0:k0 + n * lk] = _to_rows(gv, n, lk, Hkv)
    return dq, dk, dv


def _route_forward(s):
    x, k, E = s["logits"].float(), s["top"], s["experts"]
    alive = (x > -math.inf).any(1)
    top = torch.where(alive, x.max(1).values, torch.zeros((), device="cuda"))[:, None]
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    p = e / torch.where(alive[:, None], total, torch.ones((), device="cuda"))
    best, order = torch.sort(x, dim=1, descending=True, stable=True)
    best, order = best[:, :k], order[:, :k]
    chosen = torch.where(best > -math.inf, order, torch.full_like(order, -1))
    weights = torch.gather(p, 1, order)
    if s["normalise"]:
        weights = weights / torch.where(alive, weights.sum(1), torch.ones((), device="cuda"))[:, None]
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    counts.index_add_(0, torch.where(chosen >= 0, chosen, torch.full_like(chosen, E)).reshape(-1), torch.ones_like(chosen).reshape(-1))
    counts[E] = alive.sum()
    prob_sum = p.double().sum(0).float()
    share = counts[:E].float() / counts[:E].sum().clamp(min=1)
    loss = E * (share * prob_sum).sum() / counts[E].clamp(min=1)
    return {"chosen": chosen.to(torch.int32), "weights": weights, "lse": (top + torch.log(total)).squeeze(1),
            "counts": counts.to(torch.int32), "prob_sum": prob_sum, "loss": loss.reshape(1)}


def _route_backward(s):
    x, E = s["logits"].float(), s["experts"]
    live = s["lse"] > -math.inf
    p = torch.exp(x - torch.where(live, s["lse"], torch.zeros((), device="cuda"))[:, None])
    counts = s["counts"].float()
    dp = (s["dloss"] * E * counts[:E] / (counts[:E].sum().clamp(min=1) * counts[E].clamp(min=1)))[None].repeat(x.shape[0], 1)
    chosen, w, dw = s["chosen"], s["weights"], s["dweights"]
    taken = chosen >= 0
    at = chosen.clamp(min=0).long()
    if s["normalise"]:
        d = p * (dp - (p * dp).sum(1, keepdim=True))
        d.scatter_add_(1, at, torch.where(taken, w * (dw - (w * dw).sum(1, keepdim=True)), torch.zeros((), device="cuda")))
    else:
        dp.scatter_add_(1, at, torch.where(taken, dw, torch.zeros((), device="cuda")))
        d = p * (dp - (p * dp).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def _plain(s):
    op = s["op"]
    if op == "attn_fwd":
        out, lse = _attention_forward(s)
        r = {"out": out.to(torch.bfloat16), "lse": lse}
        if s["fp8"]:
            codes = (out * s["scale"]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
            r.update(out8=codes.view(out.shape[0], -1), amax=out.abs().max().reshape(1), sinv=1.0 / s["scale"])
        return r
    if op == "attn_bwd":
        return {"dqkv": torch.cat(_attention_backward(s), 1).to(torch.bfloat16)}
    return _route_forward(s) if op == "route_fwd" else {"dlogits": _route_backward(s)}


# --------------------------------------------------------------------- the framework's calls

def _own(s):
    import fp8_delayed_scaling_amd as F
    op = s["op"]
    if op == "attn_fwd":
        F.fp8_attention_fwd(s["q"], s["k"], s["v"], s["out"], s["lse"], s["offsets_q"], s["offsets_k"], s["batch"],
                            s["causal"], s["window"], out8=s.get("out8"), scale=s.get("scale"), fmt=F.E4M3,
                            scale_inv_out=s.get("sinv"), amax_slot=s.get("amax"), workspace=s["workspace"])
        r = {"out": s["out"], "lse": s["lse"]}
        if s["fp8"]:
            r.update(out8=s["out8"].view(torch.float8_e4m3fn), amax=s["amax"], sinv=s["sinv"])
        return r
    if op == "attn_bwd":
        d, Hq, Hkv = s["dqkv"], s["heads"], s["kv_heads"]
        F.fp8_attention_bwd(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], d[:, :Hq], d[:, Hq:Hq + Hkv],
                            d[:, Hq + Hkv:], s["workspace"], s["offsets_q"], s["offsets_k"], s["batch"], s["causal"],
                            s["window"])
        return {"dqkv": d}
    if op == "route_fwd":
        F.fp8_moe_route(s["logits"], s["chosen"], s["weights"], s["lse"], s["counts"], s["prob_sum"], s["loss"],
                        s["workspace"], normalise=s["normalise"])
        return {n: s[n] for n in ("chosen", "weights", "lse", "counts", "prob_sum", "loss")}
    F.fp8_moe_route_bwd(s["logits"], s["chosen"], s["weights"], s["lse"], s["counts"], s["dweights"], s["dloss"],
                        s["dlogits"], normalise=s["normalise"])
    return {"dlogits": s["dlogits"]}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- the definitions, 64 bits

def _exact_attention(c, s):
    """One query head after the other, from the definitions; the gradients too where there is an output gradient."""
    Tq, Hq, D = s["q"].shape
    Tk, Hkv = s["k"].shape[0], s["k"].shape[1]
    f64 = dict(device="cuda", dtype=torch.float64)
    out, lse = torch.zeros(Tq, Hq, D, **f64), torch.zeros(Hq, Tq, **f64)
    grads = torch.zeros(Tk, Hq + 2 * Hkv, D, **f64) if c["op"] == "attn_bwd" else None
    q0 = k0 = 0
    for lq, lk in zip(*_lengths(c)):
        behind = torch.arange(lk - lq, lk, device="cuda").view(-1, 1) - torch.arange(lk, device="cuda").view(1, -1)
        hidden = torch.zeros(lq, lk, dtype=torch.bool, device="cuda")
        if c["causal"]:
            hidden = behind < 0
            if c["window"]:
                hidden = hidden | (behind >= c["window"])
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            q, k, v = s["q"][q0:q0 + lq, h].double(), s["k"][k0:k0 + lk, kv].double(), s["v"][k0:k0 + lk, kv].double()
            score = (q @ k.t() / math.sqrt(D)).masked_fill(hidden, -math.inf)
            z = torch.logsumexp(score, 1)
            prob = torch.exp(score - z[:, None])
            o = prob @ v
            out[q0:q0 + lq, h], lse[h, q0:q0 + lq] = o, z
            if grads is not None:
                do = s["dout"][q0:q0 + lq, h].double()
                slope = prob * (do @ v.t() - (do * o).sum(1)[:, None]) / math.sqrt(D)
                grads[q0:q0 + lq, h] = slope @ k
                grads[k0:k0 + lk, Hq + kv] += slope.t() @ q
                grads[k0:k0 + lk, Hq + Hkv + kv] += prob.t() @ do
        q0, k0 = q0 + lq, k0 + lk
    if grads is not None:
        return {"dqkv": grads}
    r = {"out": out, "lse": lse}
    if c["fp8"]:                                          # the codes' values before their rounding to 8 bits
        r.update(out8=(out * s["scale"].double()).clamp(-448.0, 448.0).reshape(Tq, Hq * D), amax=out.abs().max().reshape(1),
                 sinv=1.0 / s["scale"].double())
    return r


def _exact_choice(c, s):
    """The choices by a key that orders by logit, then by expert; their softmax."""
    x = s["logits"].double()
    T, E = x.shape
    some = (x > -math.inf).any(1)
    z = torch.logsumexp(x, 1)
    p = torch.zeros_like(x)
    p[some] = torch.exp(x[some] - z[some, None])
    left, chosen = x.clone(), torch.full((T, c["top"]), -1, dtype=torch.int64, device="cuda")
    number = torch.arange(E, device="cuda").expand(T, E)
    for j in range(c["top"]):
        best = left.max(1, keepdim=True).values
        at = torch.where((left == best) & (left > -math.inf), number, torch.full_like(number, E)).min(1).values
        has = at < E
        chosen[has, j] = at[has]
        left[has, at[has]] = -math.inf
    return x, p, z, chosen, some


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("attn_fwd", "attn_bwd"):
        return _exact_attention(c, s)
    x, p, z, chosen, some = _exact_choice(c, s)
    T, E = x.shape
    taken = chosen >= 0
    w = torch.zeros(T, c["top"], dtype=torch.float64, device="cuda")
    rows = torch.arange(T, device="cuda")[:, None].expand_as(chosen)
    w[taken] = p[rows[taken], chosen[taken]]
    total = w.sum(1, keepdim=True)
    if c["normalise"]:
        w = torch.where(total > 0, w / total, w)
    counts = torch.bincount(chosen[taken], minlength=E).double()
    live = max(1, int(some.sum()))
    share = counts / max(1.0, float(counts.sum()))
    if c["op"] == "route_fwd":
        return {"chosen": chosen.to(torch.int32), "weights": w, "lse": z,
                "counts": torch.cat([counts, some.sum().reshape(1).double()]).to(torch.int32), "prob_sum": p.sum(0),
                "loss": (E * (share * p.sum(0)).sum() / live).reshape(1)}
    # weights as a function of the logits, one choice at a time: d w_j / d x_e
    dw, dx = s["dweights"].double(), torch.zeros_like(x)
    for j in range(c["top"]):
        has = taken[:, j]
        g = dw[has, j] * w[has, j]
        if c["normalise"]:
            inside = torch.zeros_like(x[has])
            for i in range(c["top"]):
                ok = taken[has, i]
                inside[ok, chosen[has, i][ok]] = w[has, i][ok]
            dx[has] -= g[:, None] * inside
        else:
            dx[has] -= g[:, None] * p[has]
        dx[has, chosen[has, j]] += g
    slope = s["dloss"].double() * E * share / live
    return {"dlogits": dx + p * (slope[None] - (p @ slope)[:, None])}
