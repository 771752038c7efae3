"""Cases of the block operators around the FP8 linear layer, for measuring them.

Three families, as one feed-forward block of experts trained in FP8 uses them:
  norm    the norms before and after a block, fused with the block's gate and the residual scale
          (forward and backward), the next block's input leaving as bfloat16 and as FP8 codes;
  sort    tokens sorted by expert and back, with the router's weights applied, and its gradient;
  experts the experts' FP8 products over the sorted tokens: forward, input gradient, weight gradient.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, one rounding
at the end), or, with ``own`` set, by the framework's calls.  ``exact`` gives the same outputs from
the definitions in 64 bits.  FP8 codes are returned as the values they stand for.
"""
import math

import torch

own = False

ALIGN = 16            # every expert's rows start at a multiple of this (the FP8 products' 16-byte loads)
EPS = 1e-5
E4M3, E5M2 = 0, 1
FP8_MAX = {E4M3: 448.0, E5M2: 57344.0}
FP8_TYPE = {E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # serving: four sequences, one new token each, between two blocks of a 4096-wide model
        dict(name="norm-decode", op="norm_fwd", kind="rms", rows=4, width=4096, gates=0, h=True, fp8=True),
        # training: 8192 tokens of the same model, a learned gate per channel, FP8 input of the next layer
        dict(name="norm-train", op="norm_fwd", kind="rms", rows=8192, width=4096, gates=1, h=True, fp8=True),
        # an image or video transformer's odd width: LayerNorm, a gate per sample, bfloat16 only
        dict(name="norm-odd", op="norm_fwd", kind="layer", rows=2051, width=1001, gates=7, h=True, fp8=False),
        # backward at the width of the 12288-wide projection, LayerNorm, one gate for each of 4 sequences of 512
        dict(name="norm-wide-bwd", op="norm_bwd", kind="layer", rows=2048, width=12288, gates=4),
        # serving: 8 tokens to 4 of 64 experts, cast to FP8 on the way
        dict(name="sort-decode", op="sort", tokens=8, top=4, experts=64, width=4096, codes=False, transpose=False),
        # training: 8192 tokens whose norm already left FP8 codes; the transpose is the weight gradient's operand
        dict(name="sort-train", op="sort", tokens=8192, top=4, experts=64, width=4096, codes=True, transpose=True),
        # training: the experts' outputs back in token order, weighted
        dict(name="combine-train", op="combine", tokens=8192, top=4, experts=64, width=4096, weighted=True),
        # its backward: weighted FP8 gradients in expert order with their transpose, and the weights' gradient
        dict(name="combine-bwd", op="combine_bwd", tokens=5000, top=6, experts=40, width=2048),
        # serving: 16 tokens to 4 of 64 experts, up projection: bound by the weights that are touched
        dict(name="experts-decode", op="experts", grad="none", tokens=16, top=4, experts=64, n=2048, k=4096),
        # training: up projection of 8192 tokens to 4 of 64 experts
        dict(name="experts-train", op="experts", grad="none", tokens=8192, top=4, experts=64, n=2048, k=4096),
        # input gradient of a ragged layer: E5M2 gradients against E4M3 weights, contraction not a power of two
        dict(name="experts-dgrad", op="experts", grad="input", tokens=3001, top=2, experts=24, n=2560, k=1424),
        # weight gradient of the up projection
        dict(name="experts-wgrad", op="experts", grad="weight", tokens=8192, top=4, experts=64, n=2048, k=4096),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "sort", "combine", "combine_bwd", "experts", "experts"])
    if op in ("norm_fwd", "norm_bwd"):
        gates = rng.choice([0, 1, 1, rng.randint(2, 9)])
        width = _log(rng, 64, 16384, rng.choice([1, 8, 64]))
        rows = _log(rng, 1, min(8192, (1 << 25) // width))
        rows = max(1, rows // max(1, gates)) * max(1, gates)
        c = dict(op=op, kind=rng.choice(["rms", "layer"]), rows=rows, width=width, gates=gates)
        if op == "norm_fwd":
            c.update(h=True, fp8=rng.random() < 0.6)
        return c
    experts = _log(rng, 4, 128)
    top = rng.randint(1, min(8, experts))
    if op == "experts":
        grad = rng.choice(["none", "input", "weight"])
        return dict(op=op, grad=grad, tokens=_log(rng, 1, 8192), top=min(top, 4), experts=min(experts, 64),
                    n=_log(rng, 128, 2048, 16), k=_log(rng, 128, 4096, 16))
    width = _log(rng, 64, 4096, 16)
    tokens = _log(rng, 1, 32768 // top)
    c = dict(op=op, tokens=tokens, top=top, experts=experts, width=width)
    if op == "sort":
        c.update(codes=rng.random() < 0.5, transpose=rng.random() < 0.7)
    if op == "combine":
        c.update(weighted=rng.random() < 0.7)
    return c


def _capacity(c):
    """Rows of the sorted buffers: enough for any routing of the tokens."""
    n = c["tokens"] * c["top"]
    return (n + min(n, c["experts"]) * (ALIGN - 1)) // ALIGN * ALIGN


def work(c):
    op = c["op"]
    if op == "norm_fwd":
        e = c["rows"] * c["width"]
        par = c["width"] * 2 * ((2 if c["kind"] == "rms" else 4) + c["gates"])
        return {"bytes": e * (2 + 2 + 2 + 2 * c["h"] + c["fp8"]) + par + 8 * c["rows"], "flops": 12 * e}
    if op == "norm_bwd":
        e = c["rows"] * c["width"]
        par = c["width"] * 6 * ((2 if c["kind"] == "rms" else 4) + c["gates"])
        return {"bytes": e * (4 * 2 + 2 * 2) + par + 8 * c["rows"], "flops": 30 * e}
    n = c["tokens"] * c["top"]
    if op == "experts":
        n_k = c["n"] * c["k"]
        used = c["experts"] * (1.0 - (1.0 - 1.0 / c["experts"]) ** n)     # experts that evenly routed tokens reach
        if c["grad"] == "weight":
            by = n * (c["n"] + c["k"]) + 2 * c["experts"] * n_k
        else:
            by = n * (c["k"] + 2 * c["n"]) + used * n_k
        return {"bytes": by, "flops": 2 * n * n_k}
    h = c["width"]
    if op == "sort":
        return {"bytes": c["tokens"] * h * (1 if c["codes"] else 2) + n * h * (2 if c["transpose"] else 1) + 12 * n,
                "flops": n * h}
    if op == "combine":
        return {"bytes": (n + c["tokens"]) * h * 2 + (8 if c["weighted"] else 4) * n, "flops": 2 * n * h}
    return {"bytes": (c["tokens"] * 2 + n * 2 + n * 2) * h + 16 * n, "flops": 4 * n * h}


# ------------------------------------------------------------------------------------ inputs

def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)


def _normal(g, *shape, sd=1.0, mean=0.0):
    return (torch.randn(*shape, device="cuda", generator=g) * sd + mean).to(torch.bfloat16)


def _codes(g, fmt, *shape, sd):
    return (torch.randn(*shape, device="cuda", generator=g) * sd).to(FP8_TYPE[fmt]).view(torch.uint8)


def _routing(c, g):
    """Uneven routing: some experts popular, some unused, one choice in fifty dropped (-1)."""
    T, k, E = c["tokens"], c["top"], c["experts"]
    popular = torch.randn(E, device="cuda", generator=g) * 0.7
    scores = torch.randn(T, E, device="cuda", generator=g) + popular
    best, chosen = torch.topk(scores, k, dim=1)
    dropped = torch.rand(T, k, device="cuda", generator=g) < 0.02
    experts = torch.where(dropped, torch.full_like(chosen, -1), chosen).to(torch.int32)
    return experts.contiguous(), torch.softmax(best, dim=1).contiguous()


def _plan(experts, c):
    """Stable sort by expert, every expert's rows padded to a multiple of ALIGN: the first row of
    each expert, the choice that each sorted row holds (-1: none), the sorted row of each choice."""
    E, cap, n = c["experts"], _capacity(c), experts.numel()
    key = experts.reshape(-1).long()
    key = torch.where((key >= 0) & (key < E), key, torch.full_like(key, E))
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.long, device=key.device).index_add_(0, key, torch.ones_like(key))
    padded = (counts[:E] + ALIGN - 1) // ALIGN * ALIGN
    first = torch.zeros(E + 1, dtype=torch.long, device=key.device)
    first[1:] = torch.cumsum(padded, 0)
    ke = key[order]
    row = first[ke] + torch.arange(n, device=key.device) - (torch.cumsum(counts, 0) - counts)[ke]
    row = torch.where(ke < E, row, torch.full_like(row, -1))
    slot = torch.empty_like(row)
    slot[order] = row
    src = torch.full((cap + 1,), -1, dtype=torch.long, device=key.device)
    src[torch.where(row >= 0, row, torch.full_like(row, cap))] = order
    return first.to(torch.int32), src[:cap].to(torch.int32).contiguous(), slot.to(torch.int32).reshape(experts.shape)


def prepare(c, seed):
    g = _rng(seed)
    f32 = dict(device="cuda", dtype=torch.float32)
    u8 = dict(device="cuda", dtype=torch.uint8)
    bf = dict(device="cuda", dtype=torch.bfloat16)
    s = dict(c)
    if c["op"] in ("norm_fwd", "norm_bwd"):
        M, H, G, ln = c["rows"], c["width"], c["gates"], c["kind"] == "layer"
        s["block_out"] = _normal(g, M, H, sd=0.7, mean=0.1 if ln else 0.0)
        s["w_post"], s["w_pre"] = _normal(g, H, sd=0.1, mean=0.5), _normal(g, H, sd=0.1, mean=1.0)
        s["b_post"], s["b_pre"] = (_normal(g, H, sd=0.1), _normal(g, H, sd=0.1)) if ln else (None, None)
        s["gate"] = _normal(g, G, H, sd=0.5, mean=0.3) if G else None
        s["resid"] = _normal(g, M, H, sd=1.5)
        s["alpha"] = 0.875
        stats = (2, M) if ln else (M,)
        s["x"], s["post_stats"], s["pre_stats"] = torch.empty(M, H, **bf), torch.empty(stats, **f32), torch.empty(stats, **f32)
        if c["op"] == "norm_fwd":
            s["out"] = torch.empty(M, H, **bf) if c["h"] else None
            s["out8"] = torch.empty(M, H, **u8) if c["fp8"] else None
            s["scale"], s["amax"], s["sinv"] = torch.full((1,), 448.0 / 7.0, **f32), torch.zeros(1, **f32), torch.zeros(1, **f32)
        else:
            x, post, pre = _norm_forward(s)[:3]
            s["x"], s["post_stats"], s["pre_stats"] = x, post, pre
            s["dh"], s["dx"] = _normal(g, M, H, sd=0.02), _normal(g, M, H, sd=0.01)
            s["d_block"], s["d_resid"] = torch.empty(M, H, **bf), torch.empty(M, H, **bf)
            for name, used, shape in (("dw_post", True, (H,)), ("dw_pre", True, (H,)), ("db_post", ln, (H,)),
                                      ("db_pre", ln, (H,)), ("dgate", G > 0, (G, H))):
                s[name] = torch.empty(shape, **f32) if used else None
            if own:
                import fp8_delayed_scaling_amd as F
                s["workspace"] = torch.empty(F.fp8_norm_residual_workspace_bytes(M, H, max(1, G)), **u8)
        return s
    experts, weights = _routing(c, g)
    cap, T, k, E = _capacity(c), c["tokens"], c["top"], c["experts"]
    if c["op"] == "experts":
        offsets = _plan(experts, c)[0]
        rows = torch.arange(cap, device="cuda")
        live = rows < offsets[E]
        s["offsets"], s["longest"] = offsets, max(ALIGN, int((offsets[1:] - offsets[:-1]).max()))
        N, K = c["n"], c["k"]
        s["a_sinv"], s["b_sinv"] = torch.full((1,), 1 / 48.0, **f32), torch.full((1,), 1 / 3000.0, **f32)
        grad = c["grad"]
        fmt_a = E4M3 if grad == "none" else E5M2
        s["fmt_a"] = fmt_a
        sd_a = 48.0 if fmt_a == E4M3 else 900.0
        if grad == "weight":
            s["a"] = _codes(g, fmt_a, N, cap, sd=sd_a) * live
            s["b"] = _codes(g, E4M3, K, cap, sd=48.0) * live
            s["d"] = torch.zeros(E, N, K, **bf)
        else:
            s["a"] = _codes(g, fmt_a, cap, K, sd=sd_a) * live[:, None]
            s["b"] = _codes(g, E4M3, E, N, K, sd=60.0)
            s["d"] = torch.zeros(cap, N, **bf)
        return s
    H = c["width"]
    if c["op"] == "sort":
        s["choice"] = experts
        s["tokens_in"] = _codes(g, E4M3, T, H, sd=60.0) if c["codes"] else _normal(g, T, H)
        s["offsets"], s["src"] = torch.empty(E + 1, device="cuda", dtype=torch.int32), torch.empty(cap, device="cuda", dtype=torch.int32)
        s["slot"] = torch.empty(T, k, device="cuda", dtype=torch.int32)
        s["out8"], s["out8_t"] = torch.empty(cap, H, **u8), torch.empty(H, cap, **u8) if c["transpose"] else None
        s["scale"], s["amax"], s["sinv"] = torch.full((1,), 448.0 / 5.0, **f32), torch.zeros(1, **f32), torch.zeros(1, **f32)
        if own:
            import fp8_delayed_scaling_amd as F
            s["workspace"] = torch.empty(F.fp8_moe_workspace_bytes(T, k, E), **u8)
        return s
    s["offsets"], s["src"], s["slot"] = _plan(experts, c)
    s["weights"] = weights
    s["ys"] = _normal(g, cap, H) * (s["src"] >= 0)[:, None]
    if c["op"] == "combine":
        s["y"] = torch.empty(T, H, **bf)
        return s
    s["dy"] = _normal(g, T, H, sd=0.01)
    s["out8"], s["out8_t"], s["dweights"] = torch.empty(cap, H, **u8), torch.empty(H, cap, **u8), torch.empty(T, k, **f32)
    s["scale"], s["amax"], s["sinv"] = torch.full((1,), 57344.0 / 0.04, **f32), torch.zeros(1, **f32), torch.zeros(1, **f32)
    return s


# -------------------------------------------------------------------------------- plain forms

def _fp8(v, scale, fmt):
    return (v * scale).clamp(-FP8_MAX[fmt], FP8_MAX[fmt]).to(FP8_TYPE[fmt])


def _normalise(v, w, b, layer):
    """The norm of the rows of ``v``, its statistics (1 / standard deviation, then the mean)."""
    if layer:
        mean = v.mean(1, keepdim=True)
        rstd = torch.rsqrt((v - mean).square().mean(1, keepdim=True) + EPS)
        return (v - mean) * rstd * w.float() + b.float(), torch.cat([rstd, mean], 1).t().contiguous()
    rstd = torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
    return v * rstd * w.float(), rstd.reshape(-1)


def _gated(gate, v):
    """``gate`` [G, H] times the rows of ``v`` [M, H], M / G rows to each gate."""
    return v if gate is None else (gate.float()[:, None] * v.view(gate.shape[0], -1, v.shape[1])).view(v.shape)


def _norm_forward(s):
    layer = s["kind"] == "layer"
    n, post = _normalise(s["block_out"].float(), s["w_post"], s["b_post"], layer)
    x = (s["alpha"] * s["resid"].float() + _gated(s["gate"], n)).to(torch.bfloat16)
    h, pre = _normalise(x.float(), s["w_pre"], s["b_pre"], layer)
    return x, post, pre, h


def _norm_backward(dout, v, w, stats, layer):
    """Gradients of one norm: its input's, its weight's, and the normalised input."""
    if layer:
        rstd, mean = stats[0][:, None], stats[1][:, None]
        hat = (v - mean) * rstd
    else:
        rstd = stats[:, None]
        hat = v * rstd
    dhat = dout * w.float()
    back = dhat - hat * (dhat * hat).mean(1, keepdim=True)
    if layer:
        back = back - dhat.mean(1, keepdim=True)
    return back * rstd, (dout * hat).sum(0), hat


def _plain(s):
    op = s["op"]
    if op == "norm_fwd":
        x, post, pre, h = _norm_forward(s)
        r = {"x": x, "post_stats": post, "pre_stats": pre, "h": h.to(torch.bfloat16) if s["h"] else None}
        if s["fp8"]:
            r.update(h8=_fp8(h, s["scale"], E4M3), amax=h.abs().max().reshape(1), sinv=1.0 / s["scale"])
        return r
    if op == "norm_bwd":
        layer, gate = s["kind"] == "layer", s["gate"]
        dh = s["dh"].float()
        d, dw_pre, _ = _norm_backward(dh, s["x"].float(), s["w_pre"], s["pre_stats"], layer)
        d = d + s["dx"].float()
        dn = _gated(gate, d)
        d_block, dw_post, hat = _norm_backward(dn, s["block_out"].float(), s["w_post"], s["post_stats"], layer)
        n = hat * s["w_post"].float()
        n = n + s["b_post"].float() if layer else n
        return {"d_block": d_block.to(torch.bfloat16), "d_resid": (s["alpha"] * d).to(torch.bfloat16),
                "dw_post": dw_post, "dw_pre": dw_pre, "db_post": dn.sum(0) if layer else None,
                "db_pre": dh.sum(0) if layer else None,
                "dgate": (d * n).view(gate.shape[0], -1, gate.shape[1]).sum(1) if gate is not None else None}
    if op == "sort":
        offsets, src, slot = _plan(s["choice"], s)
        at, live = torch.div(src.clamp(min=0), s["top"], rounding_mode="floor").long(), (src >= 0)[:, None]
        r = {"offsets": offsets, "src": src, "slot": slot}
        if s["codes"]:
            rows = torch.where(live, s["tokens_in"][at], torch.zeros_like(s["tokens_in"][:1]))
            rows = rows.view(FP8_TYPE[E4M3])
        else:
            v = s["tokens_in"].float()[at] * live
            rows = _fp8(v, s["scale"], E4M3)
            r.update(amax=v.abs().max().reshape(1), sinv=1.0 / s["scale"])
        r["rows"] = rows
        if s["transpose"]:
            r["rows_t"] = rows.view(torch.uint8).t().contiguous().view(FP8_TYPE[E4M3])
        return r
    if op in ("combine", "combine_bwd"):
        live = (s["slot"] >= 0)[:, :, None]
        ys = torch.where(live, s["ys"].float()[s["slot"].clamp(min=0).long()], torch.zeros((), device="cuda"))
        if op == "combine":
            return {"y": ((ys * s["weights"][:, :, None]) if s["weighted"] else ys).sum(1).to(torch.bfloat16)}
        src = s["src"]
        at = torch.div(src.clamp(min=0), s["top"], rounding_mode="floor").long()
        w = s["weights"].reshape(-1)[src.clamp(min=0).long()] * (src >= 0)
        v = w[:, None] * s["dy"].float()[at]
        rows = _fp8(v, s["scale"], E5M2)
        return {"rows": rows, "rows_t": rows.view(torch.uint8).t().contiguous().view(FP8_TYPE[E5M2]),
                "amax": v.abs().max().reshape(1), "sinv": 1.0 / s["scale"],
                "dweights": (ys * s["dy"].float()[:, None]).sum(2)}
    first, L = s["offsets"].long(), s["longest"]
    at = first[:-1, None] + torch.arange(L, device="cuda")
    live = at < first[1:, None]
    cap = s["a"].shape[1] if s["grad"] == "weight" else s["a"].shape[0]
    at = torch.where(live, at, torch.full_like(at, cap))
    a, b = s["a"].view(FP8_TYPE[s["fmt_a"]]).float(), s["b"].view(FP8_TYPE[E4M3]).float()
    scale = s["a_sinv"] * s["b_sinv"]
    if s["grad"] == "weight":
        a = torch.cat([a.t(), a.new_zeros(1, a.shape[0])])[at]              # [E, L, N]
        b = torch.cat([b.t(), b.new_zeros(1, b.shape[0])])[at]              # [E, L, K]
        return {"d": (torch.bmm(a.transpose(1, 2).contiguous(), b) * scale).to(torch.bfloat16)}
    a = torch.cat([a, a.new_zeros(1, a.shape[1])])[at]                      # [E, L, K]
    d = torch.bmm(a, b.transpose(1, 2).contiguous()) * scale
    out = torch.zeros(cap + 1, d.shape[2], device="cuda", dtype=torch.bfloat16)
    out[at] = d.to(torch.bfloat16)
    return {"d": out[:cap]}


# --------------------------------------------------------------------- the framework's calls

def _own(s):
    import fp8_delayed_scaling_amd as F
    op = s["op"]
    if op == "norm_fwd":
        kind = F.NORM_LAYER if s["kind"] == "layer" else F.NORM_RMS
        F.fp8_norm_residual_fwd(s["block_out"], s["w_post"], s["b_post"], s["gate"], s["resid"], s["alpha"], s["x"],
                                s["post_stats"], s["w_pre"], s["b_pre"], s["pre_stats"], s["out"], s["out8"],
                                s["scale"] if s["fp8"] else None, F.E4M3, s["sinv"] if s["fp8"] else None,
                                s["amax"] if s["fp8"] else None, kind=kind, eps=EPS)
        r = {"x": s["x"], "post_stats": s["post_stats"], "pre_stats": s["pre_stats"], "h": s["out"]}
        if s["fp8"]:
            r.update(h8=s["out8"].view(FP8_TYPE[E4M3]), amax=s["amax"], sinv=s["sinv"])
        return r
    if op == "norm_bwd":
        kind = F.NORM_LAYER if s["kind"] == "layer" else F.NORM_RMS
        F.fp8_norm_residual_bwd(s["dh"], s["dx"], s["block_out"], s["w_post"], s["b_post"], s["gate"], s["alpha"],
                                s["x"], s["post_stats"], s["w_pre"], s["pre_stats"], s["d_block"], s["d_resid"],
                                s["dw_post"], s["db_post"], s["dgate"], s["dw_pre"], s["db_pre"], s["workspace"],
                                kind=kind)
        return {n: s[n] for n in ("d_block", "d_resid", "dw_post", "dw_pre", "db_post", "db_pre", "dgate")}
    if op == "sort":
        F.fp8_moe_plan(s["choice"], s["experts"], ALIGN, s["offsets"], s["src"], s["slot"], s["workspace"])
        r = {"offsets": s["offsets"], "src": s["src"], "slot": s["slot"]}
        if s["codes"]:
            F.fp8_moe_sort_codes(s["tokens_in"], s["src"], s["top"], s["out8"], s["out8_t"])
        else:
            F.fp8_moe_sort_cast(s["tokens_in"], s["src"], s["top"], None, s["scale"], F.E4M3, s["out8"], s["out8_t"],
                                s["sinv"], s["amax"])
            r.update(amax=s["amax"], sinv=s["sinv"])
        r["rows"] = s["out8"].view(FP8_TYPE[E4M3])
        if s["transpose"]:
            r["rows_t"] = s["out8_t"].view(FP8_TYPE[E4M3])
        return r
    if op == "combine":
        F.fp8_moe_combine(s["ys"], s["slot"], s["weights"] if s["weighted"] else None, s["y"])
        return {"y": s["y"]}
    if op == "combine_bwd":
        F.fp8_moe_sort_cast(s["dy"], s["src"], s["top"], s["weights"], s["scale"], F.E5M2, s["out8"], s["out8_t"],
                            s["sinv"], s["amax"])
        F.fp8_moe_weight_grad(s["dy"], s["ys"], s["slot"], s["dweights"])
        return {"rows": s["out8"].view(FP8_TYPE[E5M2]), "rows_t": s["out8_t"].view(FP8_TYPE[E5M2]), "amax": s["amax"],
                "sinv": s["sinv"], "dweights": s["dweights"]}
    call = F.fp8_grouped_wgrad if s["grad"] == "weight" else F.fp8_grouped_gemm
    call(s["a"], s["fmt_a"], s["a_sinv"], s["b"], F.E4M3, s["b_sinv"], s["offsets"], s["d"])
    return {"d": s["d"]}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- the definitions, 64 bits

def _round_fp8(v, fmt):
    """``v`` rounded to the nearest value of the format, ties to even, and held to its range."""
    mantissa, lowest = (3, -6) if fmt == E4M3 else (2, -14)
    exponent = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** (lowest - 8)))).clamp(min=lowest)
    step = torch.exp2(exponent - mantissa)
    return (torch.round(v / step) * step).clamp(-FP8_MAX[fmt], FP8_MAX[fmt])


def _bytes_value(codes, fmt):
    """FP8 codes as 64-bit values, from the format's bit fields."""
    mantissa, bias = (3, 7) if fmt == E4M3 else (2, 15)
    u = codes.to(torch.int64)
    field, frac = (u & 0x7F) >> mantissa, (u & ((1 << mantissa) - 1)).double() / (1 << mantissa)
    size = torch.where(field == 0, frac * 2.0 ** (1 - bias), (1.0 + frac) * torch.exp2((field - bias).double()))
    return torch.where(u >= 128, -size, size)


def _exact_stats(v, layer):
    mean = v.mean(1) if layer else torch.zeros(v.shape[0], dtype=v.dtype, device=v.device)
    rstd = 1.0 / torch.sqrt(((v - mean[:, None]) ** 2).mean(1) + EPS)
    return rstd, mean


def _exact_norm_fwd(c, s):
    layer = c["kind"] == "layer"
    o = s["block_out"].double()
    rp, mp = _exact_stats(o, layer)
    n = (o - mp[:, None]) * rp[:, None] * s["w_post"].double()
    if layer:
        n = n + s["b_post"].double()
    if s["gate"] is not None:
        n = n * s["gate"].double().repeat_interleave(c["rows"] // c["gates"], 0)
    x = s["alpha"] * s["resid"].double() + n
    kept = x.float().to(torch.bfloat16).double()          # the operator normalises the stored bfloat16 value
    rq, mq = _exact_stats(kept, layer)
    h = (kept - mq[:, None]) * rq[:, None] * s["w_pre"].double()
    if layer:
        h = h + s["b_pre"].double()
    stats = lambda r, m: torch.stack([r, m]) if layer else r  # noqa: E731
    out = {"x": x, "post_stats": stats(rp, mp), "pre_stats": stats(rq, mq), "h": h if c["h"] else None}
    if c["fp8"]:                                          # the codes' values before their rounding to 8 bits
        y = (h * s["scale"].double()).clamp(-448.0, 448.0)
        out.update(h8=y, amax=h.abs().max().reshape(1), sinv=1.0 / s["scale"].double())
    return out


def _exact_norm_bwd(c, s):
    layer, M, G = c["kind"] == "layer", c["rows"], c["gates"]

    def parts(v, stats):
        st = stats.double()
        rstd, mean = (st[0], st[1]) if layer else (st, torch.zeros_like(st))
        return (v.double() - mean[:, None]) * rstd[:, None], rstd[:, None]

    def through(dout, w, hat, rstd):
        q = dout * w.double()
        low = q.sum(1, keepdim=True) / q.shape[1] if layer else 0.0
        return rstd * (q - low - hat * ((q * hat).sum(1, keepdim=True) / q.shape[1]))

    dh = s["dh"].double()
    hat_x, r_x = parts(s["x"], s["pre_stats"])
    hat_o, r_o = parts(s["block_out"], s["post_stats"])
    d = s["dx"].double() + through(dh, s["w_pre"], hat_x, r_x)
    g = s["gate"].double().repeat_interleave(M // G, 0) if G else torch.ones((), dtype=torch.float64, device="cuda")
    n = hat_o * s["w_post"].double() + (s["b_post"].double() if layer else 0.0)
    return {"d_block": through(g * d, s["w_post"], hat_o, r_o), "d_resid": s["alpha"] * d,
            "dw_post": (g * d * hat_o).sum(0), "dw_pre": (dh * hat_x).sum(0),
            "db_post": (g * d).sum(0) if layer else None, "db_pre": dh.sum(0) if layer else None,
            "dgate": (d * n).reshape(G, M // G, -1).sum(1) if G else None}


def _exact_plan(experts, c):
    """The plan by counting on the host: one pass over the choices in order."""
    E, cap = c["experts"], _capacity(c)
    ids = experts.reshape(-1).tolist()
    rows = [[] for _ in range(E)]
    for i, e in enumerate(ids):
        if 0 <= e < E:
            rows[e].append(i)
    offsets, src, slot = [0], [-1] * cap, [-1] * len(ids)
    for e in range(E):
        for j, i in enumerate(rows[e]):
            src[offsets[-1] + j], slot[i] = i, offsets[-1] + j
        offsets.append(offsets[-1] + -(-len(rows[e]) // ALIGN) * ALIGN)
    as_int = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return as_int(offsets), as_int(src), as_int(slot).reshape(experts.shape)


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "norm_fwd":
        return _exact_norm_fwd(c, s)
    if op == "norm_bwd":
        return _exact_norm_bwd(c, s)
    if op == "experts":
        a, b = _bytes_value(s["a"], s["fmt_a"]), _bytes_value(s["b"], E4M3)
        scale = s["a_sinv"].double() * s["b_sinv"].double()
        cuts = s["offsets"].tolist()
        d = torch.zeros(s["d"].shape, dtype=torch.float64, device="cuda")
        for e in range(c["experts"]):
            lo, hi = cuts[e], cuts[e + 1]
            if c["grad"] == "weight":
                d[e] = a[:, lo:hi] @ b[:, lo:hi].t() * scale
            elif hi > lo:
                d[lo:hi] = a[lo:hi] @ b[e].t() * scale
        return {"d": d}
    if op == "sort":
        offsets, src, slot = _exact_plan(s["choice"], c)
        rows = torch.zeros(src.numel(), c["width"], dtype=torch.float64, device="cuda")
        used = src >= 0
        picked = s["tokens_in"][src[used].long() // c["top"]]
        out = {"offsets": offsets, "src": src, "slot": slot}
        if c["codes"]:
            rows[used] = _bytes_value(picked, E4M3)
        else:
            rows[used] = _round_fp8(picked.double() * s["scale"].double(), E4M3)
            out.update(amax=picked.double().abs().max().reshape(1) if picked.numel() else torch.zeros(1, dtype=torch.float64),
                       sinv=1.0 / s["scale"].double())
        out["rows"] = rows
        if c["transpose"]:
            out["rows_t"] = rows.t().contiguous()
        return out
    T, k = c["tokens"], c["top"]
    slot, w = s["slot"].long(), s["weights"].double()
    if op == "combine":
        y = torch.zeros(T, c["width"], dtype=torch.float64, device="cuda")
        for j in range(k):
            has = slot[:, j] >= 0
            y[has] += s["ys"][slot[has, j]].double() * (w[has, j, None] if c["weighted"] else 1.0)
        return {"y": y}
    dy = s["dy"].double()
    v = torch.zeros(s["src"].numel(), c["width"], dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        has = slot[:, j] >= 0
        v[slot[has, j]] = dy[has] * w[has, j, None]
        dw[has, j] = (dy[has] * s["ys"][slot[has, j]].double()).sum(1)
    rows = _round_fp8(v * s["scale"].double(), E5M2)
    return {"rows": rows, "rows_t": rows.t().contiguous(), "amax": v.abs().max().reshape(1),
            "sinv": 1.0 / s["scale"].double(), "dweights": dw}
