"""Plain 64-bit forms (numpy) of the operators around the linear layer, each with the bound its
float32 computation keeps: U counts one float32 rounding, STEPS the roundings on the longest path
through a row's statistics and its element-wise formula (sums of up to 16384 columns are trees of
at most 8 V + 6 + 16 additions, the formulas at most 12 operations)."""
import numpy as np

U = 2.0 ** -24
STEPS = 64
BF16 = 2.0 ** -8       # half a step of bfloat16, relative
E4M3_HALF, E4M3_SUB = 2.0 ** -4, 2.0 ** -10
E5M2_HALF, E5M2_SUB = 2.0 ** -3, 2.0 ** -17


def stats(v, layer, eps):
    mean = v.mean(1) if layer else np.zeros(v.shape[0])
    return 1.0 / np.sqrt(((v - mean[:, None]) ** 2).mean(1) + eps), mean


def spread(gate, M):
    return None if gate is None else np.repeat(gate, M // gate.shape[0], axis=0)


def norm(v, w, b, layer, eps):
    """norm(v) * w + b, its statistics, and the error bound of a float32 evaluation."""
    rstd, mean = stats(v, layer, eps)
    r, m = rstd[:, None], mean[:, None]
    out = (v - m) * r * w + (0.0 if b is None else b)
    err = STEPS * U * ((np.abs(v) + np.abs(m)) * r * np.abs(w) + (0.0 if b is None else np.abs(b)))
    return out, rstd, mean, err


def after_block(o, w, b, gate, resid, alpha, layer, eps):
    """alpha * resid + gate * (norm(o) * w + b) before its rounding, the statistics and the bound."""
    if w is None:
        n, rstd, mean, err = o, None, None, np.zeros_like(o)
    else:
        n, rstd, mean, err = norm(o, w, b, layer, eps)
    if gate is not None:
        g = spread(gate, o.shape[0])
        n, err = g * n, np.abs(g) * err
    x = n + (0.0 if resid is None else alpha * resid)
    err = err + 4 * U * (np.abs(n) + (0.0 if resid is None else np.abs(alpha * resid)))
    return x, rstd, mean, err


def through_norm(dout, e_dout, v, w, rstd, mean, layer):
    """Gradient of norm(v) * w through dout (off by e_dout), its bound, the normalised v, and dout * w."""
    r = rstd[:, None]
    hat = (v - mean[:, None]) * r
    q, e_q = dout * w, e_dout * np.abs(w)
    ah = (np.abs(v) + np.abs(mean[:, None])) * r
    s1, a1, e1 = (q * hat).mean(1, keepdims=True), (np.abs(q) * ah).mean(1, keepdims=True), (e_q * ah).mean(1, keepdims=True)
    s0, a0, e0 = q.mean(1, keepdims=True), np.abs(q).mean(1, keepdims=True), e_q.mean(1, keepdims=True)
    if not layer:
        s0 = a0 = e0 = 0.0
    g = r * (q - s0 - hat * s1)
    err = STEPS * U * r * (np.abs(q) + a0 + ah * a1) + r * (e_q + e0 + ah * e1)
    return g, err, hat, ah


def backward(dh, dx, o, w_post, b_post, gate, alpha, x, post, w_pre, pre, layer):
    """All gradients as {name: (value, bound)}; post / pre: (rstd, mean) or None."""
    M, H = (dh if dh is not None else dx).shape
    out = {}
    d, e = np.zeros((M, H)), np.zeros((M, H))
    add = (M + STEPS) * U                     # a column sum: at most one addition per row and a tree
    if dh is not None:
        d, e, hat, ah = through_norm(dh, np.zeros((M, H)), x, w_pre, *pre, layer)
        out["dw_pre"] = ((dh * hat).sum(0), add * (np.abs(dh) * ah).sum(0))
        out["db_pre"] = (dh.sum(0), add * np.abs(dh).sum(0))
    if dx is not None:
        e = e + 2 * U * (np.abs(d) + np.abs(dx))
        d = d + dx
    out["d_resid"] = (alpha * d, np.abs(alpha) * (e + U * np.abs(d)))
    if o is None:
        return out
    g = spread(gate, M)
    dn, e_dn = (d, e) if g is None else (d * g, np.abs(g) * e + U * np.abs(d * g))
    if w_post is not None:
        d_o, e_o, hat, ah = through_norm(dn, e_dn, o, w_post, *post, layer)
        n = hat * w_post + (0.0 if b_post is None else b_post)
        an = ah * np.abs(w_post) + (0.0 if b_post is None else np.abs(b_post))
        out["dw_post"] = ((dn * hat).sum(0), add * (np.abs(dn) * ah).sum(0) + (e_dn * ah).sum(0))
        out["db_post"] = (dn.sum(0), add * np.abs(dn).sum(0) + e_dn.sum(0))
    else:
        d_o, e_o, n, an = dn, e_dn, o, np.abs(o)
    out["d_block"] = (d_o, e_o)
    if g is not None:
        G = gate.shape[0]
        fold = lambda v: v.reshape(G, M // G, H).sum(1)  # noqa: E731
        out["dgate"] = (fold(d * n), add * fold(np.abs(d) * an) + fold(e * an))
    return out


def plan(experts, E, align, cap):
    """The plan by counting: offsets, src, slot."""
    ids = experts.reshape(-1)
    slot, src, offsets, at = np.full(ids.size, -1, np.int32), np.full(cap, -1, np.int32), [0], 0
    for e in range(E):
        mine = np.nonzero(ids == e)[0]
        slot[mine] = at + np.arange(mine.size)
        src[at:at + mine.size] = mine
        at += -(-mine.size // align) * align
        offsets.append(at)
    return np.array(offsets, np.int32), src, slot.reshape(experts.shape)
