"""Attention's gradients do not depend on how the output was rounded: what <dout, out> is off by is made good from the sum of
the row's slopes."""
import math

import pytest
import torch

import attention_ref as ref
from test_gpu_attention import DEV, U16, close, inputs, offsets, run_backward

pytestmark = pytest.mark.gpu


def bounds(q, k, v, dout, out, **kw):
    """dq, dk, dv in 64 bits and what they may be off by, of `out` only through the operands' rounding: the slopes are rounded
    with the <dout, out> that was given, and the sum that makes it good is one of float32 slopes and rounded probabilities."""
    z = dict(dtype=torch.float64, device=q.device)
    grads, off = [torch.zeros(t.shape, **z) for t in (q, k, v)], [torch.zeros(t.shape, **z) for t in (q, k, v)]
    for (a, b), (c, d), h, g, scale, Q, K, V, p, _, eps, dO in ref.heads(q, k, v, dout, **kw):
        o = p @ V
        dp = dO @ V.t()
        ds = p * (dp - (dO * o).sum(1, keepdim=True))
        wrong = (dO * (out[a:b, h].double() - o)).sum(1, keepdim=True).abs()
        n, m = d - c, b - a
        fine = 2 * eps[:, None] + 4 * ref.U32 * (n + V.shape[1] + 64)
        mag = p * ((dO.abs() @ V.abs().t()) + (dO.abs() * o.abs()).sum(1, keepdim=True) + wrong)      # the slopes' terms
        e_sum = (mag * fine).sum(1, keepdim=True)
        e_q = (ds.abs() + p * wrong) * U16 + mag * fine + p * (wrong * U16 + e_sum)
        e_k = ds.abs() * U16 + (mag * fine + p * e_sum) * (1 + U16)
        grads[0][a:b, h] += scale * ds @ K
        off[0][a:b, h] += scale * (e_q + 4 * ref.U32 * (n + 64) * (ds.abs() + p * wrong)) @ K.abs()
        grads[1][c:d, g] += scale * ds.t() @ Q
        off[1][c:d, g] += scale * (e_k + 4 * ref.U32 * (8 * m + 64) * ds.abs()).t() @ Q.abs()
        grads[2][c:d, g] += p.t() @ dO
        off[2][c:d, g] += (p * (U16 + 2 * eps[:, None] + 4 * ref.U32 * (8 * m + 64))).t() @ dO.abs()
    return [(x, e + U16 * (x.abs() + e)) for x, e in zip(grads, off)]


# (sequences, query tokens, keys, heads, key/value heads, head size, causal, window): heads of up to 96 over any number of keys, above
# over up to 256 that a block's rows see
CASES = [(1, 400, 400, 4, 2, 64, True, 0), (2, 150, 700, 2, 1, 16, True, 0), (1, 900, 900, 2, 2, 40, False, 0), (1, 600, 600, 6, 2, 64, True, 100),
         (1, 500, 500, 4, 4, 96, True, 0), (2, 300, 300, 3, 1, 72, False, 0), (1, 1, 900, 4, 2, 80, True, 0),
         (1, 256, 256, 4, 2, 128, True, 0), (3, 200, 200, 8, 2, 128, False, 0), (2, 64, 64, 4, 4, 104, True, 0), (1, 700, 700, 4, 1, 128, True, 90),
         (1, 33, 190, 5, 1, 112, True, 0), (1, 400, 400, 2, 2, 128, True, 1), (4, 7, 65, 4, 2, 128, True, 5)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_gradients_from_a_coarse_output(case):
    """The output rounded to a few bits, as far off as 2^-4 of it."""
    B, lq, lk, Hq, Hkv, D, causal, window = case
    q, k, v, dout = inputs(sum(case), B * lq, B * lk, Hq, Hkv, D)
    kw = dict(batch=B, causal=causal, window=window)
    o, l, _, _, _ = ref.forward(q, k, v, **kw)
    for out in (o.bfloat16(), o.to(torch.float8_e4m3fn).bfloat16()):
        got = run_backward(dout, q, k, v, out, l.float(), **kw)
        for g, (want, bound) in zip(got, bounds(q, k, v, dout, out, **kw)):
            close(g, want, bound)


@pytest.mark.parametrize("D", [64, 128])
def test_packed(D):
    lens = [130, 1, 0, 256, 77]
    q, k, v, dout = inputs(D, sum(lens), sum(lens), 4, 2, D)
    kw = dict(offsets_q=offsets(lens), offsets_k=offsets(lens))
    o, l, _, _, _ = ref.forward(q, k, v, **kw)
    out = o.to(torch.float8_e4m3fn).bfloat16()
    for g, (want, bound) in zip(run_backward(dout, q, k, v, out, l.float(), **kw), bounds(q, k, v, dout, out, **kw)):
        close(g, want, bound)


@pytest.mark.parametrize("case", [(512, 64, 4), (700, 64, 256), (300, 128, 5), (64, 128, 0), (256, 96, 16), (512, 16, 0), (2048, 128, 0)], ids=str)
def test_error_of_all_gradients(case):
    """In the root of the mean square no more than the roundings that are meant: P and dS as operands and the results, to bfloat16.
    The same sums with these roundings and no others, in 64 bits, are as far off, give or take 4 % for the float32 parts and for
    other values' roundings being drawn."""
    L, D, window = case
    q, k, v, dout = inputs(L + D, L, L, 4, 2, D, sd=1.4)
    kw = dict(window=window)
    o, l, _, _, _ = ref.forward(q, k, v, **kw)
    got = run_backward(dout, q, k, v, o.bfloat16(), l.float(), **kw)
    r = lambda t: t.bfloat16().double()  # noqa: E731
    want, meant = ([torch.zeros(t.shape, dtype=torch.float64, device=DEV) for t in (q, k, v)] for _ in range(2))
    for _, _, h, g, scale, Q, K, V, p, _, _, dO in ref.heads(q, k, v, dout, **kw):
        ds = p * (dO @ V.t() - (dO * (p @ V)).sum(1, keepdim=True))
        given = p * (dO @ V.t() - (dO * r(p @ V)).sum(1, keepdim=True)) if L > 256 and D > 96 else ds      # there <dout, out> is the rounded output's
        for into, dsq, dsk, pv in ((want, ds, ds, p), (meant, r(given), r(ds), r(p))):
            into[0][:, h] = scale * dsq @ K
            into[1][:, g] += scale * dsk.t() @ Q
            into[2][:, g] += pv.t() @ dO
    size = sum(w.square().sum() for w in want)
    off = math.sqrt(sum((g.double() - w).square().sum() for g, w in zip(got, want)) / size)
    most = math.sqrt(sum((r(m) - w).square().sum() for m, w in zip(meant, want)) / size)
    assert off <= 1.04 * most, (off, most)
