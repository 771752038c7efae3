"""Attention against the definitions in 64 bits: head sizes and layouts, lengths from none to many, masks that leave
rows empty, windows, packed sequences, strides, the split over the keys, FP8 output, gradients."""
import math

import pytest
import torch

import attention_ref as ref
import fp8_delayed_scaling_amd as F

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U16 = ref.U16
E4M3_HALF_STEP, E4M3_LOWEST = 2.0 ** -4, 2.0 ** -10      # relative; half of the smallest subnormal


def inputs(seed, Tq, Tk, Hq, Hkv, D, sd=1.2):
    g = torch.Generator(device=DEV).manual_seed(seed)
    make = lambda *s: (torch.randn(*s, device=DEV, generator=g) * sd).bfloat16()  # noqa: E731
    return make(Tq, Hq, D), make(Tk, Hkv, D), make(Tk, Hkv, D), make(Tq, Hq, D)


def offsets(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def workspace(fn, q, k, batch):
    n = fn(q.shape[0], k.shape[0], batch, q.shape[1], k.shape[1], q.shape[2])
    return torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device=DEV)       # NaNs: nothing in it may count


def run_forward(q, k, v, offsets_q=None, offsets_k=None, batch=1, causal=True, window=0, scale=None, fp8=False, fill=7.0):
    B = batch if offsets_q is None else offsets_q.numel() - 1
    out = torch.full(q.shape, fill, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((q.shape[1], q.shape[0]), fill, dtype=torch.float32, device=DEV)
    kw = {}
    if fp8:
        kw = dict(out8=torch.full((q.shape[0], q.shape[1] * q.shape[2]), 0x11, dtype=torch.uint8, device=DEV),
                  scale=torch.full((1,), 60.0, device=DEV), scale_inv_out=torch.zeros(1, device=DEV), amax_slot=torch.zeros(1, device=DEV))
    F.fp8_attention_fwd(q, k, v, out, lse, offsets_q, offsets_k, batch, causal, window, scale, **kw,
                        workspace=workspace(F.fp8_attention_workspace_bytes, q, k, B))
    return out, lse, kw


def close(got, want, bound):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} past their bound, first at {bad.nonzero()[0].tolist()}: got "
                           f"{got[bad][0].item()}, want {want[bad][0].item()}, off by {off[bad][0].item()}, bound {bound[bad][0].item()}")


def check_forward(q, k, v, fp8=False, **kw):
    out, lse, f = run_forward(q, k, v, fp8=fp8, **kw)
    w_out, w_lse, e_out, e_lse, rows = ref.forward(q, k, v, **kw)
    assert bool((out[~rows] == 7.0).all()) and bool((lse[:, ~rows] == 7.0).all())      # rows of no sequence
    empty = w_lse == -math.inf
    assert bool((lse[empty] == -math.inf).all())
    live = rows[None].expand_as(empty) & ~empty
    close(lse[live], w_lse[live], e_lse[live])
    close(out[rows], w_out[rows], (e_out + U16 * (w_out.abs() + e_out))[rows])
    if fp8:
        s = 60.0
        codes = f["out8"].view(q.shape)
        assert bool((codes[~rows] == 0x11).all())
        y = (w_out * s).clamp(-448, 448)
        close(codes.view(torch.float8_e4m3fn).float()[rows], y[rows],
              (e_out * s * (1 + E4M3_HALF_STEP) + E4M3_HALF_STEP * y.abs() + E4M3_LOWEST)[rows])
        amax = w_out[rows].abs().max() if bool(rows.any()) else torch.zeros((), device=DEV).double()
        # outputs within 1/64 of the largest are computed again with unrounded probabilities, one a wave: what their
        # rounding is off by is left only where two rows of one wave are nearer than it
        assert abs(f["amax_slot"].item() - amax.item()) <= float(e_out.max())
        assert f["scale_inv_out"].item() == (torch.ones(1) / torch.tensor([s])).item()
    return out, lse


def run_backward(dout, q, k, v, out, lse, offsets_q=None, offsets_k=None, batch=1, causal=True, window=0, scale=None):
    B = batch if offsets_q is None else offsets_q.numel() - 1
    dq, dk, dv = (torch.full(t.shape, 7.0, dtype=torch.bfloat16, device=DEV) for t in (q, k, v))
    F.fp8_attention_bwd(dout, q, k, v, out, lse, dq, dk, dv, workspace(F.fp8_attention_bwd_workspace_bytes, q, k, B), offsets_q,
                        offsets_k, batch, causal, window, scale)
    return dq, dk, dv


def check_backward(dout, q, k, v, **kw):
    o, l, _, _, rows = ref.forward(q, k, v, **kw)
    got = run_backward(dout, q, k, v, o.bfloat16(), l.float(), **kw)
    keys = torch.zeros(k.shape[0], dtype=torch.bool, device=DEV)
    B = kw.get("batch", 1) if kw.get("offsets_k") is None else kw["offsets_k"].numel() - 1
    for a, b in ref.spans(kw.get("offsets_k"), k.shape[0], B):
        keys[a:b] = True
    for g, (want, bound), there in zip(got, ref.backward(q, k, v, dout, **kw), (rows, keys, keys)):
        assert bool((g[~there] == 7.0).all())
        close(g[there], want[there], bound[there])


# (sequences, query tokens, keys, heads, key/value heads, head size, causal, window)
EQUAL = [
    (1, 1, 1, 1, 1, 8, True, 0), (1, 1, 1, 1, 1, 128, False, 0), (3, 1, 77, 4, 1, 64, True, 0), (2, 1, 300, 8, 2, 128, True, 0),
    (1, 31, 31, 2, 2, 64, True, 0), (1, 32, 32, 2, 2, 64, True, 0), (1, 33, 33, 2, 2, 64, True, 0), (2, 64, 64, 4, 4, 128, True, 0),
    (1, 127, 127, 2, 1, 128, True, 0), (1, 128, 128, 1, 1, 96, True, 0), (1, 129, 129, 3, 1, 128, True, 0), (2, 200, 200, 6, 2, 72, False, 0),
    (1, 257, 257, 5, 1, 40, True, 0), (1, 100, 163, 4, 2, 104, True, 0), (1, 100, 163, 4, 2, 104, False, 0), (1, 9, 500, 7, 1, 128, True, 0),
    (2, 163, 100, 4, 2, 64, True, 0), (1, 90, 10, 8, 1, 128, True, 0), (1, 5, 2, 4, 4, 128, True, 0), (2, 12, 0, 2, 1, 64, True, 0),
    (1, 200, 200, 4, 4, 128, True, 1), (1, 200, 200, 4, 2, 64, True, 7), (2, 333, 333, 3, 3, 80, True, 100), (1, 300, 300, 8, 1, 128, True, 64),
    (1, 150, 400, 2, 2, 128, True, 33), (1, 400, 150, 2, 1, 128, True, 33), (1, 64, 64, 2, 2, 128, True, 64), (1, 512, 512, 2, 2, 128, True, 2000),
    (1, 513, 700, 16, 2, 128, True, 0), (5, 3, 129, 16, 1, 128, True, 0), (4, 1, 1025, 32, 32, 64, True, 0), (2, 8, 65, 8, 2, 88, True, 20),
]


@pytest.mark.parametrize("case", EQUAL, ids=str)
def test_forward_of_equal_sequences(case):
    B, lq, lk, Hq, Hkv, D, causal, window = case
    q, k, v, _ = inputs(sum(case), B * lq, B * lk, Hq, Hkv, D)
    check_forward(q, k, v, batch=B, causal=causal, window=window, fp8=D % 16 == 0)


@pytest.mark.parametrize("case", EQUAL, ids=str)
def test_backward_of_equal_sequences(case):
    B, lq, lk, Hq, Hkv, D, causal, window = case
    q, k, v, dout = inputs(sum(case) + 1, B * lq, B * lk, Hq, Hkv, D)
    check_backward(dout, q, k, v, batch=B, causal=causal, window=window)


# (query lengths, key lengths, heads, key/value heads, head size, causal, window)
PACKED = [
    ([5, 0, 17, 1, 130], None, 4, 2, 64, True, 0), ([1, 1, 1], [7, 300, 64], 8, 2, 128, True, 0), ([3], [3], 2, 1, 128, True, 0),
    ([40, 200, 0, 0, 77], None, 3, 1, 72, False, 0), ([300, 33, 129], None, 6, 3, 128, True, 50), ([0, 0], [0, 0], 2, 2, 64, True, 0),
    ([10, 20, 30], [0, 40, 5], 4, 1, 96, True, 0), ([0, 64, 2], [50, 0, 90], 4, 4, 128, False, 0),
    ([1] * 70, [i % 37 for i in range(70)], 4, 2, 64, True, 0), ([2, 1] * 66, [40 + i % 5 for i in range(132)], 2, 1, 128, True, 9),
    ([257] * 3, [512, 257, 300], 8, 8, 128, True, 0),
]


@pytest.mark.parametrize("case", PACKED, ids=lambda c: str(c)[:60])
@pytest.mark.parametrize("direction", ["forward", "backward"])
def test_packed_sequences(case, direction):
    lq, lk, Hq, Hkv, D, causal, window = case
    lk = lq if lk is None else lk
    tail = 9
    q, k, v, dout = inputs(len(lq) + sum(lk), sum(lq) + tail, sum(lk) + tail, Hq, Hkv, D)
    for t in (q, k, v, dout):
        t[-tail:] = math.nan                         # rows behind the last sequence: never read
    kw = dict(offsets_q=offsets(lq), offsets_k=offsets(lk), causal=causal, window=window)
    if direction == "forward":
        check_forward(q, k, v, fp8=True, **kw)
    else:
        check_backward(dout, q, k, v, **kw)


def test_padding_between_sequences():
    """Sequences that do not start where the one before ends: the rows between are neither read nor written."""
    q, k, v, dout = inputs(3, 200, 260, 4, 2, 128)
    # three sequences of which the middle one stands for padding: its rows hold NaNs and reach nobody
    oq, ok = torch.tensor([0, 60, 90, 200], dtype=torch.int32, device=DEV), torch.tensor([0, 100, 133, 260], dtype=torch.int32, device=DEV)
    o, l, _ = run_forward(q, k, v, oq, ok)
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    q2[60:90], k2[100:133], v2[100:133] = math.nan, math.inf, math.nan
    o2, l2, _ = run_forward(q2, k2, v2, oq, ok)
    for rows in (slice(0, 60), slice(90, 200)):
        assert torch.equal(o[rows], o2[rows]) and torch.equal(l[:, rows], l2[:, rows])
    d = run_backward(dout, q, k, v, o, l, oq, ok)
    dout2 = dout.clone()
    dout2[60:90] = math.nan
    d2 = run_backward(dout2, q2, k2, v2, o2, l2, oq, ok)
    assert torch.equal(d[0][:60], d2[0][:60]) and torch.equal(d[0][90:], d2[0][90:])
    for a, b in zip(d[1:], d2[1:]):
        assert torch.equal(a[:100], b[:100]) and torch.equal(a[133:], b[133:])


@pytest.mark.parametrize("lq,lk,Hq,Hkv,D", [(1, 5000, 8, 2, 128), (1, 3001, 4, 4, 64), (7, 4099, 4, 1, 96), (256, 6000, 4, 1, 128), (130, 2500, 2, 2, 64)])
@pytest.mark.parametrize("window", [0, 1500])
def test_split_over_the_keys(lq, lk, Hq, Hkv, D, window):
    q, k, v, _ = inputs(lq + lk, lq, lk, Hq, Hkv, D)
    assert F.fp8_attention_workspace_bytes(lq, lk, 1, Hq, Hkv, D) > 0
    check_forward(q, k, v, causal=True, window=window, fp8=True)


def test_split_with_ragged_lengths():
    lk = [4000, 1, 0, 700, 3999, 64]
    q, k, v, _ = inputs(5, 6 + 3, sum(lk) + 3, 8, 2, 128)
    assert F.fp8_attention_workspace_bytes(9, sum(lk) + 3, 6, 8, 2, 128) > 0
    check_forward(q, k, v, offsets_q=offsets([1] * 6), offsets_k=offsets(lk), fp8=True)


@pytest.mark.parametrize("layout", ["packed", "head_major", "shared", "padded"])
def test_strides(layout):
    B, L, Hq, Hkv, D = 2, 150, 6, 2, 64
    T = B * L
    g = torch.Generator(device=DEV).manual_seed(9)
    make = lambda *s: torch.randn(*s, device=DEV, generator=g).bfloat16()  # noqa: E731
    empty = lambda *s: torch.full(s, 7.0, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    if layout == "packed":                               # slices of one QKV output and of its gradient
        x, d = make(T, (Hq + 2 * Hkv) * D), empty(T, (Hq + 2 * Hkv) * D)
        cut = lambda t: (t[:, :Hq * D].view(T, Hq, D), t[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D), t[:, (Hq + Hkv) * D:].view(T, Hkv, D))  # noqa: E731
        (q, k, v), (dq, dk, dv), dout, out = cut(x), cut(d), make(T, Hq, D), empty(T, Hq, D)
    elif layout == "head_major":
        new = lambda f, H: f(H, T, D).transpose(0, 1)  # noqa: E731
        q, k, v, dout, out = new(make, Hq), new(make, Hkv), new(make, Hkv), new(make, Hq), new(empty, Hq)
        dq, dk, dv = new(empty, Hq), new(empty, Hkv), new(empty, Hkv)
    elif layout == "shared":                             # one head broadcast to all key/value heads, and to the output gradient's
        q, k, v = make(T, Hq, D), make(T, 1, D).expand(T, Hkv, D), make(T, 1, D).expand(T, Hkv, D)
        dout, out, dq, dk, dv = make(T, 1, D).expand(T, Hq, D), empty(T, Hq, D), empty(T, Hq, D), empty(T, Hkv, D), empty(T, Hkv, D)
    else:
        new = lambda f, H: f(T, H + 1, D + 24)[:, :H, :D]  # noqa: E731
        q, k, v, dout, out = new(make, Hq), new(make, Hkv), new(make, Hkv), new(make, Hq), new(empty, Hq)
        dq, dk, dv = new(empty, Hq), new(empty, Hkv), new(empty, Hkv)
    lse = torch.empty(Hq, T, device=DEV)
    F.fp8_attention_fwd(q, k, v, out, lse, batch=B)
    w_out, w_lse, e_out, e_lse, _ = ref.forward(q, k, v, batch=B)
    close(out, w_out, e_out + U16 * (w_out.abs() + e_out))
    close(lse, w_lse, e_lse)
    F.fp8_attention_bwd(dout, q, k, v, w_out.bfloat16(), w_lse.float(), dq, dk, dv, workspace(F.fp8_attention_bwd_workspace_bytes, q, k, B), batch=B)
    for got, (want, bound) in zip((dq, dk, dv), ref.backward(q, k, v, dout, batch=B)):
        close(got, want, bound)


def test_large_scores():
    """Scores of hundreds, of either sign, whose row maxima grow along the keys: no overflow, no lost sums."""
    q, k, v, dout = inputs(11, 300, 300, 4, 2, 128, sd=1.0)
    k *= torch.linspace(0.1, 20, 300, device=DEV)[:, None, None].bfloat16()
    check_forward(q, k, v)
    check_backward(dout, q, k, v)
    k = -q[:, ::2].abs() * 8                              # every score far below zero
    q = q.abs()
    check_forward(q, k, v)
    check_backward(dout, q, k, v)
    check_backward(dout, q, k, v, causal=False)


def test_lowest_and_scaled():
    """A given softmax scale; keys that a row sees with the lowest scores there are."""
    q, k, v, dout = inputs(12, 130, 130, 2, 2, 64)
    check_forward(q, k, v, scale=0.5)
    check_backward(dout, q, k, v, scale=0.5)
    q[:, :, 0], k[:, :, 0] = 1.0, 0.0
    k[::3, :, 0] = -1e30                                 # masked by value: exp gives zero
    o, l, _ = run_forward(q, k, v, causal=False)
    some = torch.ones(130, dtype=torch.bool, device=DEV)
    some[::3] = False
    w, _, e, _, _ = ref.forward(q, k[some], v[some], causal=False)
    close(o, w, e + U16 * (w.abs() + e))
    d = run_backward(dout, q, k, v, o, l, causal=False)
    assert bool((d[1][::3] == 0).all()) and bool((d[2][::3] == 0).all()) and all(bool(x.isfinite().all()) for x in d)


def test_only_codes_and_no_lse():
    q, k, v, _ = inputs(13, 100, 100, 4, 2, 128)
    want = torch.empty(100, 4 * 128, dtype=torch.uint8, device=DEV)
    s, amax = torch.full((1,), 60.0, device=DEV), torch.zeros(1, device=DEV)
    ws = workspace(F.fp8_attention_workspace_bytes, q, k, 1)
    F.fp8_attention_fwd(q, k, v, torch.empty_like(q), None, out8=want, scale=s, amax_slot=amax, workspace=ws)
    got, amax2 = torch.empty_like(want), torch.full((1,), 99.0, device=DEV)
    F.fp8_attention_fwd(q, k, v, None, None, out8=got, scale=s, amax_slot=amax2, workspace=ws)
    assert torch.equal(got, want) and amax2.item() == 99.0        # an amax that is larger stays
    e5 = torch.empty_like(want)
    F.fp8_attention_fwd(q, k, v, None, None, out8=e5, scale=s, fmt=F.E5M2)
    w, _, e, _, _ = ref.forward(q, k, v)
    close(e5.view(torch.float8_e5m2).float().view(q.shape), w * 60, e * 60 * 1.125 + 2.0 ** -3 * (w * 60).abs() + 2.0 ** -17)


@pytest.mark.parametrize("B,lq,lk,Hq,Hkv,D,causal,ragged", [
    (1, 500, 500, 8, 2, 128, True, False), (4, 300, 300, 4, 4, 64, False, False), (3, 1, 3000, 8, 1, 128, True, False), (1, 200, 5000, 4, 2, 96, True, True),
    (1, 64, 40, 4, 2, 128, True, False), (5, 129, 400, 6, 3, 72, False, True), (2, 700, 700, 16, 2, 128, True, True)])
def test_amax_is_that_of_unrounded_probabilities(B, lq, lk, Hq, Hkv, D, causal, ragged):
    """To the float32 roundings of the largest output: its scores, exponentials and sums."""
    for seed in range(4):
        q, k, v, _ = inputs(30 + seed, B * lq, B * lk, Hq, Hkv, D)
        kw = dict(causal=causal, batch=B)
        if ragged:
            kw.update(offsets_q=offsets([lq] * B), offsets_k=offsets([lk] * B))
        f = run_forward(q, k, v, fp8=True, **kw)[2]
        out = ref.forward(q, k, v, **kw)[0]
        at = out.abs().flatten().argmax().item()
        token, head = at // (Hq * D), at // D % Hq
        # what the float32 parts of this output's error allow (its terms' magnitudes times each one's relative error)
        hidden = next(x for x in ref.heads(q, k, v, **kw) if x[0][0] <= token < x[0][1] and x[2] == head)
        p, V, eps = hidden[8][token - hidden[0][0]], hidden[7], hidden[10][token - hidden[0][0]]
        bound = (p @ V.abs())[at % D] * (3 * eps + 2 ** -22)
        assert abs(f["amax_slot"].item() - out.abs().max().item()) <= bound


def test_amax_of_equal_rows():
    """Every row a candidate, more than are computed again."""
    q, k, v = torch.zeros(600, 4, 64, device=DEV).bfloat16(), torch.zeros(600, 4, 64, device=DEV).bfloat16(), torch.ones(600, 4, 64, device=DEV).bfloat16()
    assert run_forward(q, k, v, fp8=True)[2]["amax_slot"].item() == 1.0
    v[:] = 0
    assert run_forward(q, k, v, fp8=True)[2]["amax_slot"].item() == 0.0
    v[7, 2, 5] = math.inf
    assert not math.isfinite(run_forward(q, k, v, fp8=True)[2]["amax_slot"].item())


def test_repeats_bit_for_bit():
    q, k, v, dout = inputs(14, 700, 700, 8, 2, 128)
    a = run_forward(q, k, v, batch=2)
    d = run_backward(dout, q, k, v, a[0], a[1], batch=2)
    for _ in range(3):
        b = run_forward(q, k, v, batch=2)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert all(torch.equal(x, y) for x, y in zip(d, run_backward(dout, q, k, v, b[0], b[1], batch=2)))


def test_differences():
    """The gradients against differences of the definition's forward, along random directions."""
    q, k, v, dout = inputs(15, 60, 90, 4, 2, 64)
    kw = dict(causal=True, window=40)
    o, l, _, _, _ = ref.forward(q, k, v, **kw)
    got = run_backward(dout, q, k, v, o.bfloat16(), l.float(), **kw)
    bounds = [b for _, b in ref.backward(q, k, v, dout, **kw)]
    g = torch.Generator(device=DEV).manual_seed(4)
    h = 1e-5
    for i in range(3):
        way = torch.randn((q, k, v)[i].shape, device=DEV, generator=g).double()
        ends = []
        for sign in (1, -1):
            x = [t.double() for t in (q, k, v)]
            x[i] = x[i] + sign * h * way
            ends.append((ref.forward(*x, **kw)[0] * dout.double()).sum())
        slope = (ends[0] - ends[1]) / (2 * h)
        # the difference's own error is of order h^2 of the third derivative: far below the gradient's rounding
        assert abs((got[i].double() * way).sum() - slope) <= (bounds[i] * way.abs()).sum()


def test_captured_and_replayed():
    """One graph holds both directions; every replay reads the inputs as they are then."""
    q, k, v, dout = inputs(16, 256, 256, 8, 2, 128)
    long_q, long_k, long_v, _ = inputs(17, 2, 4000, 8, 2, 128)
    lens_q, lens_k = offsets([1, 1]), offsets([2500, 1500])
    out, lse = torch.empty_like(q), torch.empty(8, 256, device=DEV)
    out8, s, amax = torch.empty(256, 1024, dtype=torch.uint8, device=DEV), torch.full((1,), 60.0, device=DEV), torch.zeros(1, device=DEV)
    dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
    one = torch.empty_like(long_q)
    ws_fwd = workspace(F.fp8_attention_workspace_bytes, q, k, 2)
    ws, ws_long = workspace(F.fp8_attention_bwd_workspace_bytes, q, k, 2), workspace(F.fp8_attention_workspace_bytes, long_q, long_k, 2)

    def step():
        F.fp8_attention_fwd(q, k, v, out, lse, batch=2, out8=out8, scale=s, amax_slot=amax, workspace=ws_fwd)
        F.fp8_attention_bwd(dout, q, k, v, out, lse, dq, dk, dv, ws, batch=2)
        F.fp8_attention_fwd(long_q, long_k, long_v, one, None, lens_q, lens_k, workspace=ws_long)

    step()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step()
    for turn in range(4):
        g = torch.Generator(device=DEV).manual_seed(100 + turn)
        for t in (q, k, v, dout, long_q, long_k, long_v):
            t.copy_(torch.randn(t.shape, device=DEV, generator=g).bfloat16())
        lens_k.copy_(offsets([3000 - 700 * turn, 1000 + 700 * turn]))
        amax.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, lse, out8, amax, dq, dk, dv, one)]
        amax.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, lse, out8, amax, dq, dk, dv, one)))


def test_on_another_stream():
    q, k, v, dout = inputs(18, 500, 500, 4, 4, 128)
    out, lse, _ = run_forward(q, k, v)
    want = run_backward(dout, q, k, v, out, lse)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    d2 = [torch.zeros_like(t) for t in (q, k, v)]
    ws = workspace(F.fp8_attention_bwd_workspace_bytes, q, k, 1)
    torch.cuda.synchronize()
    F.fp8_attention_fwd(q, k, v, o2, l2, stream=side)
    F.fp8_attention_bwd(dout, q, k, v, o2, l2, *d2, ws, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2) and all(torch.equal(a, b) for a, b in zip(want, d2))


def test_offsets_of_any_content():
    """Offsets out of range or falling: held to the tensors, nothing outside is touched."""
    q, k, v, dout = inputs(19, 64, 64, 2, 1, 64)
    guard = torch.full((3, 64, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    for o in ([-5, 20, 1000], [40, 10, 64], [64, 64, 64], [2 ** 31 - 1, -2 ** 31, 7], [0, 64, 0]):
        off = torch.tensor(o, dtype=torch.int32, device=DEV)
        lse = torch.zeros(2, 64, device=DEV)
        F.fp8_attention_fwd(q, k, v, guard[1], lse, off, off, workspace=workspace(F.fp8_attention_workspace_bytes, q, k, 2))
        run_backward(dout, q, k, v, guard[1].clone(), lse, off, off)
        torch.cuda.synchronize()
        assert bool((guard[0] == 5).all()) and bool((guard[2] == 5).all())


def test_through_the_plain_binding():
    """A prepared call runs the same entry point."""
    q, k, v, dout = inputs(20, 90, 90, 4, 2, 128)
    out, lse = torch.empty_like(q), torch.empty(4, 90, device=DEV)
    F.prepare(F.fp8_attention_fwd, q, k, v, out, lse)()
    want = run_forward(q, k, v)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    d = [torch.empty_like(t) for t in (q, k, v)]
    F.prepare(F.fp8_attention_bwd, dout, q, k, v, out, lse, *d, workspace(F.fp8_attention_bwd_workspace_bytes, q, k, 1))()
    assert all(torch.equal(a, b) for a, b in zip(d, run_backward(dout, q, k, v, out, lse)))
