"""Tokens sorted by expert and back (fp8_moe_*): the plan against counting, sorted rows and their
codes bit for bit, combine and the weights' gradient against 64 bits; one token to many, dropped
choices, experts without tokens, bad index buffers, graphs, buffers past 2^31 elements."""
import numpy as np
import pytest
import torch

import block_ref as R
import fp8_delayed_scaling_amd as F
import oracle
from helpers import DEV, bf16_host, f32_bits, to_f64, u8_host

pytestmark = pytest.mark.gpu

BF = dict(device=DEV, dtype=torch.bfloat16)
F32 = dict(device=DEV, dtype=torch.float32)
U8 = dict(device=DEV, dtype=torch.uint8)
I32 = dict(device=DEV, dtype=torch.int32)


def _choices(T, k, E, seed, drop=0.05, skew=1.0):
    rng = np.random.default_rng(seed)
    p = np.exp(skew * rng.standard_normal(E))
    e = rng.choice(E, size=(T, k), p=p / p.sum()).astype(np.int32)
    e[rng.random((T, k)) < drop] = -1
    e[rng.random((T, k)) < drop / 4] = E + 5
    return e


def _plan(e, E, align=16, extra=0):
    T, k = e.shape
    cap = F.fp8_moe_capacity(T, k, E, align) + extra
    offsets, src, slot = torch.full((E + 1,), 77, **I32), torch.full((cap,), 77, **I32), torch.full((T, k), 77, **I32)
    ws = torch.full((F.fp8_moe_workspace_bytes(T, k, E),), 0xA5, **U8)
    F.fp8_moe_plan(torch.from_numpy(e).to(DEV), E, align, offsets, src, slot, ws)
    return offsets, src, slot


@pytest.mark.parametrize("T,k,E,align", [(1, 1, 1, 16), (1, 8, 64, 16), (3, 2, 5, 32), (64, 4, 64, 16), (1000, 1, 3, 128),
                                         (1024, 4, 64, 16), (1025, 4, 63, 16), (4097, 1, 1024, 16), (700, 6, 1000, 48),
                                         (20000, 4, 128, 16), (33000, 8, 17, 1024), (70001, 1, 256, 16)])
def test_plan(T, k, E, align):
    print(f"plan T={T} k={k} E={E} align={align}", flush=True)
    for seed, drop, skew, extra in ((1, 0.05, 1.0, 0), (2, 0.0, 4.0, 160), (3, 1.0, 0.0, 0)):
        e = _choices(T, k, E, seed, drop, skew)
        offsets, src, slot = _plan(e, E, align, extra)
        want = R.plan(e, E, align, src.numel())
        for got, w, n in zip((offsets, src, slot), want, ("offsets", "src", "slot")):
            assert np.array_equal(got.cpu().numpy(), w), (n, seed)


def test_plan_of_no_tokens():
    print("plan of no tokens", flush=True)
    offsets, src, slot = _plan(np.zeros((0, 2), np.int32), 9, extra=64)
    assert (offsets == 0).all() and (src == -1).all()


SORTS = [(1, 1, 4, 16), (1, 8, 64, 4096), (5, 2, 3, 48), (37, 3, 8, 272), (300, 4, 16, 1040), (1111, 2, 7, 2048), (3000, 6, 40, 2064)]


@pytest.mark.parametrize("T,k,E,H", SORTS)
@pytest.mark.parametrize("weighted", [False, True])
def test_sort_cast(T, k, E, H, weighted):
    print(f"sort cast T={T} k={k} E={E} H={H} weighted={weighted}", flush=True)
    e = _choices(T, k, E, T + H)
    _, src, _ = _plan(e, E)
    cap = src.numel()
    g = torch.Generator().manual_seed(H)
    x = (torch.randn(T, H, generator=g) * 3).to(torch.bfloat16).to(DEV)
    w = torch.rand(T, k, generator=g).to(DEV) if weighted else None
    src_h = src.cpu().numpy()
    live = src_h >= 0
    x32 = x.float().cpu().numpy()
    v = np.zeros((cap, H), np.float32)
    v[live] = x32[src_h[live] // k]
    if weighted:
        v[live] = v[live] * w.cpu().numpy().reshape(-1)[src_h[live]][:, None]
    for fmt, scale in ((F.E4M3, 37.7), (F.E5M2, 4000.0)):
        want = oracle.encode(v * np.float32(scale), fmt).reshape(cap, H)
        want[~live] = 0
        for transpose in (False, True):
            out, out_t = torch.full((cap, H), 0xA5, **U8), torch.full((H, cap), 0xA5, **U8) if transpose else None
            amax, sinv = torch.zeros(1, **F32), torch.zeros(1, **F32)
            F.fp8_moe_sort_cast(x, src, k, w, torch.tensor([scale], **F32), fmt, out, out_t, sinv, amax)
            assert np.array_equal(u8_host(out), want)
            if transpose:
                assert np.array_equal(u8_host(out_t), want.T)
            assert f32_bits(amax.item()) == f32_bits(np.abs(v).max() if v.size else 0.0)
            assert f32_bits(sinv.item()) == f32_bits(np.float32(1.0) / np.float32(scale))
    # bfloat16 rows
    out = torch.full((cap, H), float("nan"), **BF)
    F.fp8_moe_sort_bf16(x, src, k, w, out)
    assert np.array_equal(bf16_host(out), bf16_host(torch.from_numpy(v).to(torch.bfloat16)))


@pytest.mark.parametrize("T,k,E,H", SORTS)
def test_sort_codes(T, k, E, H):
    print(f"sort codes T={T} k={k} E={E} H={H}", flush=True)
    _, src, _ = _plan(_choices(T, k, E, T + H), E)
    cap = src.numel()
    x8 = torch.randint(0, 256, (T, H), dtype=torch.uint8, generator=torch.Generator().manual_seed(T)).to(DEV)
    s = src.cpu().numpy()
    want = np.zeros((cap, H), np.uint8)
    want[s >= 0] = u8_host(x8)[s[s >= 0] // k]
    out, out_t = torch.full((cap, H), 0xA5, **U8), torch.full((H, cap), 0xA5, **U8)
    F.fp8_moe_sort_codes(x8, src, k, out)
    assert np.array_equal(u8_host(out), want)
    out.fill_(0x5A)
    F.fp8_moe_sort_codes(x8, src, k, out, out_t)
    assert np.array_equal(u8_host(out), want) and np.array_equal(u8_host(out_t), want.T)


def test_sort_special_values_and_bad_indices():
    """NaN and infinities keep the cast's rules; weights of dropped choices and indices out of range
    are not read; a row that no choice fills is zeros even where its neighbours are NaN."""
    T, k, E, H = 40, 2, 5, 256
    print("sort special values", flush=True)
    _, src, slot = _plan(_choices(T, k, E, 4, drop=0.3), E)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    x[3, 7], x[4, 9], x[5, 1] = float("nan"), float("inf"), float("-inf")
    w = torch.ones(T, k, **F32)
    w[slot < 0] = float("nan")
    src[2], src[9], src[11] = 2 ** 31 - 1, -7, T * k          # three indices out of range
    s = src.cpu().numpy()
    live = (s >= 0) & (s < T * k)
    v = np.zeros((s.size, H), np.float32)
    v[live] = x.float().cpu().numpy()[s[live] // k]
    for with_t in (False, True):
        out, out_t = torch.empty(s.size, H, **U8), torch.empty(H, s.size, **U8) if with_t else None
        amax = torch.zeros(1, **F32)
        F.fp8_moe_sort_cast(x, src, k, w, torch.full((1,), 8.0, **F32), F.E4M3, out, out_t, None, amax)
        want = oracle.encode(v * np.float32(8.0), F.E4M3).reshape(v.shape)
        want[~live] = 0
        assert np.array_equal(u8_host(out), want)
        assert np.isnan(amax.item()) == np.isnan(v).any()


@pytest.mark.parametrize("T,k,E,H", SORTS + [(50, 1, 4, 64), (50, 5, 9, 8192), (9, 13, 30, 96)])
def test_combine_and_weight_grad(T, k, E, H):
    print(f"combine T={T} k={k} E={E} H={H}", flush=True)
    e = _choices(T, k, E, 3 * T + H, drop=0.1)
    if T > 2:
        e[1] = -1                                             # a token without any expert
    _, src, slot = _plan(e, E)
    cap = src.numel()
    g = torch.Generator().manual_seed(H + 1)
    ys = torch.randn(cap, H, generator=g).to(torch.bfloat16).to(DEV)
    ys[src < 0] = float("nan")                                # padding rows are not read
    w = (torch.rand(T, k, generator=g) + 0.1).to(DEV)
    w[slot < 0] = float("inf")                                # nor are dropped choices' weights
    dy = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    s = slot.cpu().numpy()
    rows = np.zeros((T, k, H))
    rows[s >= 0] = to_f64(ys)[s[s >= 0]]
    wh = np.where(s >= 0, w.cpu().numpy().astype(np.float64), 0.0)
    for weights, ww in ((w, wh), (None, (s >= 0) * 1.0)):
        y = torch.full((T, H), float("nan"), **BF)
        F.fp8_moe_combine(ys, slot, weights, y)
        terms = rows * ww[:, :, None]
        want, err = terms.sum(1), (k + 1) * R.U * np.abs(terms).sum(1)
        bound = err + R.BF16 * (np.abs(want) + err)
        assert (np.abs(to_f64(y) - want) <= bound).all()
    dw = torch.full((T, k), float("nan"), **F32)
    F.fp8_moe_weight_grad(dy, ys, slot, dw)
    terms = rows * to_f64(dy)[:, None]
    assert (np.abs(dw.double().cpu().numpy() - terms.sum(2)) <= (H + 8) * R.U * np.abs(terms).sum(2)).all()
    bad = slot.clone()
    bad[0, 0], bad[-1, -1] = cap, 2 ** 31 - 1                 # out of range: as if dropped
    keep = slot.clone()
    keep[0, 0], keep[-1, -1] = -1, -1
    out = []
    for sl in (bad, keep):
        y, dw = torch.empty(T, H, **BF), torch.empty(T, k, **F32)
        F.fp8_moe_combine(ys, sl, w, y)
        F.fp8_moe_weight_grad(dy, ys, sl, dw)
        out.append((y, dw))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


def test_sort_and_back_is_the_identity_and_its_gradient():
    """Every choice back once: combine(sort(x)) = top * x exactly for small integers, and
    <sort(x), u> = <x, combine(u)> (the sort's gradient is the combine without weights)."""
    T, k, E, H = 200, 4, 16, 512
    print("sort and back", flush=True)
    _, src, slot = _plan(_choices(T, k, E, 8, drop=0.0) % E, E)
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.integers(-8, 9, (T, H)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    xs, y = torch.empty(src.numel(), H, **BF), torch.empty(T, H, **BF)
    F.fp8_moe_sort_bf16(x, src, k, None, xs)
    F.fp8_moe_combine(xs, slot, None, y)
    assert torch.equal(y.float(), 4.0 * x.float())
    u = torch.from_numpy(rng.integers(-8, 9, (src.numel(), H)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    du = torch.empty(T, H, **BF)
    F.fp8_moe_combine(u, slot, None, du)
    assert (xs.double() * u.double()).sum().item() == (x.double() * du.double()).sum().item()


def test_graph_replays_with_new_routing():
    T, k, E, H = 3000, 2, 24, 512
    print("moe graph", flush=True)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    cap = F.fp8_moe_capacity(T, k, E)
    e = torch.from_numpy(_choices(T, k, E, 0)).to(DEV)
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(3)).to(DEV)
    b = dict(offsets=torch.empty(E + 1, **I32), src=torch.empty(cap, **I32), slot=torch.empty(T, k, **I32),
             xs=torch.empty(cap, H, **U8), xt=torch.empty(H, cap, **U8), rows=torch.empty(cap, H, **BF), y=torch.empty(T, H, **BF),
             amax=torch.zeros(1, **F32), sinv=torch.zeros(1, **F32), dw=torch.empty(T, k, **F32))
    ws = torch.empty(F.fp8_moe_workspace_bytes(T, k, E), **U8)
    scale = torch.full((1,), 40.0, **F32)

    def step(b):
        F.fp8_moe_plan(e, E, 16, b["offsets"], b["src"], b["slot"], ws)
        F.fp8_moe_sort_cast(x, b["src"], k, w, scale, F.E4M3, b["xs"], b["xt"], b["sinv"], b["amax"])
        F.fp8_moe_sort_bf16(x, b["src"], k, None, b["rows"])
        F.fp8_moe_combine(b["rows"], b["slot"], w, b["y"])
        F.fp8_moe_weight_grad(x, b["rows"], b["slot"], b["dw"])

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        step(b)
    for seed in (1, 2, 3):
        e.copy_(torch.from_numpy(_choices(T, k, E, seed)))
        g.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in b.items()}
        want = {n: torch.zeros_like(t) for n, t in b.items()}
        step(want)
        torch.cuda.synchronize()
        for n in b:
            if n != "amax":
                assert torch.equal(got[n], want[n]), (seed, n)


def test_rows_past_2_31_elements():
    T, k, E, H = 40, 8, 8, 8192
    cap = (1 << 18) + 320
    print(f"moe {cap}x{H}", flush=True)
    e = _choices(T, k, E, 1, drop=0.0) % E
    offsets, src, slot = torch.empty(E + 1, **I32), torch.empty(cap, **I32), torch.empty(T, k, **I32)
    F.fp8_moe_plan(torch.from_numpy(e).to(DEV), E, 16, offsets, src, slot, None)
    x8 = torch.randint(0, 256, (T, H), dtype=torch.uint8, generator=torch.Generator().manual_seed(1)).to(DEV)
    src = torch.roll(src, cap - 320 - int(offsets[E].item()) + 320)     # the live rows at the far end
    out, out_t = torch.empty(cap, H, **U8), torch.empty(H, cap, **U8)
    F.fp8_moe_sort_codes(x8, src, k, out, out_t)
    live = src >= 0
    assert torch.equal(out[live], x8[(src[live] // k).long()])
    tail = out[-512:]
    assert torch.equal(out_t[:, -512:].t(), tail)
    assert (out[:1000] == 0).all() and (out_t[-1, :1000] == 0).all()
    ys = torch.zeros(cap, H, **BF)
    ys[-512:] = 1.0
    y = torch.empty(T, H, **BF)
    far = torch.full((T, k), -1, **I32)
    far[:, 0] = cap - 1
    F.fp8_moe_combine(ys, far, None, y)
    assert (y == 1).all()
