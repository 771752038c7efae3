"""The router's choice, its weights, counts and balance loss, and their gradient, against the definitions in 64 bits."""
import math

import pytest
import torch

import fp8_delayed_scaling_amd as F

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U32 = 2.0 ** -24


def make(T, E, seed, bf16=False, padded=0.1, ties=False, sd=1.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, E, device=DEV, generator=g) * sd + torch.randn(E, device=DEV, generator=g) * 0.5
    if ties:
        x = torch.round(x * 2) / 2
    x = torch.where(torch.rand(T, 1, device=DEV, generator=g) < padded, torch.full_like(x, -math.inf), x)
    x = torch.where(torch.rand(T, E, device=DEV, generator=g) < padded / 2, torch.full_like(x, -math.inf), x)     # experts closed to a token
    return x.bfloat16() if bf16 else x


def buffers(T, E, top):
    f, i = dict(dtype=torch.float32, device=DEV), dict(dtype=torch.int32, device=DEV)
    return dict(experts=torch.full((T, top), -7, **i), weights=torch.full((T, top), 7.0, **f), lse=torch.full((T,), 7.0, **f),
                counts=torch.full((E + 1,), -7, **i), prob_sum=torch.full((E,), 7.0, **f), loss=torch.full((1,), 7.0, **f))


def run(x, top, normalise=True, stream=None):
    b = buffers(x.shape[0], x.shape[1], top)
    ws = torch.full((max(4, F.fp8_moe_route_workspace_bytes(*x.shape)),), 0xFF, dtype=torch.uint8, device=DEV)
    if stream is not None:
        torch.cuda.synchronize()                       # the buffers' filling, on the current stream
    F.fp8_moe_route(x, *b.values(), ws, normalise, stream=stream)
    return b


def reference(x, top, normalise):
    """As the definition says, the choices by repeated first maxima; weights with the derivative's factors."""
    x = x.double()
    T, E = x.shape
    alive = (x > -math.inf).any(1)
    lse = torch.logsumexp(x, 1)
    p = torch.where(alive[:, None], torch.exp(x - torch.where(alive, lse, torch.zeros_like(lse))[:, None]), torch.zeros_like(x))
    left, experts = x.clone(), torch.full((T, top), -1, dtype=torch.long, device=DEV)
    for j in range(top):
        best = left.max(1).values
        at = (left == best[:, None]).to(torch.int8).argmax(1)      # the first of the largest
        at = torch.where(best > -math.inf, at, torch.full_like(at, -1))
        experts[:, j] = at
        left[at >= 0, at[at >= 0]] = -math.inf
    taken = experts >= 0
    w = torch.where(taken, torch.gather(p, 1, experts.clamp(min=0)), torch.zeros((), dtype=torch.float64, device=DEV))
    if normalise:
        w = w / torch.where(w.sum(1) > 0, w.sum(1), torch.ones_like(lse))[:, None]
    counts = torch.bincount(experts[taken], minlength=E)
    share = counts.double() / max(1, int(counts.sum()))
    live = max(1, int(alive.sum()))
    return dict(experts=experts, weights=w, lse=lse, counts=torch.cat([counts, alive.sum()[None]]), prob_sum=p.sum(0),
                loss=E * (share * p.sum(0)).sum()[None] / live), p, share, live


def rel_of(x, p):
    """What a probability may be off by, relative: the exponential's argument (|x - lse|, float32), the sum of E
    terms and its reciprocal, a few roundings more."""
    E = x.shape[1]
    far = torch.where(p > 0, -torch.log(p.clamp(min=1e-300)), torch.zeros_like(p))
    big = torch.where(x > -math.inf, x.double().abs(), torch.zeros_like(p))
    return 2 * U32 * (4 * far + 4 * big + E / 8 + 32)


def close(got, want, bound):
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), f"off by {off.max().item()}, at most {(off - bound).max().item()} past its bound"


def check(x, top, normalise=True):
    got, (want, p, share, live) = run(x, top, normalise), reference(x, top, normalise)
    assert torch.equal(got["experts"].long(), want["experts"])
    assert torch.equal(got["counts"].long(), want["counts"])
    rel = rel_of(x, p)
    most = rel.max(1).values
    tiny = 1e-37                                       # below it float32 has no full precision
    close(got["weights"], want["weights"], 3 * most[:, None] * want["weights"] + tiny)
    empty = want["lse"] == -math.inf
    assert bool((got["lse"][empty] == -math.inf).all())
    close(got["lse"][~empty], want["lse"][~empty], (2 * U32 * (want["lse"].abs() + 64) + most)[~empty])
    T, E = x.shape
    off = (rel * p).sum(0) + 2 * U32 * (T / 64 + 300) * want["prob_sum"] + T * tiny
    close(got["prob_sum"], want["prob_sum"], off)
    close(got["loss"], want["loss"], E * (share * off).sum() / live + 2 * U32 * (E + 64) * want["loss"].abs())
    return got


CASES = [(1, 1, 1), (1, 64, 4), (3, 5, 5), (16, 64, 4), (17, 63, 8), (100, 65, 3), (128, 128, 2), (129, 128, 8), (500, 40, 6), (1000, 256, 8),
         (777, 257, 4), (300, 512, 8), (260, 1000, 10), (200, 1024, 1), (140, 100, 100), (130, 70, 66), (5000, 64, 4), (4097, 16, 2)]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("normalise", [False, True])
def test_forward(case, bf16, normalise):
    T, E, top = case
    check(make(T, E, T + E, bf16), top, normalise)


def test_ties_go_to_the_lowest_expert():
    for E in (7, 64, 100, 300, 1024):
        check(make(300, E, E, ties=True), min(E, 8))
    x = torch.zeros(130, 200, device=DEV)
    got = check(x, 6)
    assert got["experts"][0].tolist() == [0, 1, 2, 3, 4, 5]


def test_rows_and_experts_that_are_closed():
    x = torch.full((200, 70), -math.inf, device=DEV)
    got = run(x, 3)
    assert bool((got["experts"] == -1).all()) and bool((got["weights"] == 0).all()) and bool((got["lse"] == -math.inf).all())
    assert int(got["counts"].abs().sum()) == 0 and float(got["prob_sum"].abs().sum()) == 0 and got["loss"].item() == 0
    x[5, 66], x[9, 3], x[9, 65] = 2.0, 1.0, 1.0
    got = check(x, 3)
    assert got["experts"][5].tolist() == [66, -1, -1] and got["experts"][9].tolist() == [3, 65, -1]
    assert got["weights"][5].tolist() == [1, 0, 0] and got["weights"][9].tolist() == [0.5, 0.5, 0]
    lowest = torch.finfo(torch.float32).min             # the lowest value is a logit like any other
    x = torch.full((140, 20), lowest, device=DEV)
    got = check(x, 2)
    assert got["experts"][0].tolist() == [0, 1]
    x[:, 4] = 0
    assert check(x, 2)["experts"][0].tolist() == [4, 0]


def test_no_rows():
    got = run(torch.empty(0, 9, device=DEV), 2)
    assert bool((got["counts"] == 0).all()) and bool((got["prob_sum"] == 0).all()) and got["loss"].item() == 0


def test_not_a_number():
    """A NaN or an infinity shows in the loss; the row's choices stay in range, the other rows are as they were."""
    for bad in (math.nan, math.inf):
        x = make(300, 50, 3, padded=0.0)
        want = run(x, 4)
        x[7, 11] = bad
        got = run(x, 4)
        assert math.isnan(got["loss"].item()) and math.isnan(got["lse"][7].item())
        assert int(got["experts"].min()) >= -1 and int(got["experts"].max()) < 50
        keep = torch.arange(300, device=DEV) != 7
        for n in ("experts", "weights", "lse"):
            assert torch.equal(got[n][keep], want[n][keep])
        assert int(got["counts"][-1]) == 300
    x[7] = math.nan
    got = run(x, 4)
    assert math.isnan(got["loss"].item()) and got["experts"][7].tolist() == [-1] * 4


def test_strided_rows():
    wide = torch.randn(400, 100, device=DEV)
    for x in (wide[:, 3:70], wide[::3, :64], wide.bfloat16()[:, 5:38]):
        got, want = run(x, 4), run(x.contiguous(), 4)
        assert all(torch.equal(got[n], want[n]) for n in got)


# ------------------------------------------------------------------------------------ gradient

def backward(x, f, dweights, dloss, normalise):
    d = torch.full_like(x, 7.0)
    F.fp8_moe_route_bwd(x, f["experts"], f["weights"], f["lse"], f["counts"], dweights, dloss, d, normalise)
    return d


def reference_backward(x, top, normalise, dweights, dloss):
    want, p, share, live = reference(x, top, normalise)
    T, E = x.shape
    dx, mag = torch.zeros_like(p), torch.zeros_like(p)
    if dloss is not None:
        c = dloss.double() * E * share / live
        dx += p * (c - (p * c).sum(1, keepdim=True))
        mag += p * (c.abs() + (p * c.abs()).sum(1, keepdim=True))
    if dweights is not None:
        taken, at = want["experts"] >= 0, want["experts"].clamp(min=0)
        g = torch.where(taken, want["weights"] * dweights.double(), torch.zeros((), dtype=torch.float64, device=DEV))
        inside = torch.zeros_like(p).scatter_add_(1, at, torch.where(taken, want["weights"], torch.zeros_like(want["weights"])))
        base = inside if normalise else p
        dx += torch.zeros_like(p).scatter_add_(1, at, g) - base * g.sum(1, keepdim=True)
        mag += torch.zeros_like(p).scatter_add_(1, at, g.abs()) + base * g.abs().sum(1, keepdim=True)
    return dx, mag, p


def forward_as_given(x, top, normalise):
    """What the forward writes, from the definition: the backward is checked on its own."""
    w = reference(x, top, normalise)[0]
    return dict(experts=w["experts"].int(), weights=w["weights"].float(), lse=w["lse"].float(), counts=w["counts"].int())


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("normalise", [False, True])
@pytest.mark.parametrize("parts", ["both", "weights", "loss"])
def test_backward(case, bf16, normalise, parts):
    T, E, top = case
    x = make(T, E, T * 3 + E, bf16)
    g = torch.Generator(device=DEV).manual_seed(T)
    dweights = torch.randn(T, top, device=DEV, generator=g) if parts != "loss" else None
    dloss = torch.full((1,), 3.0, device=DEV) if parts != "weights" else None
    want, mag, p = reference_backward(x, top, normalise, dweights, dloss)
    got = backward(x, forward_as_given(x, top, normalise), dweights, dloss, normalise)
    most = rel_of(x, p).max(1, keepdim=True).values
    bound = mag * (3 * most + 2 * U32 * (E + top)) + 1e-37
    close(got, want, bound + (2.0 ** -8 * (want.abs() + bound) if bf16 else 0))


def test_backward_of_padding_and_dropped_choices():
    x = make(200, 33, 8, padded=0.0)
    x[3] = -math.inf
    f = run(x, 4)
    f["experts"][10, 1], f["experts"][11, 2] = -1, 33            # choices that were dropped afterwards
    dw = torch.randn(200, 4, device=DEV)
    got = backward(x, f, dw, torch.ones(1, device=DEV), False)
    assert bool((got[3] == 0).all()) and bool(got.isfinite().all())
    dw[10, 1] = dw[11, 2] = math.nan                             # their weights' gradients are not read
    assert torch.equal(got, backward(x, f, dw, torch.ones(1, device=DEV), False))


def test_differences():
    """Against differences of the definition along random directions: choices and counts stay, logits move."""
    x = make(60, 20, 5, padded=0.0)
    for normalise in (False, True):
        dw, dl = torch.randn(60, 3, device=DEV), torch.full((1,), 2.0, device=DEV)
        f = forward_as_given(x, 3, normalise)
        got = backward(x, f, dw, dl, normalise).double()
        at, share, E = f["experts"].long(), f["counts"][:-1].double() / f["counts"][:-1].sum(), 20

        def value(z):
            p = torch.softmax(z, 1)
            w = torch.gather(p, 1, at)
            w = w / w.sum(1, keepdim=True) if normalise else w
            return (w * dw.double()).sum() + dl.double() * E * (share * p.mean(0)).sum()

        way, h = torch.randn(60, 20, device=DEV).double(), 1e-5
        slope = (value(x.double() + h * way) - value(x.double() - h * way)) / (2 * h)
        _, mag, p = reference_backward(x, 3, normalise, dw, dl)
        bound = (mag * (3 * rel_of(x, p) + 2 * U32 * 23) * way.abs()).sum() + 1e-9 * (mag * way.abs()).sum()
        assert abs((got * way).sum() - slope) <= bound


def test_backward_strided():
    wide = torch.randn(300, 90, device=DEV)
    x = wide[:, 10:60]
    f = run(x, 4)
    dw, dl = torch.randn(300, 4, device=DEV), torch.ones(1, device=DEV)
    into = torch.full((300, 80), 7.0, device=DEV)
    F.fp8_moe_route_bwd(x, f["experts"], f["weights"], f["lse"], f["counts"], dw, dl, into[:, 4:54])
    assert torch.equal(into[:, 4:54], backward(x.contiguous(), f, dw, dl, True))
    assert bool((into[:, :4] == 7).all()) and bool((into[:, 54:] == 7).all())


def test_repeats_captured_and_on_other_streams():
    x = make(3000, 64, 6)
    b, ws = buffers(3000, 64, 4), torch.empty(F.fp8_moe_route_workspace_bytes(3000, 64), dtype=torch.uint8, device=DEV)
    dw, dl, d = torch.randn(3000, 4, device=DEV), torch.ones(1, device=DEV), torch.empty_like(x)

    def step():
        F.fp8_moe_route(x, *b.values(), ws)
        F.fp8_moe_route_bwd(x, b["experts"], b["weights"], b["lse"], b["counts"], dw, dl, d)

    step()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step()
    for turn in range(4):
        x.copy_(make(3000, 64, 50 + turn))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*b.values(), d)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, (*b.values(), d)))
    torch.cuda.synchronize()
    want, side = run(x, 4), torch.cuda.Stream()
    other = run(x, 4, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(want[n], other[n]) for n in want)
    step()
    torch.cuda.synchronize()
    other = torch.zeros_like(x)
    torch.cuda.synchronize()
    F.fp8_moe_route_bwd(x, want["experts"], want["weights"], want["lse"], want["counts"], dw, dl, other, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(d, other)


def test_feeds_the_plan():
    """The choices as fp8_moe_plan reads them: every expert's rows are its count."""
    x = make(700, 24, 9)
    f = run(x, 3)
    cap = F.fp8_moe_capacity(700, 3, 24)
    i32 = dict(dtype=torch.int32, device=DEV)
    off, src, slot = torch.empty(25, **i32), torch.empty(cap, **i32), torch.empty(700, 3, **i32)
    ws = torch.empty(max(4, F.fp8_moe_workspace_bytes(700, 3, 24)), dtype=torch.uint8, device=DEV)
    F.fp8_moe_plan(f["experts"], 24, 16, off, src, slot, ws)
    rows = [int((src[a:b] >= 0).sum()) for a, b in zip(off.tolist(), off.tolist()[1:])]
    assert rows == f["counts"][:-1].tolist() and torch.equal(slot >= 0, f["experts"] >= 0)
