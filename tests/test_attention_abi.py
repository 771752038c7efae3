"""Refusals of attention and of the router, on the CPU: the C entry points reject bad arguments before any HIP
call, the binding rejects mis-sized tensors before it takes a pointer."""
import ctypes

import pytest
import torch

import fp8_delayed_scaling_amd as F

A16 = 1 << 20        # a fake 16-byte aligned address: never dereferenced, validation fails first
BIG = 1 << 40        # workspace bytes that are always enough


def _call(name, ok):
    f = getattr(F.lib(), name)

    def call(**kw):
        a = dict(ok, **kw)
        assert set(a) == set(ok)
        return f(*a.values())
    return call


def H(data=A16, ts=None, hs=None, heads=4, D=64):
    return F._Heads(data, heads * D if ts is None else ts, D if hs is None else hs)


FWD = dict(q=H(), k=H(heads=2), v=H(heads=2), out=H(), lse=A16, out8=None, scale=None, fmt=0, sinv=None, amax=None, oq=None, ok=None, B=2,
           Tq=100, Tk=200, Hq=4, Hkv=2, D=64, sc=0.125, causal=1, window=0, ws=A16, bytes=BIG, st=None)
BWD = dict(do=H(), q=H(), k=H(heads=2), v=H(heads=2), out=H(), lse=A16, dq=H(), dk=H(heads=2), dv=H(heads=2), oq=None, ok=None, B=2, Tq=100,
           Tk=200, Hq=4, Hkv=2, D=64, sc=0.125, causal=1, window=0, ws=A16, bytes=BIG, st=None)


@pytest.mark.parametrize("name,ok", [("fp8_attention_fwd", FWD), ("fp8_attention_bwd", BWD)])
def test_attention_validation(name, ok):
    call = _call(name, ok)
    assert call(Hq=3) == -2 and call(Hkv=0) == -2 and call(Hq=0) == -2
    for D in (0, 4, 60, 136, -8):
        assert call(D=D) == -2
    assert call(B=-1) == -2 and call(Tq=-2) == -2 and call(Tk=-2) == -2
    assert call(Tq=101) == -2 and call(Tk=201) == -2                   # not equal parts
    assert call(Tq=1 << 27) == -2 and call(Tk=1 << 28) == -2           # tokens x heads past 2^28
    assert call(oq=A16) == -1 and call(ok=A16) == -1                   # offsets go together
    assert call(oq=A16 + 2, ok=A16) == -3 and call(oq=A16, ok=A16 + 1) == -3
    assert call(sc=0.0) == -7 and call(sc=-1.0) == -7 and call(sc=float("nan")) == -7 and call(sc=float("inf")) == -7
    assert call(window=-1) == -7 and call(window=5, causal=0) == -7
    inputs = ["q"] + (["do", "out"] if "do" in ok else [])
    outputs = ["dq", "dk", "dv"] if "do" in ok else ["out"]
    for n in [*inputs, "k", "v", *outputs]:
        assert call(**{n: H(data=A16 + 8)}) == -3, n
        assert call(**{n: H(ts=260)}) == -3 and call(**{n: H(hs=68)}) == -3, n
        assert call(**{n: H(ts=56)}) == -2 and call(**{n: H(ts=-256)}) == -2 and call(**{n: H(hs=-64)}) == -2, n
        assert call(**{n: H(ts=1 << 23)}) == -2, n
        if n != "out" or "do" in ok:
            assert call(**{n: H(data=None)}) == -1, n
    for n in outputs:
        assert call(**{n: H(hs=0)}) == -2 and call(**{n: H(hs=56)}) == -2, n
    assert call(q=H(hs=1 << 29)) == -2                                 # a group's heads within 2^30 elements
    assert call(lse=A16 + 2) == -3 and call(ws=A16 + 8) == -3
    assert call(B=0) == 0
    assert call(oq=A16, ok=A16, B=1 << 31) == -2
    assert call(oq=A16, ok=A16, B=1 << 30) == -2                       # more tiles than a launch numbers


def test_attention_forward_only():
    call = _call("fp8_attention_fwd", FWD)
    assert call(fmt=2) == -4
    assert call(out=H(data=None)) == -1 and call(out8=A16) == -1       # nothing to write, codes without a scale
    assert call(out8=A16 + 8, scale=A16) == -3 and call(out8=A16, scale=A16 + 2) == -3
    assert call(amax=A16 + 1) == -3 and call(sinv=A16 + 1) == -3
    assert call(Tq=0) == 0
    need = F.fp8_attention_workspace_bytes(2, 8000, 2, 4, 2, 64)
    assert need > 0
    assert call(Tq=2, Tk=8000, ws=None) == -5 and call(Tq=2, Tk=8000, bytes=need - 1) == -5
    # an amax is made sure of in a second pass over the waves' largest outputs
    need = F.fp8_attention_workspace_bytes(100, 200, 2, 4, 2, 64)
    assert need > 0 and call(out8=A16, scale=A16, amax=A16, bytes=16) == -5 and call(out8=A16, scale=A16, amax=A16, ws=None) == -5
    for bad in ((-1, 8, 1, 4, 2, 64), (8, 8, 0, 4, 2, 64), (8, 8, 1, 4, 3, 64), (1 << 40, 8, 1, 4, 2, 64)):
        assert F.fp8_attention_workspace_bytes(*bad) == 0


def test_attention_backward_only():
    call = _call("fp8_attention_bwd", BWD)
    assert call(lse=None) == -1
    need = F.fp8_attention_bwd_workspace_bytes(100, 200, 2, 4, 2, 64)
    assert need > 0 and call(ws=None) == -5 and call(bytes=need - 1) == -5
    assert call(Tq=0, Tk=0) == 0
    assert F.fp8_attention_bwd_workspace_bytes(0, 200, 2, 4, 2, 64) == 0


def test_workspace_holds_either_kind_of_batch():
    """The bytes asked for do not depend on whether offsets will be given."""
    for Tq, Tk, B in ((4, 9000, 4), (5, 9001, 4), (256, 16384, 1), (300, 16383, 2)):
        assert F.fp8_attention_workspace_bytes(Tq, Tk, B, 8, 2, 128) % 4 == 0


ROUTE = dict(l=A16, dt=1, ld=64, T=1000, E=64, top=4, norm=1, ex=A16, w=A16, lse=A16, cnt=A16, ps=A16, loss=A16, ws=A16, bytes=BIG, st=None)
ROUTE_BWD = dict(l=A16, dt=1, ld=64, T=1000, E=64, top=4, norm=1, ex=A16, w=A16, lse=A16, cnt=A16, dw=A16, dl=A16, d=A16, ldd=64, st=None)


@pytest.mark.parametrize("name,ok", [("fp8_moe_route", ROUTE), ("fp8_moe_route_bwd", ROUTE_BWD)])
def test_route_validation(name, ok):
    call = _call(name, ok)
    assert call(dt=2) == -4 and call(dt=-1) == -4
    assert call(E=0) == -2 and call(E=1025, ld=2000) == -2 and call(top=0) == -2 and call(top=65) == -2
    assert call(ld=63) == -2 and call(T=-1) == -2 and call(T=1 << 30) == -2 and call(ld=1 << 40) == -2
    assert call(l=None) == -1 and call(lse=None) == -1
    assert call(l=A16 + 2) == -3 and call(l=A16 + 1, dt=0) == -3 and call(ex=A16 + 2) == -3 and call(w=A16 + 1) == -3
    assert call(lse=A16 + 2) == -3 and call(cnt=A16 + 2) == -3


def test_route_directions():
    call = _call("fp8_moe_route", ROUTE)
    for n in ("ex", "w", "cnt", "ps", "loss"):
        assert call(**{n: None}) == -1, n
    need = F.fp8_moe_route_workspace_bytes(1000, 64)
    assert need > 0 and call(ws=None) == -5 and call(bytes=need - 1) == -5 and call(ws=A16 + 2) == -3
    assert F.fp8_moe_route_workspace_bytes(16, 64) == 0 and F.fp8_moe_route_workspace_bytes(-1, 64) == 0
    call = _call("fp8_moe_route_bwd", ROUTE_BWD)
    assert call(ldd=63) == -2 and call(d=None) == -1 and call(ex=None) == -1 and call(w=None) == -1 and call(cnt=None) == -1
    assert call(d=A16 + 2) == -3 and call(dl=A16 + 2) == -3
    assert call(T=0) == 0


def _raises(match, fn, *a, **kw):
    with pytest.raises((ValueError, TypeError), match=match):
        fn(*a, **kw)


def test_attention_binding_checks():
    bf = dict(dtype=torch.bfloat16)
    t = lambda *s: torch.zeros(s, **bf)  # noqa: E731
    ok = dict(q=t(6, 4, 16), k=t(9, 2, 16), v=t(9, 2, 16), out=t(6, 4, 16), lse=torch.zeros(4, 6))

    def bad(match, **kw):
        _raises(match, F.fp8_attention_fwd, **dict(ok, **kw))

    off = torch.tensor([0, 6], dtype=torch.int32)
    bad("offsets_q and offsets_k", offsets_q=off)
    bad("offsets_k", offsets_q=off, offsets_k=torch.tensor([0, 1, 9], dtype=torch.int32))
    bad("offsets_q", offsets_q=off.long(), offsets_k=off)
    bad("k", k=t(9, 2))
    bad("v", v=t(8, 2, 16))
    bad("v", v=t(9, 2, 16).float())
    bad("out", out=t(6, 4, 24))
    bad("lse", lse=torch.zeros(6, 4))
    bad("out8", out8=torch.zeros(6, 4, 16, dtype=torch.uint8))
    bad("contiguous", q=t(6, 4, 32)[:, :, ::2])
    bad("GPU", stream=0)
    ok = dict(dout=t(6, 4, 16), q=t(6, 4, 16), k=t(9, 2, 16), v=t(9, 2, 16), out=t(6, 4, 16), lse=torch.zeros(4, 6), dq=t(6, 4, 16),
              dk=t(9, 2, 16), dv=t(9, 2, 16), workspace=None)

    def bad_bwd(match, **kw):
        _raises(match, F.fp8_attention_bwd, **dict(ok, **kw))

    for n in ("dout", "out", "dq", "dk", "dv"):
        bad_bwd(n, **{n: t(5, 4, 16)})
        bad_bwd(n, **{n: None})
    bad_bwd("lse", lse=None)
    bad_bwd("GPU", stream=0)


def test_route_binding_checks():
    f = torch.zeros
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ok = dict(logits=f(5, 8), experts=i(5, 2), weights=f(5, 2), lse=f(5), counts=i(9), prob_sum=f(8), loss=f(1))

    def bad(match, fn=F.fp8_moe_route, **kw):
        _raises(match, fn, **dict(ok, **kw))

    bad("logits", logits=f(5, 8).double())
    bad("logits", logits=f(40))
    bad("logits rows", logits=f(5, 16)[:, ::2])
    bad("experts", experts=i(10))
    bad("experts", experts=i(4, 2))
    bad("weights", weights=f(5, 3))
    bad("lse", lse=f(4))
    bad("counts", counts=i(8))
    bad("prob_sum", prob_sum=f(9))
    bad("GPU", stream=0)
    ok = dict(logits=f(5, 8), experts=i(5, 2), weights=f(5, 2), lse=f(5), counts=i(9), dweights=f(5, 2), dloss=f(1), dlogits=f(5, 8))
    bad("dlogits", F.fp8_moe_route_bwd, dlogits=f(5, 8).bfloat16())
    bad("dlogits", F.fp8_moe_route_bwd, dlogits=f(5, 9))
    bad("dweights", F.fp8_moe_route_bwd, dweights=f(5, 1))
    bad("GPU", F.fp8_moe_route_bwd, stream=0)


def test_structure_of_heads():
    assert ctypes.sizeof(F._Heads) == 24


@pytest.mark.parametrize("name,ok", [("fp8_attention_fwd", FWD), ("fp8_attention_bwd", BWD)])
def test_softmax_scale_range(name, ok):
    """lse / softmax_scale and softmax_scale * log2(e) have to stay finite."""
    call = _call(name, ok)
    assert call(sc=1e-31) == -7 and call(sc=1e31) == -7 and call(sc=3e38) == -7
    assert call(sc=1e-29, B=0) == 0 and call(sc=1e29, B=0) == 0


def test_attention_group_reach():
    """Heads that share a key/value head are reached by 32-bit byte offsets from one base, 34 tokens on at most."""
    call = _call("fp8_attention_bwd", BWD)
    reach = (1 << 30) // 2 - 34 * 256 // 2 - 64
    for n in ("q", "do"):
        assert call(**{n: H(hs=(reach // 8 + 1) * 8)}) == -2
        assert call(**{n: H(hs=reach // 8 * 8)}, ws=None) == -5        # passes: the next refusal is the workspace's
