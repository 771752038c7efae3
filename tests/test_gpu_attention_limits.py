"""Attention and the router where their addressing, their ranges and their order end: caches past 32-bit offsets, calls
that overlap in time, no tokens on one side, more candidates for the amax than are computed again, one expert twice."""
import pytest
import torch

import attention_ref as ref
import fp8_delayed_scaling_amd as F
from test_gpu_attention import DEV, U16, close, inputs, run_backward, run_forward, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lq", [1, 300])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
def test_offsets_past_32_bits(lq, layout):
    """Keys and values whose tokens, or whose heads, lie gigabytes apart in one buffer; their gradients as well."""
    lk, Hq, Hkv, D = 600, 4, 2, 64
    q, k, v, dout = inputs(lq, lq, lk, Hq, Hkv, D)
    far = torch.empty(600 * 2 ** 22, dtype=torch.bfloat16, device=DEV)               # 5 GB
    ts, hs = (2 ** 22, 64) if layout == "tokens" else (64, 2 ** 31)
    far_k, far_v, dk, dv = (far.as_strided((lk, Hkv, D), (ts, hs, 1), at) for at in (0, 2 ** 21, 2 ** 20, 3 * 2 ** 20))
    far_k.copy_(k)
    far_v.copy_(v)
    out, lse, _ = run_forward(q, far_k, far_v)
    want = run_forward(q, k, v)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    w_out, _, e_out, _, _ = ref.forward(q, k, v)
    close(out, w_out, e_out + U16 * (w_out.abs() + e_out))
    dq = torch.empty_like(q)
    F.fp8_attention_bwd(dout, q, far_k, far_v, out, lse, dq, dk, dv, workspace(F.fp8_attention_bwd_workspace_bytes, q, k, 1))
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), run_backward(dout, q, k, v, out, lse)))
    assert torch.equal(far_k, k) and torch.equal(far_v, v)


def test_queries_far_apart():
    lq, Hq, Hkv, D = 600, 4, 2, 64
    q, k, v, dout = inputs(2, lq, lq, Hq, Hkv, D)
    far = torch.empty(600 * 2 ** 22, dtype=torch.bfloat16, device=DEV)
    far_q, far_do, far_o, far_dq = (far.as_strided((lq, Hq, D), (2 ** 22, 64, 1), i * 2 ** 20) for i in range(4))
    far_q.copy_(q)
    far_do.copy_(dout)
    out, lse, _ = run_forward(q, k, v)
    lse2 = torch.empty_like(lse)
    F.fp8_attention_fwd(far_q, k, v, far_o, lse2)
    assert torch.equal(out, far_o) and torch.equal(lse, lse2)
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    F.fp8_attention_bwd(far_do, far_q, k, v, far_o, lse, far_dq, dk, dv, workspace(F.fp8_attention_bwd_workspace_bytes, q, k, 1))
    assert all(torch.equal(a, b) for a, b in zip((far_dq, dk, dv), run_backward(dout, q, k, v, out, lse)))


def test_two_calls_at_once():
    """Two streams, each with outputs and workspaces of its own, over the same inputs."""
    q, k, v, dout = inputs(3, 1500, 1500, 8, 2, 128)
    x = torch.randn(5000, 96, device=DEV)

    def buffers():
        b = dict(out=torch.empty_like(q), lse=torch.empty(8, 1500, device=DEV), out8=torch.empty(1500, 1024, dtype=torch.uint8, device=DEV),
                 amax=torch.zeros(1, device=DEV), dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v))
        b.update(ex=torch.empty(5000, 4, dtype=torch.int32, device=DEV), we=torch.empty(5000, 4, device=DEV), le=torch.empty(5000, device=DEV),
                 cnt=torch.empty(97, dtype=torch.int32, device=DEV), sums=torch.empty(96, device=DEV), loss=torch.empty(1, device=DEV),
                 d=torch.empty_like(x))
        ws = workspace(F.fp8_attention_workspace_bytes, q, k, 1), workspace(F.fp8_attention_bwd_workspace_bytes, q, k, 1), \
            torch.empty(F.fp8_moe_route_workspace_bytes(5000, 96), dtype=torch.uint8, device=DEV)
        return b, ws

    s = torch.full((1,), 60.0, device=DEV)

    def step(both, stream):
        b, (w1, w2, w3) = both
        F.fp8_attention_fwd(q, k, v, b["out"], b["lse"], out8=b["out8"], scale=s, amax_slot=b["amax"], workspace=w1, stream=stream)
        F.fp8_moe_route(x, b["ex"], b["we"], b["le"], b["cnt"], b["sums"], b["loss"], workspace=w3, stream=stream)
        F.fp8_attention_bwd(dout, q, k, v, b["out"], b["lse"], b["dq"], b["dk"], b["dv"], w2, stream=stream)
        F.fp8_moe_route_bwd(x, b["ex"], b["we"], b["le"], b["cnt"], b["we"], b["loss"], b["d"], stream=stream)

    sets, streams = [buffers() for _ in range(3)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    step(sets[2], streams[0])
    torch.cuda.synchronize()
    for _ in range(3):
        for both, stream in zip(sets, streams):
            step(both, stream)
    torch.cuda.synchronize()
    for both in sets[:2]:
        for name, t in both[0].items():
            assert torch.equal(t, sets[2][0][name]), name


def test_no_tokens_on_one_side():
    q, k, v, dout = inputs(4, 5, 70, 4, 2, 64)
    none_q, none_k = q[:0], k[:0]
    lse = torch.empty(4, 0, device=DEV)
    dq, dk, dv = run_backward(none_q, none_q, k, v, none_q, lse)
    assert dq.numel() == 0 and bool((dk == 0).all()) and bool((dv == 0).all())
    out, lse, f = run_forward(q, none_k, none_k, fp8=True)
    assert bool((out == 0).all()) and bool((lse == -torch.inf).all()) and bool((f["out8"] == 0).all()) and f["amax_slot"].item() == 0
    dq, dk, dv = run_backward(dout, q, none_k, none_k, out, lse)
    assert bool((dq == 0).all()) and dk.numel() == 0
    out, lse, _ = run_forward(none_q, k, v)
    assert out.numel() == 0


@pytest.mark.parametrize("heads", [8, 40, 200])
@pytest.mark.parametrize("largest", [0, 5, -1])
def test_amax_among_many_candidates(heads, largest):
    """One head's outputs are the largest, all others' within 1/64 of it: of more candidates than are computed again, and
    of more than are listed at a time, the largest is taken.  With equal scores every output is its head's value."""
    q = torch.zeros(256, heads, 64, device=DEV).bfloat16()
    v = torch.full((256, heads, 64), 1 - 3 * 2.0 ** -8, device=DEV).bfloat16()
    v[:, largest] = 1.0
    f = run_forward(q, q, v, fp8=True, causal=False)[2]
    assert abs(f["amax_slot"].item() - 1.0) <= 256 * 2.0 ** -24


def test_one_expert_twice():
    """Choices that were changed afterwards: an expert named twice takes both choices' gradients."""
    T, E = 50, 20
    x = torch.randn(T, E, device=DEV)
    p = torch.softmax(x.double(), 1)
    at = torch.randint(0, E, (T, 3), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    at[:, 2] = at[:, 0]
    w, dw = torch.gather(p, 1, at), torch.randn(T, 3, device=DEV)
    got = torch.empty_like(x)
    counts = torch.ones(E + 1, dtype=torch.int32, device=DEV)
    F.fp8_moe_route_bwd(x, at.int(), w.float(), torch.logsumexp(x.double(), 1).float(), counts, dw, None, got, normalise=False)
    part = w * dw.double()
    want = -p * part.sum(1, keepdim=True)
    want.scatter_add_(1, at, part)
    mag = p * part.abs().sum(1, keepdim=True)
    mag.scatter_add_(1, at, part.abs())
    # p: the float32 lse and the exponential of a difference of numbers below 16, three roundings of at most 2^-21 each; sums of 23 terms
    assert bool(((got.double() - want).abs() <= mag * (3 * 16 * 2.0 ** -23 + 26 * 2.0 ** -24)).all())


@pytest.mark.parametrize("lq,lk", [(1, 300), (1, 6000), (4, 4000), (200, 300), (200, 6000)])
def test_a_row_that_is_not_a_number(lq, lk):
    """A query of NaNs gives NaNs, also where its keys are shared among waves or blocks, and no other row does."""
    q, k, v, dout = inputs(6, 2 * lq, 2 * lk, 4, 2, 64)
    want = run_forward(q, k, v, batch=2)
    q[0, 1] = torch.nan
    out, lse, _ = run_forward(q, k, v, batch=2)
    assert bool(out[0, 1].isnan().all()) and bool(lse[1, 0].isnan())
    out[0, 1], lse[1, 0] = want[0][0, 1], want[1][1, 0]
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    f = run_forward(q, k, v, batch=2, fp8=True)[2]
    assert bool((f["out8"].view(q.shape)[0, 1] == 0x7F).all()) and f["amax_slot"].isnan().all()
