"""The example block of experts: every operator around the linear layer in one training step, against
automatic differentiation of the same block in float32.

The tolerance counts the FP8 roundings.  A code is off by at most half a step, 2^-4 (E4M3) or 2^-3
(E5M2) of its value, evenly spread: 0.036 and 0.072 in the root of the mean square.  Independent
errors add in squares along the longest path: u 0.051 (two operands), relu(u)^2 twice that, its own
cast, W2: y 0.114; through the gradients' two E5M2 casts at most 0.13.  Twice that bounds the
relative error of each result's norm here.  The scales are settled on the step's own inputs first:
delayed scales of other inputs saturate the values past the amaxes that they were made of."""
import importlib.util
import os

import pytest
import torch

import fp8_delayed_scaling_amd as F

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_block.py")
    spec = importlib.util.spec_from_file_location("expert_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _norm(v):
    return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-5)


def _reference(b, o, resid, choice, weights, dx, dy):
    T, H, N, E, top = b.shape
    leaf = lambda t: t.float().clone().requires_grad_()  # noqa: E731
    o, resid, weights, w1, w2 = leaf(o), leaf(resid), leaf(weights), leaf(b.w1), leaf(b.w2)
    w_post, w_pre, gate = leaf(b.w_post), leaf(b.w_pre), leaf(b.gate)
    x = resid + gate * _norm(o) * w_post
    h = _norm(x) * w_pre
    y = torch.zeros_like(h)
    for e in range(E):
        for j in range(top):
            t = torch.nonzero(choice[:, j] == e).reshape(-1)
            if t.numel():
                out = torch.relu(h[t] @ w1[e].t()).square() @ w2[e].t()
                y = y.index_add(0, t, out * weights[t, j, None])
    torch.autograd.backward([x, y], [dx.float(), dy.float()])
    return dict(x=x, y=y, d_o=o.grad, d_resid=resid.grad, dweights=weights.grad, dw1=w1.grad, dw2=w2.grad, dw_post=w_post.grad,
                dw_pre=w_pre.grad, dgate=gate.grad)


@pytest.mark.parametrize("tokens,width,hidden,experts,top", [(300, 256, 192, 6, 2), (1, 128, 64, 4, 3), (700, 512, 384, 20, 4)])
def test_step_against_autograd(tokens, width, hidden, experts, top):
    print(f"expert block tokens={tokens} width={width} experts={experts}", flush=True)
    m = _example()
    b = m.ExpertBlock(tokens, width, hidden, experts, top, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(2)
    bf = dict(device="cuda", dtype=torch.bfloat16)
    o, resid = torch.randn(tokens, width, generator=g, **bf), torch.randn(tokens, width, generator=g, **bf)
    dx, dy = (torch.randn(tokens, width, generator=g, **bf) * 0.01 for _ in range(2))
    best, choice = torch.topk(torch.randn(tokens, experts, device="cuda", generator=g), top, dim=1)
    choice, weights = choice.to(torch.int32), torch.softmax(best, dim=1)
    if tokens > 1:
        choice[::17, 0] = -1                             # dropped choices
    for step in range(3):                                # the same step: its amaxes settle the scales, no value saturates
        x, y = b.forward(o, resid, choice, weights)
        b.backward(dx, dy)
        if step < 2:
            b.update_scales()
    want = _reference(b, o, resid, choice, weights, dx, dy)
    got = dict(x=x, y=y, **{n: getattr(b, n) for n in ("d_o", "d_resid", "dweights", "dw1", "dw2", "dw_post", "dw_pre", "dgate")})
    for name, w in want.items():
        err = (got[name].float() - w.detach()).norm() / w.detach().norm()
        assert err <= 0.26, f"{name}: relative error {err:.3f}"


def test_prepared_calls_repeat_the_operators():
    """prepare() takes the block operators' calls too."""
    s = torch.ones(1, device="cuda")
    bf = dict(device="cuda", dtype=torch.bfloat16)
    o, w, x, h = torch.randn(5, 64, **bf), torch.ones(64, **bf), torch.empty(5, 64, **bf), torch.empty(5, 64, **bf)
    call = F.prepare(F.fp8_norm_residual_fwd, o, w, None, None, None, 1.0, x, None, w, None, None, h, None, s)
    call()
    first = h.clone()
    o.copy_(torch.randn(5, 64, **bf))
    call()
    F.fp8_norm_residual_fwd(o, w, None, None, None, 1.0, x, None, w, None, None, x2 := torch.empty_like(h))
    assert torch.equal(h, x2) and not torch.equal(h, first)
