"""The operators together, as a block uses them: the attention half of a block against automatic differentiation in
float32, and the router in front of the experts with its gradients.

The tolerances count the FP8 roundings, in the root of the mean square: a code of E4M3 is off by 0.036 of its value, one
of E5M2 by 0.072, and independent errors add in squares along the longest path.  Attention: qkv 0.051 (two operands), so
that a score, of order one, is off by about 0.07 and a probability by as much; a 0.09, y with its cast and Wo 0.10.  Back:
dy and Wo 0.08, ds with the probabilities' and the values' errors 0.13, the cast and Wqkv 0.15, with the recomputed forward
0.18.  Twice that bounds the relative error of each result's norm."""
import importlib.util
import os

import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def example(name):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", name + ".py")
    spec = importlib.util.spec_from_file_location(name, path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def attention(q, k, v, parts, causal, window):
    """Differentiable attention in float32, sequence by sequence."""
    G, rows = q.shape[1] // k.shape[1], []
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    for a, b in parts:
        n = b - a
        see = ref.visible(n, n, causal, window, q.device)
        heads = []
        for h in range(q.shape[1]):
            s = (q[a:b, h] @ k[a:b, h].t()) * q.shape[2] ** -0.5
            heads.append(torch.softmax(s.masked_fill(~see, float("-inf")), 1) @ v[a:b, h])
        rows.append(torch.stack(heads, 1))
    return torch.cat(rows)


@pytest.mark.parametrize("tokens,width,heads,kv,dim,batch,window,lengths", [
    (320, 256, 4, 2, 64, 2, 0, None), (256, 128, 6, 2, 40, 1, 50, None), (240, 256, 4, 4, 128, 1, 0, [100, 1, 90, 49])])
def test_attention_half_against_autograd(tokens, width, heads, kv, dim, batch, window, lengths):
    m = example("attention_block")
    b = m.AttentionBlock(tokens, width, heads, kv, dim, batch, window=window, seed=tokens)
    g = torch.Generator(device=DEV).manual_seed(7)
    x, dy = torch.randn(tokens, width, device=DEV, generator=g).bfloat16(), torch.randn(tokens, width, device=DEV, generator=g).bfloat16() * 0.01
    offsets = None
    if lengths is not None:
        offsets = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device=DEV)
    for step in range(3):                                # the same step: its amaxes settle the scales, no value saturates
        y = b.forward(x, offsets)
        b.backward(dy)
        if step < 2:
            b.update_scales()
    leaf = lambda t: t.float().clone().requires_grad_()  # noqa: E731
    xr, wq, wo = leaf(x), leaf(b.w_qkv), leaf(b.w_o)
    qkv = (xr @ wq.t()).view(tokens, heads + 2 * kv, dim)
    a = attention(qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:], ref.spans(offsets, tokens, batch), True, window)
    want = a.reshape(tokens, -1) @ wo.t()
    want.backward(dy.float())
    assert abs(b.history[0, m.ATT].item() / a.abs().max().item() - 1) < 0.2
    for name, got, w, most in (("y", y, want, 0.2), ("dx", b.dx, xr.grad, 0.36), ("dw_qkv", b.dw_qkv, wq.grad, 0.36), ("dw_o", b.dw_o, wo.grad, 0.26)):
        err = ((got.float() - w.detach()).norm() / w.detach().norm()).item()
        assert err <= most, f"{name}: relative error {err:.3f}"


@pytest.mark.parametrize("tokens,width,hidden,experts,top", [(300, 256, 192, 6, 2), (700, 512, 384, 20, 4)])
def test_router_and_experts_against_autograd(tokens, width, hidden, experts, top):
    """The choice goes into the plan as it is; the weights' gradient of the combine goes back to the router's matrix."""
    m = example("expert_block")
    block, router = m.ExpertBlock(tokens, width, hidden, experts, top, seed=3), m.Router(tokens, width, experts, top, seed=4)
    g = torch.Generator(device=DEV).manual_seed(8)
    o, resid, dx, dy = (torch.randn(tokens, width, device=DEV, generator=g).bfloat16() for _ in range(4))
    dloss = torch.full((1,), 0.5, device=DEV)
    for step in range(3):
        block.forward(o, resid, *router.forward(resid))
        block.backward(dx, dy)
        router.backward(block.dweights, dloss)
        if step < 2:
            block.update_scales()
    # the router on its own, from the same gradient of the weights
    w = router.w.clone().requires_grad_()
    x = resid.float().clone().requires_grad_()
    p = torch.softmax(x @ w.t(), 1)
    at = router.choice.long()
    taken = torch.gather(p, 1, at)
    weights = taken / taken.sum(1, keepdim=True)
    share = torch.bincount(at.flatten(), minlength=experts).float() / at.numel()
    loss = experts * (share * p.mean(0)).sum()
    torch.autograd.backward([weights, loss], [block.dweights, dloss[0]])
    assert torch.equal(router.counts[:-1].long(), torch.bincount(at.flatten(), minlength=experts))
    # float32 on both sides: the products of the two libraries' orders and the exponentials, far below 1e-4 of the norm
    assert abs(loss.item() - router.loss.item()) < 1e-5 * loss.item() and torch.allclose(weights, router.weights, rtol=1e-4, atol=1e-6)
    assert (router.dw - w.grad).norm() < 1e-4 * w.grad.norm() and (router.dx - x.grad).norm() < 1e-4 * x.grad.norm()
    # and the experts' weights' gradient, which it was given
    want = torch.zeros_like(block.dweights)
    rows = torch.where(block.slot >= 0, block.slot, torch.zeros_like(block.slot)).long()
    want = (dy.float()[:, None] * block.ys.float()[rows]).sum(2) * (block.slot >= 0)
    assert (block.dweights - want).norm() < 1e-4 * want.norm()


def test_examples_run():
    example("attention_block").main(tokens=512, width=256, heads=4, kv_heads=2, dim=64, batch=2, steps=2)
    example("expert_block").main(tokens=256, width=256, hidden=128, experts=8, top=2, steps=2)


def test_training_step_in_a_graph():
    """Forward and backward of the attention half in one graph, while the eager one lives; every replay as the eager step."""
    m = example("attention_block")
    b = m.AttentionBlock(256, 128, 4, 2, 64, 2)
    g = torch.Generator(device=DEV).manual_seed(9)
    x, dy = torch.randn(256, 128, device=DEV, generator=g).bfloat16(), torch.randn(256, 128, device=DEV, generator=g).bfloat16() * 0.01
    b.forward(x)
    b.backward(dy)
    b.update_scales()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        b.forward(x)
        b.backward(dy)
    for turn in range(3):
        x.copy_(torch.randn(256, 128, device=DEV, generator=g).bfloat16())
        b.history.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (b.y, b.dx, b.dw_qkv, b.dw_o, b.history)]
        b.history.zero_()
        b.forward(x)
        b.backward(dy)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, (b.y, b.dx, b.dw_qkv, b.dw_o, b.history)))
