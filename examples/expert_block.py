"""A block of experts trained in FP8 with per-tensor delayed scaling: the norms around the residual
stream, tokens sorted by expert, two FP8 products with their gradients, the weighted way back.

    python examples/expert_block.py        # one MI355X: a few steps, the loss and the time of each

    x = resid + gate * norm(o)      h = norm(x), as FP8 codes            fp8_norm_residual_fwd
    hs = h in expert order, and its transpose                            fp8_moe_plan, fp8_moe_sort_codes
    u = hs W1[e]^T      a = relu(u)^2, cast      ys = a W2[e]^T          fp8_grouped_gemm, fp8_cast_transpose
    y[t] = sum_j weights[t, j] ys[slot[t, j]]                            fp8_moe_combine

Every cast collects its amax in row 0 of the history; fp8_scale_update turns it into the next step's
scales.  Nothing is read back to the host: routing, offsets and scales stay on the GPU.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_delayed_scaling_amd as F  # noqa: E402

ALIGN = 16
H_, ACT, W1_, W2_, DY, DU = range(6)          # the scaled tensors
FORMATS = [F.E4M3, F.E4M3, F.E4M3, F.E4M3, F.E5M2, F.E5M2]


class ExpertBlock:
    def __init__(self, tokens, width, hidden, experts, top, history=16, seed=0):
        dev = "cuda"
        g = torch.Generator(device=dev).manual_seed(seed)
        f32, bf, u8 = (dict(device=dev, dtype=t) for t in (torch.float32, torch.bfloat16, torch.uint8))
        i32 = dict(device=dev, dtype=torch.int32)
        self.shape = (tokens, width, hidden, experts, top)
        self.cap = cap = F.fp8_moe_capacity(tokens, top, experts, ALIGN)
        self.w1 = (torch.randn(experts, hidden, width, device=dev, generator=g) * width ** -0.5).bfloat16()
        self.w2 = (torch.randn(experts, width, hidden, device=dev, generator=g) * hidden ** -0.5).bfloat16()
        self.gate = torch.ones(1, width, **bf)
        self.w_post, self.w_pre = torch.ones(width, **bf), torch.ones(width, **bf)
        # delayed scaling: amaxes of the last steps, the scales made of them, the casts' own inverse scales
        self.history, self.scale, self.scale_inv = torch.zeros(history, 6, **f32), torch.ones(6, **f32), torch.ones(6, **f32)
        self.sinv = torch.ones(6, **f32)
        # weights as codes, [E N, K] and transposed [K, E N]
        self.w1_8, self.w1_8t = torch.empty(experts * hidden, width, **u8), torch.empty(width, experts * hidden, **u8)
        self.w2_8, self.w2_8t = torch.empty(experts * width, hidden, **u8), torch.empty(hidden, experts * width, **u8)
        self.offsets, self.src = torch.empty(experts + 1, **i32), torch.empty(cap, **i32)
        self.slot = torch.empty(tokens, top, **i32)
        self.plan_ws = torch.empty(F.fp8_moe_workspace_bytes(tokens, top, experts), **u8)
        self.norm_ws = torch.empty(F.fp8_norm_residual_workspace_bytes(tokens, width, 1), **u8)
        self.x, self.h8 = torch.empty(tokens, width, **bf), torch.empty(tokens, width, **u8)
        self.post, self.pre = torch.empty(tokens, **f32), torch.empty(tokens, **f32)
        self.hs, self.hs_t = torch.empty(cap, width, **u8), torch.empty(width, cap, **u8)
        # rows past the last expert's are never written: they stay zero as long as the routing does not shrink
        self.u, self.ys = torch.zeros(cap, hidden, **bf), torch.zeros(cap, width, **bf)
        self.act8, self.act8_t = torch.empty(cap, hidden, **u8), torch.empty(hidden, cap, **u8)
        self.y = torch.empty(tokens, width, **bf)
        self.dys, self.dys_t = torch.empty(cap, width, **u8), torch.empty(width, cap, **u8)
        self.da, self.dhs = torch.zeros(cap, hidden, **bf), torch.zeros(cap, width, **bf)
        self.du8, self.du8_t = torch.empty(cap, hidden, **u8), torch.empty(hidden, cap, **u8)
        self.dh = torch.empty(tokens, width, **bf)
        self.d_o, self.d_resid = torch.empty(tokens, width, **bf), torch.empty(tokens, width, **bf)
        self.dw1, self.dw2 = torch.empty(experts, hidden, width, **f32), torch.empty(experts, width, hidden, **f32)
        self.dw_post, self.dw_pre, self.dgate = torch.empty(width, **f32), torch.empty(width, **f32), torch.empty(1, width, **f32)
        self.dweights = torch.empty(tokens, top, **f32)

    def _s(self, i):
        """Scale, the cast's inverse scale and the amax slot of scaled tensor i."""
        return self.scale[i:i + 1], self.sinv[i:i + 1], self.history[0, i:i + 1]

    def forward(self, o, resid, choice, weights):
        """o: the block before's output, resid: the residual stream, choice / weights: the router's, [T, top]."""
        T, H, N, E, top = self.shape
        self.o, self.resid, self.weights = o, resid, weights
        for w, i, w8, w8t in ((self.w1, W1_, self.w1_8, self.w1_8t), (self.w2, W2_, self.w2_8, self.w2_8t)):
            s, inv, amax = self._s(i)
            F.fp8_cast_transpose(w.view(-1, w.shape[2]), s, F.E4M3, w8, w8t, inv, amax)
        s, inv, amax = self._s(H_)
        F.fp8_norm_residual_fwd(o, self.w_post, None, self.gate, resid, 1.0, self.x, self.post, self.w_pre, None, self.pre, None,
                                self.h8, s, F.E4M3, inv, amax)
        F.fp8_moe_plan(choice, E, ALIGN, self.offsets, self.src, self.slot, self.plan_ws)
        F.fp8_moe_sort_codes(self.h8, self.src, top, self.hs, self.hs_t)
        self.u.zero_()
        F.fp8_grouped_gemm(self.hs, F.E4M3, self.sinv[H_:], self.w1_8.view(E, N, H), F.E4M3, self.sinv[W1_:], self.offsets, self.u)
        s, inv, amax = self._s(ACT)
        F.fp8_cast_transpose(torch.relu(self.u).square(), s, F.E4M3, self.act8, self.act8_t, inv, amax)
        F.fp8_grouped_gemm(self.act8, F.E4M3, self.sinv[ACT:], self.w2_8.view(E, H, N), F.E4M3, self.sinv[W2_:], self.offsets,
                           self.ys)
        F.fp8_moe_combine(self.ys, self.slot, weights, self.y)
        return self.x, self.y

    def backward(self, dx, dy):
        """dx, dy: gradients of forward's outputs.  Leaves the gradients in d_o, d_resid, dw1, dw2, dw_post,
        dw_pre, dgate and dweights."""
        T, H, N, E, top = self.shape
        s, inv, amax = self._s(DY)
        F.fp8_moe_sort_cast(dy, self.src, top, self.weights, s, F.E5M2, self.dys, self.dys_t, inv, amax)
        F.fp8_moe_weight_grad(dy, self.ys, self.slot, self.dweights)
        w2t = self.w2_8t.view(N, E, H).transpose(0, 1)         # [E, N, H], a view of the cast's transpose
        self.da.zero_()
        F.fp8_grouped_gemm(self.dys, F.E5M2, self.sinv[DY:], w2t, F.E4M3, self.sinv[W2_:], self.offsets, self.da)
        F.fp8_grouped_wgrad(self.dys_t, F.E5M2, self.sinv[DY:], self.act8_t, F.E4M3, self.sinv[ACT:], self.offsets, self.dw2)
        s, inv, amax = self._s(DU)
        F.fp8_cast_transpose(self.da * torch.relu(self.u) * 2, s, F.E5M2, self.du8, self.du8_t, inv, amax)
        w1t = self.w1_8t.view(H, E, N).transpose(0, 1)
        F.fp8_grouped_gemm(self.du8, F.E5M2, self.sinv[DU:], w1t, F.E4M3, self.sinv[W1_:], self.offsets, self.dhs)
        F.fp8_grouped_wgrad(self.du8_t, F.E5M2, self.sinv[DU:], self.hs_t, F.E4M3, self.sinv[H_:], self.offsets, self.dw1)
        F.fp8_moe_combine(self.dhs, self.slot, None, self.dh)
        F.fp8_norm_residual_bwd(self.dh, dx, self.o, self.w_post, None, self.gate, 1.0, self.x, self.post, self.w_pre, self.pre,
                                self.d_o, self.d_resid, self.dw_post, None, self.dgate, self.dw_pre, None, self.norm_ws)

    def update_scales(self):
        F.fp8_scale_update(self.history, self.scale, self.scale_inv, FORMATS)


def main(tokens=8192, width=4096, hidden=2048, experts=64, top=4, steps=6):
    block = ExpertBlock(tokens, width, hidden, experts, top)
    g = torch.Generator(device="cuda").manual_seed(1)
    bf = dict(device="cuda", dtype=torch.bfloat16)
    o, resid = torch.randn(tokens, width, generator=g, **bf), torch.randn(tokens, width, generator=g, **bf)
    target = torch.randn(tokens, width, generator=g, **bf)
    scores = torch.randn(tokens, experts, device="cuda", generator=g)
    best, choice = torch.topk(scores, top, dim=1)
    choice, weights = choice.to(torch.int32), torch.softmax(best, dim=1)
    for step in range(steps):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        x, y = block.forward(o, resid, choice, weights)
        err = (x.float() + y.float() - target.float())
        grad = (err / tokens).bfloat16()
        block.backward(grad, grad)
        with torch.no_grad():
            for w, dw in ((block.w1, block.dw1), (block.w2, block.dw2)):
                w.sub_((dw * (0.03 * w.float().norm() / dw.norm())).bfloat16())      # a fixed part of the weights' size
        block.update_scales()
        end.record()
        torch.cuda.synchronize()
        print(f"step {step}: loss {err.square().mean().item():.4f}, {begin.elapsed_time(end):.2f} ms", flush=True)


if __name__ == "__main__":
    main()
