"""The attention half of a transformer block trained in FP8 with per-tensor delayed scaling.

    python examples/attention_block.py     # one MI355X: a few steps, the time of each

    qkv = x Wqkv^T                 one FP8 linear layer                          fp8_linear_fwd
    a = attention(q, k, v)         slices of qkv; FP8 codes of the output        fp8_attention_fwd
    y = a Wo^T                     reads those codes                             fp8_gemm_bias

The gradients of q, k and v are written as slices of the QKV layer's output gradient, which its backward
reads.  Every cast collects its amax in row 0 of the history; fp8_scale_update turns it into the next
step's scales.  Nothing is read back to the host.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_delayed_scaling_amd as F  # noqa: E402

X_, WQKV, ATT, WO, DY, DQKV = range(6)        # the scaled tensors
FORMATS = [F.E4M3, F.E4M3, F.E4M3, F.E4M3, F.E5M2, F.E5M2]


class AttentionBlock:
    """Sequences of equal lengths, or packed behind each other with ``offsets`` [sequences + 1]; a multiple of 16 tokens."""

    def __init__(self, tokens, width, heads, kv_heads, dim, batch=1, causal=True, window=0, history=16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        f32, bf, u8 = (dict(device="cuda", dtype=t) for t in (torch.float32, torch.bfloat16, torch.uint8))
        self.shape = (tokens, width, heads, kv_heads, dim)
        self.batch, self.mask = batch, dict(causal=causal, window=window)
        out, inner = (heads + 2 * kv_heads) * dim, heads * dim
        new = lambda n, k: (torch.randn(n, k, device="cuda", generator=g) * k ** -0.5).bfloat16()  # noqa: E731
        self.w_qkv, self.w_o = new(out, width), new(width, inner)
        self.history, self.scale, self.scale_inv = torch.zeros(history, 6, **f32), torch.ones(6, **f32), torch.ones(6, **f32)
        self.sinv = torch.ones(6, **f32)
        self.x8, self.x8_t = torch.empty(tokens, width, **u8), torch.empty(width, tokens, **u8)
        self.wqkv8, self.wqkv8_t = torch.empty(out, width, **u8), torch.empty(width, out, **u8)
        self.wo8, self.wo8_t = torch.empty(width, inner, **u8), torch.empty(inner, width, **u8)
        self.qkv, self.dqkv = torch.empty(tokens, heads + 2 * kv_heads, dim, **bf), torch.zeros(tokens, heads + 2 * kv_heads, dim, **bf)
        self.a, self.a8, self.a8_t = torch.zeros(tokens, heads, dim, **bf), torch.zeros(tokens, inner, **u8), torch.empty(inner, tokens, **u8)
        self.lse, self.da = torch.empty(heads, tokens, **f32), torch.empty(tokens, heads, dim, **bf)
        self.y, self.dx = torch.empty(tokens, width, **bf), torch.empty(tokens, width, **bf)
        self.dy8, self.dy8_t = torch.empty(tokens, width, **u8), torch.empty(width, tokens, **u8)
        self.dqkv8, self.dqkv8_t = torch.empty(tokens, out, **u8), torch.empty(out, tokens, **u8)
        self.dw_qkv, self.dw_o = torch.empty(out, width, **f32), torch.empty(width, inner, **f32)
        self.ws = None

    def _s(self, i):
        """Scale, amax slot and the cast's inverse scale of scaled tensor i."""
        return self.scale[i:i + 1], self.history[0, i:i + 1], self.sinv[i:i + 1]

    def _heads(self, t):
        """Queries, keys and values in the QKV layer's output, or in its gradient."""
        _, _, H, kv, _ = self.shape
        return t[:, :H], t[:, H:H + kv], t[:, H + kv:]

    def forward(self, x, offsets=None):
        T, width, H, kv, D = self.shape
        self.offsets, batch = offsets, self.batch if offsets is None else offsets.numel() - 1
        if offsets is not None:                              # rows of no sequence are not written: an earlier batch may have been longer
            self.a8.zero_()
            self.dqkv.zero_()
        size = [F.fp8_attention_workspace_bytes(T, T, batch, H, kv, D), F.fp8_attention_bwd_workspace_bytes(T, T, batch, H, kv, D)]
        if self.ws is None or self.ws.numel() < max(size):
            self.ws = torch.empty(max(size), device="cuda", dtype=torch.uint8)
        s, amax, inv = self._s(X_)
        w_s, w_amax, w_inv = self._s(WQKV)
        F.fp8_linear_fwd(x, self.w_qkv, None, s, amax, self.x8, self.x8_t, inv, w_s, w_amax, self.wqkv8, self.wqkv8_t, w_inv, None,
                         self.qkv.view(T, -1))
        s, amax, inv = self._s(ATT)
        F.fp8_attention_fwd(*self._heads(self.qkv), self.a, self.lse, offsets, offsets, self.batch, **self.mask, out8=self.a8, scale=s,
                            fmt=F.E4M3, scale_inv_out=inv, amax_slot=amax, workspace=self.ws)
        s, amax, inv = self._s(WO)
        F.fp8_cast_transpose(self.w_o, s, F.E4M3, self.wo8, self.wo8_t, inv, amax)
        F.fp8_gemm_bias(self.a8, F.E4M3, self.sinv[ATT:], self.wo8, F.E4M3, self.sinv[WO:], None, self.y)
        return self.y

    def backward(self, dy):
        """dy: the output's gradient.  Leaves the gradients in dx, dw_qkv and dw_o."""
        T, width, H, kv, D = self.shape
        s, amax, inv = self._s(DY)
        F.fp8_transpose(self.a8, self.a8_t)
        F.fp8_linear_bwd(dy, H * D, s, amax, self.dy8, self.dy8_t, inv, None, None, self.a8_t, self.sinv[ATT:], self.wo8_t,
                         self.sinv[WO:], self.da.view(T, -1), self.dw_o)
        F.fp8_attention_bwd(self.da, *self._heads(self.qkv), self.a, self.lse, *self._heads(self.dqkv), self.ws, self.offsets,
                            self.offsets, self.batch, **self.mask)
        s, amax, inv = self._s(DQKV)
        F.fp8_linear_bwd(self.dqkv.view(T, -1), width, s, amax, self.dqkv8, self.dqkv8_t, inv, None, None, self.x8_t, self.sinv[X_:],
                         self.wqkv8_t, self.sinv[WQKV:], self.dx, self.dw_qkv)
        return self.dx

    def update_scales(self):
        F.fp8_scale_update(self.history, self.scale, self.scale_inv, FORMATS)


def main(tokens=8192, width=4096, heads=32, kv_heads=8, dim=128, batch=4, steps=6):
    block = AttentionBlock(tokens, width, heads, kv_heads, dim, batch)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randn(tokens, width, device="cuda", generator=g).bfloat16() for _ in range(2))
    for step in range(steps):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        block.forward(x)
        block.backward(dy)
        block.update_scales()
        end.record()
        torch.cuda.synchronize()
        print(f"step {step}: {begin.elapsed_time(end):.2f} ms", flush=True)


if __name__ == "__main__":
    main()
