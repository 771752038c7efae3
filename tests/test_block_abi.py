"""Refusals of the operators around the linear layer, on the CPU: the C entry points reject bad
arguments before any HIP call, the binding rejects mis-sized buffers before it takes a pointer."""
import pytest
import torch

import fp8_delayed_scaling_amd as F

A16 = 1 << 20        # a fake 16-byte aligned address: never dereferenced, validation fails first
u8, f32, bf, i32 = (dict(dtype=t) for t in (torch.uint8, torch.float32, torch.bfloat16, torch.int32))


def _call(name, ok):
    f = getattr(F.lib(), name)

    def call(**kw):
        a = dict(ok, **kw)
        assert set(a) == set(ok)
        return f(*a.values())
    return call


def test_norm_fwd_validation():
    call = _call("fp8_norm_residual_fwd", dict(
        o=A16, w_post=A16, b_post=None, gate=None, n_gates=0, resid=A16, alpha=1.0, x=A16, post=None, w_pre=A16, b_pre=None,
        pre=None, h=A16, h8=None, scale=None, fmt=0, sinv=None, amax=None, kind=0, eps=1e-5, rows=4, width=64, st=None))
    assert call(kind=2) == -4 and call(fmt=3) == -4
    assert call(rows=-1) == -2 and call(width=16385) == -2
    assert call(gate=A16) == -2                               # a gate without its number
    assert call(gate=A16, n_gates=3) == -2                    # 4 rows do not split over 3 gates
    assert call(n_gates=2) == -2
    assert call(eps=-1.0) == -7 and call(eps=float("nan")) == -7 and call(eps=float("inf")) == -7
    assert call(b_pre=A16) == -7 and call(b_post=A16) == -7   # biases belong to layer norms
    assert call(o=None) == -7                                 # without a block no post norm, no x
    assert call(w_pre=None) == -7                             # h without its norm
    assert call(kind=1, w_post=None, b_post=A16) == -7
    assert call(x=None) == -1 and call(h=None) == -1 and call(h8=A16) == -1
    assert call(o=None, w_post=None, x=None, resid=None) == -1
    assert call(x=A16 + 2) == -3 and call(h8=A16 + 8, scale=A16) == -3 and call(post=A16 + 2) == -3
    assert call(scale=A16 + 1, h8=A16) == -3
    assert call(rows=0) == 0 and call(width=0) == 0


def test_norm_bwd_validation():
    need = F.fp8_norm_residual_workspace_bytes(4, 64, 0)
    assert need > 0 and F.fp8_norm_residual_workspace_bytes(0, 64, 0) == 0
    call = _call("fp8_norm_residual_bwd", dict(
        dh=A16, dx=A16, o=A16, w_post=A16, b_post=None, gate=None, n_gates=0, alpha=1.0, x=A16, post=A16, w_pre=A16, pre=A16,
        d_block=A16, d_resid=A16, dw_post=A16, db_post=None, dgate=None, dw_pre=A16, db_pre=None, ws=A16, ws_bytes=need,
        kind=0, rows=4, width=64, st=None))
    assert call(kind=-1) == -4
    assert call(rows=-4) == -2 and call(width=1 << 20) == -2 and call(gate=A16, n_gates=3) == -2
    assert call(db_pre=A16) == -7 and call(db_post=A16) == -7 and call(dgate=A16) == -7
    assert call(dh=None) == -7                                # dw_pre without dh
    assert call(w_post=None) == -7 and call(o=None) == -7
    assert call(dh=None, dw_pre=None, dx=None) == -1
    assert call(x=None) == -1 and call(pre=None) == -1 and call(post=None) == -1 and call(d_block=None) == -1
    assert call(ws=None) == -5 and call(ws_bytes=need - 1) == -5
    assert call(ws=A16 + 4) == -3 and call(dw_pre=A16 + 4) == -3 and call(d_block=A16 + 2) == -3
    assert call(width=0) == 0


def test_moe_plan_validation():
    assert F.fp8_moe_capacity(100, 4, 8, 16) == (400 + 8 * 15) // 16 * 16
    assert F.fp8_moe_capacity(1, 2, 64, 16) == 32 and F.fp8_moe_capacity(0, 2, 64, 16) == 0
    for bad in ((1, 2, 0, 16), (1, 2, 1025, 16), (1, 2, 4, 8), (1, 2, 4, 24), (1, 2, 4, 2048), (1, 0, 4, 16), (-1, 2, 4, 16),
                (1 << 30, 4, 4, 16)):
        with pytest.raises(ValueError):
            F.fp8_moe_capacity(*bad)
    assert F.fp8_moe_workspace_bytes(4096, 1, 64) == 0 and F.fp8_moe_workspace_bytes(4097, 1, 64) == 5 * 64 * 4
    call = _call("fp8_moe_plan", dict(e=A16, T=5000, top=2, E=8, align=16, cap=10112, off=A16, src=A16, slot=A16, ws=A16,
                                      bytes=1 << 20, st=None))
    assert F.fp8_moe_capacity(5000, 2, 8, 16) == 10112
    assert call(cap=10096) == -2 and call(cap=10120) == -2 and call(E=0) == -2 and call(align=8) == -2
    assert call(T=(1 << 31) - 64, top=1, cap=(1 << 31) - 16) == -2     # padded rows past 31 bits
    assert call(e=None) == -1 and call(off=None) == -1 and call(src=None) == -1 and call(slot=None) == -1
    assert call(ws=None) == -5 and call(bytes=16) == -5
    assert call(src=A16 + 2) == -3


def test_moe_sort_validation():
    cast = _call("fp8_moe_sort_cast", dict(x=A16, T=10, src=A16, cap=48, top=2, w=None, scale=A16, fmt=0, out=A16, out_t=A16,
                                           sinv=None, amax=None, width=64, st=None))
    assert cast(fmt=2) == -4
    assert cast(width=72) == -2 and cast(cap=40) == -2 and cast(top=0) == -2 and cast(T=-1) == -2 and cast(T=1 << 31) == -2
    assert cast(x=None) == -1 and cast(src=None) == -1 and cast(out=None) == -1 and cast(scale=None) == -1
    assert cast(out=A16 + 8) == -3 and cast(out_t=A16 + 8) == -3 and cast(src=A16 + 4) == -3 and cast(w=A16 + 2) == -3
    assert cast(cap=0) == 0 and cast(width=0) == 0
    codes = _call("fp8_moe_sort_codes", dict(x=A16, T=10, src=A16, cap=48, top=2, out=A16, out_t=None, width=64, st=None))
    assert codes(width=8) == -2 and codes(out=None) == -1 and codes(x=A16 + 1) == -3 and codes(out_t=A16 + 4) == -3
    rows = _call("fp8_moe_sort_bf16", dict(x=A16, T=10, src=A16, cap=48, top=2, w=None, out=A16, width=64, st=None))
    assert rows(cap=-16) == -2 and rows(out=A16 + 2) == -3 and rows(w=A16 + 1) == -3 and rows(x=None) == -1


def test_moe_back_validation():
    comb = _call("fp8_moe_combine", dict(ys=A16, cap=48, slot=A16, w=None, T=10, top=2, y=A16, width=64, st=None))
    assert comb(width=40) == -2 and comb(top=0) == -2 and comb(cap=-1) == -2
    assert comb(ys=None) == -1 and comb(slot=None) == -1 and comb(y=None) == -1
    assert comb(ys=A16 + 2) == -3 and comb(slot=A16 + 2) == -3 and comb(w=A16 + 2) == -3 and comb(y=A16 + 8) == -3
    assert comb(T=0) == 0
    grad = _call("fp8_moe_weight_grad", dict(dy=A16, ys=A16, cap=48, slot=A16, T=10, top=2, dw=A16, width=64, st=None))
    assert grad(width=63) == -2 and grad(dy=None) == -1 and grad(dw=None) == -1 and grad(dy=A16 + 4) == -3
    assert grad(T=0) == 0


def test_grouped_validation():
    gemm = _call("fp8_grouped_gemm", dict(A=A16, fa=0, sa=A16, lda=64, B=A16, fb=1, sb=A16, ldb=64, stride=64 * 32, off=A16,
                                          E=4, D=A16, ldd=32, dt=0, cap=128, N=32, K=64, st=None))
    assert gemm(fa=2) == -4 and gemm(fb=-1) == -4 and gemm(dt=2) == -4
    assert gemm(K=40) == -2 and gemm(lda=48) == -2 and gemm(ldb=48) == -2 and gemm(ldd=31) == -2 and gemm(cap=-1) == -2
    assert gemm(lda=1 << 23) == -2 and gemm(E=-1) == -2 and gemm(N=1 << 31) == -2 and gemm(stride=-16) == -2
    assert gemm(cap=(1 << 31) - 16, N=(1 << 31) - 1, ldd=(1 << 31) - 1) == -2     # more tiles than a launch numbers
    assert gemm(lda=72) == -3 and gemm(ldb=72) == -3 and gemm(stride=72) == -3
    assert gemm(A=A16 + 8) == -3 and gemm(D=A16 + 1) == -3 and gemm(off=A16 + 2) == -3 and gemm(sa=A16 + 1) == -3
    assert gemm(A=None) == -1 and gemm(B=None) == -1 and gemm(sa=None) == -1 and gemm(off=None) == -1 and gemm(D=None) == -1
    assert gemm(cap=0) == 0 and gemm(N=0) == 0 and gemm(E=0) == 0
    wg = _call("fp8_grouped_wgrad", dict(A=A16, fa=1, sa=A16, lda=128, B=A16, fb=0, sb=A16, ldb=128, off=A16, E=4, D=A16, dt=1,
                                         cap=128, N=32, K=64, st=None))
    assert wg(cap=120) == -2 and wg(lda=112) == -2 and wg(dt=3) == -4 and wg(D=A16 + 2) == -3 and wg(lda=136) == -3
    assert wg(E=1 << 30, N=1 << 20, K=1 << 20) == -2
    assert wg(A=None) == -1 and wg(off=None) == -1 and wg(D=None) == -1
    assert wg(N=0) == 0 and wg(E=0) == 0


def _raises(match, fn, *a, **kw):
    with pytest.raises((ValueError, TypeError), match=match):
        fn(*a, **kw)


def test_norm_binding_checks():
    M, H = 6, 32
    t = lambda *s: torch.zeros(s, **bf)  # noqa: E731
    ok = dict(block_out=t(M, H), w_post=t(H), b_post=None, gate=t(2, H), resid=t(M, H), alpha=1.0, x=t(M, H),
              post_stats=torch.zeros(M, **f32), w_pre=t(H), b_pre=None, pre_stats=torch.zeros(M, **f32), h=t(M, H),
              h8=torch.zeros(M, H, **u8), scale=torch.ones(1, **f32))

    def bad(match, **kw):
        _raises(match, F.fp8_norm_residual_fwd, **dict(ok, **kw))

    bad("w_post", w_post=t(H + 1))
    bad("gate", gate=t(4, H))
    bad("gate", gate=t(H))
    bad("resid", resid=t(M + 1, H))
    bad("x", x=None)
    bad("x", x=t(H, M).t())
    bad("post_stats", post_stats=torch.zeros(M - 1, **f32))
    bad("pre_stats", kind=F.NORM_LAYER, post_stats=torch.zeros(2, M, **f32))      # a layer norm keeps the mean too
    bad("h8", h8=torch.zeros(M, H, **f32))
    bad("scale", scale=torch.ones(1, dtype=torch.float64))
    bad("block_out", block_out=torch.zeros(M, H, **f32))
    bad("resid", block_out=None, resid=None)
    w = torch.zeros(F.fp8_norm_residual_workspace_bytes(M, H, 0), **u8)
    okb = dict(dh=t(M, H), dx=t(M, H), block_out=t(M, H), w_post=t(H), b_post=None, gate=None, alpha=1.0, x=t(M, H),
               post_stats=torch.zeros(M, **f32), w_pre=t(H), pre_stats=torch.zeros(M, **f32), d_block=t(M, H), d_resid=t(M, H),
               dw_post=torch.zeros(H, **f32), db_post=None, dgate=None, dw_pre=torch.zeros(H, **f32), db_pre=None, workspace=w)
    for match, kw in (("dw_post", dict(dw_post=torch.zeros(H + 1, **f32))), ("dw_pre", dict(dw_pre=torch.zeros(H, **bf))),
                      ("d_block", dict(d_block=t(M, H - 1))), ("dx", dict(dx=t(M, H + 1))),
                      ("dgate", dict(gate=t(3, H), dgate=torch.zeros(2, H, **f32))), ("dx", dict(dh=None, dx=None)),
                      ("workspace", dict(workspace=torch.zeros(64, 64, **u8)[:, ::2]))):
        _raises(match, F.fp8_norm_residual_bwd, **dict(okb, **kw))


def test_moe_binding_checks():
    T, k, E, H = 6, 2, 4, 32
    cap = F.fp8_moe_capacity(T, k, E)
    e, off, src, slot = torch.zeros(T, k, **i32), torch.zeros(E + 1, **i32), torch.zeros(cap, **i32), torch.zeros(T, k, **i32)
    _raises("experts", F.fp8_moe_plan, e.long(), E, 16, off, src, slot)
    _raises("experts", F.fp8_moe_plan, e.reshape(-1), E, 16, off, src, slot)
    _raises("offsets", F.fp8_moe_plan, e, E, 16, off[:-1], src, slot)
    _raises("slot", F.fp8_moe_plan, e, E, 16, off, src, slot[:-1])
    x, s = torch.zeros(T, H, **bf), torch.ones(1, **f32)
    out = torch.zeros(cap, H, **u8)
    _raises("out", F.fp8_moe_sort_cast, x, src, k, None, s, 0, out[:-1])
    _raises("out_t", F.fp8_moe_sort_cast, x, src, k, None, s, 0, out, out)
    _raises("weights", F.fp8_moe_sort_cast, x, src, k, torch.zeros(T, k + 1, **f32), s, 0, out)
    _raises("x", F.fp8_moe_sort_cast, x[:, ::2], src, k, None, s, 0, out)
    _raises("x", F.fp8_moe_sort_codes, x, src, k, out)
    _raises("out", F.fp8_moe_sort_bf16, x, src, k, None, out)
    ys, y = torch.zeros(cap, H, **bf), torch.zeros(T, H, **bf)
    _raises("y", F.fp8_moe_combine, ys, slot, None, y[:-1])
    _raises("weights", F.fp8_moe_combine, ys, slot, torch.zeros(T * k, **f32), y)
    _raises("slot", F.fp8_moe_combine, ys, slot.long(), None, y)
    _raises("dy", F.fp8_moe_weight_grad, ys, ys, slot, torch.zeros(T, k, **f32))
    _raises("dweights", F.fp8_moe_weight_grad, y, ys, slot, torch.zeros(T, k, **bf))


def test_grouped_binding_checks():
    E, N, K, cap = 3, 32, 48, 64
    s = torch.ones(1, **f32)
    A, B, off, D = torch.zeros(cap, K, **u8), torch.zeros(E, N, K, **u8), torch.zeros(E + 1, **i32), torch.zeros(cap, N, **bf)
    _raises("share K", F.fp8_grouped_gemm, A[:, :32], 0, s, B, 0, s, off, D)
    _raises("offsets", F.fp8_grouped_gemm, A, 0, s, B, 0, s, off[:-1], D)
    _raises("D", F.fp8_grouped_gemm, A, 0, s, B, 0, s, off, D[:-1])
    _raises("D", F.fp8_grouped_gemm, A, 0, s, B, 0, s, off, torch.zeros(N, cap, **bf).t())
    _raises("B", F.fp8_grouped_gemm, A, 0, s, B.transpose(1, 2).contiguous().transpose(1, 2), 0, s, off, D)
    _raises("D", F.fp8_grouped_gemm, A, 0, s, B, 0, s, off, torch.zeros(cap, N, dtype=torch.float16))
    _raises("share", F.fp8_grouped_wgrad, torch.zeros(N, cap, **u8), 0, s, torch.zeros(K, cap - 16, **u8), 0, s, off,
            torch.zeros(E, N, K, **bf))
    _raises("dW", F.fp8_grouped_wgrad, torch.zeros(N, cap, **u8), 0, s, torch.zeros(K, cap, **u8), 0, s, off,
            torch.zeros(E, K, N, **bf))


def test_host_tensors_are_refused():
    """Tensors that pass every check but are not on the GPU: refused, also by prepare()."""
    M, H, E, T, k = 4, 32, 3, 6, 2
    t = lambda *s: torch.zeros(s, **bf)  # noqa: E731
    norm = (t(M, H), t(H), None, None, t(M, H), 1.0, t(M, H), None, t(H), None, None, t(M, H))
    cap = F.fp8_moe_capacity(T, k, E)
    plan = (torch.zeros(T, k, **i32), E, 16, torch.zeros(E + 1, **i32), torch.zeros(cap, **i32), torch.zeros(T, k, **i32))
    s = torch.ones(1, **f32)
    for fn, args in ((F.fp8_norm_residual_fwd, norm), (F.fp8_moe_plan, plan),
                     (F.fp8_moe_combine, (t(cap, H), torch.zeros(T, k, **i32), None, t(T, H))),
                     (F.fp8_moe_sort_cast, (t(T, H), torch.zeros(cap, **i32), k, None, s, 0, torch.zeros(cap, H, **u8)))):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):      # the stream may be asked for first
            fn(*args)
        with pytest.raises(ValueError, match="on the GPU"):
            fn(*args, stream=0)
        with pytest.raises(ValueError, match="on the GPU"):
            F.prepare(fn, *args, stream=0)


def test_grouped_leading_dimensions():
    gemm = _call("fp8_grouped_gemm", dict(A=A16, fa=0, sa=A16, lda=64, B=A16, fb=1, sb=A16, ldb=64, stride=64 * 32, off=A16,
                                          E=4, D=A16, ldd=1 << 23, dt=0, cap=128, N=32, K=64, st=None))
    assert gemm() == -2
    wg = _call("fp8_grouped_wgrad", dict(A=A16, fa=1, sa=A16, lda=128, B=A16, fb=0, sb=A16, ldb=128, off=A16, E=1, D=A16, dt=1,
                                         cap=128, N=16, K=1 << 23, st=None))
    assert wg() == -2
