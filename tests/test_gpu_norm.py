"""The block norms (fp8_norm_residual_fwd / _bwd) against their 64-bit forms: both kinds of norm,
widths on both sides of every thread layout, odd widths, every gate layout, the parts left out,
rows of zeros and of special values, captured graphs, another stream, buffers past 2^31 elements."""
import itertools

import numpy as np
import pytest
import torch

import block_ref as R
import fp8_delayed_scaling_amd as F
import oracle
from helpers import DEV, to_f64, u8_host

pytestmark = pytest.mark.gpu

BF = dict(device=DEV, dtype=torch.bfloat16)
F32 = dict(device=DEV, dtype=torch.float32)
U8 = dict(device=DEV, dtype=torch.uint8)
EPS = 1e-5


def _rand(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *shape, sd=1.0, mean=0.0: (torch.randn(*shape, generator=g) * sd + mean).to(torch.bfloat16).to(DEV)


def _f64(t):
    return None if t is None else to_f64(t)


def _inputs(M, H, kind, G, seed):
    r = _rand(seed)
    ln = kind == F.NORM_LAYER
    return dict(o=r(M, H, sd=0.7, mean=0.3), resid=r(M, H, sd=1.5), w_post=r(H, sd=0.2, mean=0.6),
                w_pre=r(H, sd=0.2, mean=1.0), b_post=r(H, sd=0.2) if ln else None, b_pre=r(H, sd=0.2) if ln else None,
                gate=r(G, H, sd=0.5, mean=0.2) if G else None)


def _close(got, ref, err, half=0.0, name=""):
    ref = np.asarray(ref)
    bound = err + half * (np.abs(ref) + err)
    bad = np.abs(got - ref) > bound
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{name}{i}: got {got[i]} want {ref[i]} bound {np.broadcast_to(bound, ref.shape)[i]}")


def _check_codes(codes, h, err, scale, fmt):
    half, sub = (R.E4M3_HALF, R.E4M3_SUB) if fmt == F.E4M3 else (R.E5M2_HALF, R.E5M2_SUB)
    y = np.clip(h * scale, -oracle.fp8_max(fmt), oracle.fp8_max(fmt))
    e = (err + R.U * np.abs(h)) * scale
    _close(oracle.decode(codes, fmt).reshape(y.shape).astype(np.float64), y, e + sub, half, "codes")


def _forward(p, kind, alpha, scale=None, fmt=F.E4M3, want_h=True, x=None, stream=None):
    M, H = p["o"].shape
    n = 2 if kind == F.NORM_LAYER else 1
    out = dict(x=torch.full((M, H), float("nan"), **BF) if x is None else x, post=torch.full((n, M), float("nan"), **F32),
               pre=torch.full((n, M), float("nan"), **F32), h=torch.full((M, H), float("nan"), **BF) if want_h else None,
               h8=torch.full((M, H), 0x55, **U8) if scale is not None else None, amax=torch.zeros(1, **F32),
               sinv=torch.zeros(1, **F32))
    sc = torch.tensor([scale], **F32) if scale is not None else None
    F.fp8_norm_residual_fwd(p["o"], p["w_post"], p["b_post"], p["gate"], p["resid"], alpha, out["x"], out["post"],
                            p["w_pre"], p["b_pre"], out["pre"], out["h"], out["h8"], sc, fmt,
                            out["sinv"] if scale is not None else None, out["amax"] if scale is not None else None,
                            kind=kind, eps=EPS, stream=stream)
    return out


def _check_forward(p, out, kind, alpha, scale=None, fmt=F.E4M3):
    ln = kind == F.NORM_LAYER
    x, rstd, mean, err = R.after_block(_f64(p["o"]), _f64(p["w_post"]), _f64(p["b_post"]), _f64(p["gate"]),
                                       _f64(p["resid"]), alpha, ln, EPS)
    _close(to_f64(out["x"]), x, err, R.BF16, "x")
    h, r2, m2, herr = R.norm(to_f64(out["x"]), _f64(p["w_pre"]), _f64(p["b_pre"]), ln, EPS)
    for got, r, m in ((out["post"], rstd, mean), (out["pre"], r2, m2)):
        g = to_f64(got)
        # the mean of values of size a is off by STEPS U a; the deviation carries that too
        _close(g[0], r, R.STEPS * R.U * np.abs(r) * (1 + (np.abs(m) * r if ln else 0)), 0.0, "rstd")
        if ln:
            _close(g[1], m, R.STEPS * R.U * (np.abs(m) + 1.0 / r), 0.0, "mean")
    if out["h"] is not None:
        _close(to_f64(out["h"]), h, herr, R.BF16, "h")
    if scale is not None:
        _check_codes(u8_host(out["h8"]), h, herr, scale, fmt)
        assert abs(out["amax"].item() - np.abs(h).max()) <= herr.max()
        assert out["sinv"].item() == np.float32(1.0) / np.float32(scale)


WIDTHS = [1, 7, 8, 64, 129, 504, 512, 513, 520, 1000, 1001, 1024, 1032, 2048, 2056, 2304, 4096, 4097, 4104, 8192, 8200, 12288,
          12291, 16376, 16383, 16384]


@pytest.mark.parametrize("kind", [F.NORM_RMS, F.NORM_LAYER])
@pytest.mark.parametrize("H", WIDTHS)
def test_forward_widths(kind, H):
    print(f"norm fwd kind={kind} width={H}", flush=True)
    for M, G, scale, fmt in ((1, 0, 64.0, F.E4M3), (6, 2, 63.3, F.E5M2), (13, 1, None, F.E4M3)):
        p = _inputs(M, H, kind, G, 7 * H + M)
        out = _forward(p, kind, 0.875, scale, fmt)
        _check_forward(p, out, kind, 0.875, scale, fmt)


@pytest.mark.parametrize("kind", [F.NORM_RMS, F.NORM_LAYER])
def test_forward_many_rows(kind):
    """More rows than a grid holds teams, a gate per row, codes without bfloat16 h."""
    for M, H in ((9000, 264), (2500, 2112), (2100, 4608)):
        print(f"norm fwd kind={kind} {M}x{H}", flush=True)
        p = _inputs(M, H, kind, M, 3)
        out = _forward(p, kind, -1.25, 30.0, want_h=False)
        _check_forward(p, out, kind, -1.25, 30.0)


@pytest.mark.parametrize("kind", [F.NORM_RMS, F.NORM_LAYER])
@pytest.mark.parametrize("H", [96, 2048, 2051])
def test_forward_parts_left_out(kind, H):
    print(f"norm fwd parts kind={kind} width={H}", flush=True)
    M = 5
    for drop in (("w_post", "b_post"), ("gate",), ("resid",), ("b_post", "b_pre"), ("w_post", "b_post", "gate", "resid")):
        p = _inputs(M, H, kind, 5, H)
        for d in drop:
            p[d] = None
        out = dict(x=torch.empty(M, H, **BF), h=torch.empty(M, H, **BF))
        F.fp8_norm_residual_fwd(p["o"], p["w_post"], p["b_post"], p["gate"], p["resid"], 0.5, out["x"], None, p["w_pre"],
                                p["b_pre"], None, out["h"], kind=kind, eps=EPS)
        ln = kind == F.NORM_LAYER
        x, _, _, err = R.after_block(_f64(p["o"]), _f64(p["w_post"]), _f64(p["b_post"]), _f64(p["gate"]), _f64(p["resid"]),
                                     0.5, ln, EPS)
        _close(to_f64(out["x"]), x, err, R.BF16, "x")
        h, _, _, herr = R.norm(to_f64(out["x"]), _f64(p["w_pre"]), _f64(p["b_pre"]), ln, EPS)
        _close(to_f64(out["h"]), h, herr, R.BF16, "h")
    # the first norm of a model (no block before it), and the last block (no norm after it)
    p = _inputs(M, H, kind, 0, H + 1)
    h = torch.empty(M, H, **BF)
    F.fp8_norm_residual_fwd(None, None, None, None, p["resid"], 3.0, None, None, p["w_pre"], p["b_pre"], None, h, kind=kind,
                            eps=EPS)
    want, _, _, err = R.norm(to_f64(p["resid"]), _f64(p["w_pre"]), _f64(p["b_pre"]), kind == F.NORM_LAYER, EPS)
    _close(to_f64(h), want, err, R.BF16, "first h")
    x = torch.empty(M, H, **BF)
    F.fp8_norm_residual_fwd(p["o"], p["w_post"], p["b_post"], None, p["resid"], 2.0, x, None, None, None, None, None,
                            kind=kind, eps=EPS)
    want, _, _, err = R.after_block(_f64(p["o"]), _f64(p["w_post"]), _f64(p["b_post"]), None, _f64(p["resid"]), 2.0,
                                    kind == F.NORM_LAYER, EPS)
    _close(to_f64(x), want, err, R.BF16, "last x")


@pytest.mark.parametrize("H", [512, 4096, 1003])
def test_forward_in_place_and_empty(H):
    print(f"norm fwd in place width={H}", flush=True)
    p = _inputs(9, H, F.NORM_RMS, 1, 5)
    want = _forward(p, F.NORM_RMS, 0.9, 50.0)
    p2 = dict(p, resid=p["resid"].clone())
    got = _forward(p2, F.NORM_RMS, 0.9, 50.0, x=p2["resid"])
    for n in ("x", "h", "h8", "post", "pre", "amax"):
        assert torch.equal(got[n], want[n]), n
    e = torch.empty(0, H, **BF)
    F.fp8_norm_residual_fwd(e, p["w_post"], None, None, e, 1.0, e, None, p["w_pre"], None, None, e)


@pytest.mark.parametrize("kind", [F.NORM_RMS, F.NORM_LAYER])
def test_forward_special_rows(kind):
    """Rows of zeros give the bias, rows with a NaN or an infinity do not touch other rows, tiny and
    huge rows stay finite where the formula is."""
    H = 1024
    print(f"norm fwd special rows kind={kind}", flush=True)
    p = _inputs(8, H, kind, 0, 11)
    for t in (p["o"], p["resid"]):
        t[1] = 0.0
        t[3] = t[3] * 2.0 ** -60
        t[5] = t[5] * 2.0 ** 40
    clean = _forward(p, kind, 1.0, 20.0)
    _check_forward(p, clean, kind, 1.0, 20.0)
    p["o"][6, 17] = float("nan")
    p["o"][2, 5] = float("inf")
    out = _forward(p, kind, 1.0, 20.0)
    keep = [0, 1, 3, 4, 5, 7]
    for n in ("x", "h", "h8"):
        assert torch.equal(out[n][keep], clean[n][keep]), n
    assert torch.isnan(out["h"][6]).all() and (out["h8"][6] == 0x7F).all()
    assert np.isnan(out["amax"].item())


def test_forward_amax_folds_and_equals_separate_codes_range():
    p = _inputs(4, 256, F.NORM_RMS, 0, 2)
    out = dict(x=torch.empty(4, 256, **BF), h8=torch.empty(4, 256, **U8), amax=torch.full((1,), 1e6, **F32))
    F.fp8_norm_residual_fwd(p["o"], p["w_post"], None, None, p["resid"], 1.0, out["x"], None, p["w_pre"], None, None, None,
                            out["h8"], torch.ones(1, **F32), F.E4M3, None, out["amax"])
    assert out["amax"].item() == 1e6      # a larger value already in the slot stays


def _bwd_buffers(M, H, kind, G):
    ln = kind == F.NORM_LAYER
    nan = lambda *s: torch.full(s, float("nan"), **F32)  # noqa: E731
    return dict(d_block=torch.full((M, H), float("nan"), **BF), d_resid=torch.full((M, H), float("nan"), **BF),
                dw_post=nan(H), db_post=nan(H) if ln else None, dgate=nan(G, H) if G else None, dw_pre=nan(H),
                db_pre=nan(H) if ln else None,
                ws=torch.full((F.fp8_norm_residual_workspace_bytes(M, H, G),), 0xA5, **U8))


def _backward(p, out, b, dh, dx, kind, alpha, stream=None):
    F.fp8_norm_residual_bwd(dh, dx, p["o"], p["w_post"], p["b_post"], p["gate"], alpha, out["x"], out["post"], p["w_pre"],
                            out["pre"], b["d_block"], b["d_resid"], b["dw_post"], b["db_post"], b["dgate"], b["dw_pre"],
                            b["db_pre"], b["ws"], kind=kind, stream=stream)


def _check_backward(p, out, b, dh, dx, kind, alpha):
    ln = kind == F.NORM_LAYER
    two = lambda t: (to_f64(t)[0], to_f64(t)[1] if ln else np.zeros(t.shape[1]))  # noqa: E731
    ref = R.backward(_f64(dh), _f64(dx), _f64(p["o"]), _f64(p["w_post"]), _f64(p["b_post"]), _f64(p["gate"]), alpha,
                     to_f64(out["x"]), two(out["post"]), _f64(p["w_pre"]), two(out["pre"]), ln)
    for n, (want, err) in ref.items():
        if b.get(n) is not None:
            _close(to_f64(b[n]), want, err, R.BF16 if b[n].dtype == torch.bfloat16 else R.U, n)


@pytest.mark.parametrize("kind", [F.NORM_RMS, F.NORM_LAYER])
@pytest.mark.parametrize("H", WIDTHS)
def test_backward_widths(kind, H):
    print(f"norm bwd kind={kind} width={H}", flush=True)
    for M, G in ((1, 1), (6, 3), (7, 0), (40, 1)):
        p = _inputs(M, H, kind, G, 5 * H + M)
        out = _forward(p, kind, 0.75)
        r = _rand(H + 1)
        dh, dx = r(M, H, sd=0.1), r(M, H, sd=0.1)
        b = _bwd_buffers(M, H, kind, G)
        _backward(p, out, b, dh, dx, kind, 0.75)
        _check_backward(p, out, b, dh, dx, kind, 0.75)


@pytest.mark.parametrize("kind", [F.NORM_RMS, F.NORM_LAYER])
@pytest.mark.parametrize("shape", [(1540, 520, 1), (1540, 520, 7), (1540, 520, 1540), (1540, 520, 770), (600, 2056, 2), (1100, 264, 0)])
def test_backward_units(kind, shape):
    """Row counts that give blocks several rows, gates of one unit, of several, and of one row."""
    M, H, G = shape
    print(f"norm bwd kind={kind} {shape}", flush=True)
    p = _inputs(M, H, kind, G, 17)
    out = _forward(p, kind, 1.5)
    r = _rand(4)
    dh, dx = r(M, H, sd=0.1), r(M, H, sd=0.1)
    b = _bwd_buffers(M, H, kind, G)
    _backward(p, out, b, dh, dx, kind, 1.5)
    _check_backward(p, out, b, dh, dx, kind, 1.5)
    again = _bwd_buffers(M, H, kind, G)
    _backward(p, out, again, dh, dx, kind, 1.5)
    for n in b:
        if n != "ws" and b[n] is not None:
            assert torch.equal(b[n], again[n]), f"{n} differs between two runs"


@pytest.mark.parametrize("kind", [F.NORM_RMS, F.NORM_LAYER])
def test_backward_parts_left_out(kind):
    M, H = 11, 776
    ln = kind == F.NORM_LAYER
    for no_dh, no_dx, no_post, no_gate in itertools.product((0, 1), (0, 1), (0, 1), (0, 1)):
        if no_dh and no_dx:
            continue
        print(f"norm bwd parts kind={kind} {no_dh}{no_dx}{no_post}{no_gate}", flush=True)
        p = _inputs(M, H, kind, 0 if no_gate else 11, 23)
        if no_post:
            p["w_post"] = p["b_post"] = None
        out = _forward(p, kind, 0.5)
        if no_post:
            out["post"] = torch.ones(2 if ln else 1, M, **F32)
        r = _rand(5)
        dh, dx = None if no_dh else r(M, H), None if no_dx else r(M, H)
        b = _bwd_buffers(M, H, kind, 0 if no_gate else 11)
        if no_dh:
            b["dw_pre"] = b["db_pre"] = None
        if no_post:
            b["dw_post"] = b["db_post"] = None
        F.fp8_norm_residual_bwd(dh, dx, p["o"], p["w_post"], p["b_post"], p["gate"], 0.5, None if no_dh else out["x"],
                                None if no_post else out["post"], None if no_dh else p["w_pre"],
                                None if no_dh else out["pre"], b["d_block"], b["d_resid"], b["dw_post"], b["db_post"],
                                b["dgate"], b["dw_pre"], b["db_pre"], b["ws"], kind=kind)
        _check_backward(p, out, b, dh, dx, kind, 0.5)
    # the norm alone: x is the first norm's input
    p = _inputs(M, H, kind, 0, 29)
    n = 2 if ln else 1
    h, pre = torch.empty(M, H, **BF), torch.empty(n, M, **F32)
    F.fp8_norm_residual_fwd(None, None, None, None, p["resid"], 1.0, None, None, p["w_pre"], p["b_pre"], pre, h, kind=kind,
                            eps=EPS)
    dh = _rand(6)(M, H)
    b = _bwd_buffers(M, H, kind, 0)
    F.fp8_norm_residual_bwd(dh, None, None, None, None, None, 9.0, p["resid"], None, p["w_pre"], pre, None, b["d_resid"],
                            None, None, None, b["dw_pre"], b["db_pre"], b["ws"], kind=kind)
    two = (to_f64(pre)[0], to_f64(pre)[1] if ln else np.zeros(M))
    ref = R.backward(to_f64(dh), None, None, None, None, None, 1.0, to_f64(p["resid"]), None, _f64(p["w_pre"]), two, ln)
    for nm in ("d_resid", "dw_pre") + (("db_pre",) if ln else ()):
        _close(to_f64(b[nm]), *ref[nm], R.BF16 if nm == "d_resid" else R.U, nm)


def test_backward_of_no_rows_gives_zero_sums():
    print("norm bwd of no rows", flush=True)
    H = 264
    e = torch.empty(0, H, **BF)
    w = torch.ones(H, **BF)
    gate = torch.ones(3, H, **BF)
    out = [torch.full((H,), 7.0, **F32) for _ in range(4)] + [torch.full((3, H), 7.0, **F32)]
    st = torch.empty(0, **F32)
    F.fp8_norm_residual_bwd(e, e, e, w, w, gate, 1.0, e, st, w, st, e, e, out[0], out[1], out[4], out[2], out[3], None,
                            kind=F.NORM_LAYER)
    assert all((t == 0).all() for t in out)


@pytest.mark.parametrize("kind", [F.NORM_RMS, F.NORM_LAYER])
def test_gradient_against_differences(kind):
    """d_block and d_resid against central differences of the 64-bit forward along random
    directions; a difference's own error is of the order of the step squared."""
    M, H, G, alpha = 3, 40, 3, 0.8
    print(f"norm differences kind={kind}", flush=True)
    ln = kind == F.NORM_LAYER
    p = _inputs(M, H, kind, G, 31)
    out = _forward(p, kind, alpha)
    r = _rand(8)
    dh, dx = r(M, H), r(M, H)
    b = _bwd_buffers(M, H, kind, G)
    _backward(p, out, b, dh, dx, kind, alpha)
    v = {n: _f64(t) for n, t in p.items()}
    rng = np.random.default_rng(3)

    def value(q):
        x, _, _, _ = R.after_block(q["o"], q["w_post"], q["b_post"], q["gate"], q["resid"], alpha, ln, EPS)
        h, _, _, _ = R.norm(x, q["w_pre"], q["b_pre"], ln, EPS)
        return (h * to_f64(dh)).sum() + (x * to_f64(dx)).sum()

    names = {"o": "d_block", "resid": "d_resid", "w_post": "dw_post", "w_pre": "dw_pre", "gate": "dgate"}
    if ln:
        names.update(b_post="db_post", b_pre="db_pre")
    for n, g in names.items():
        u = rng.standard_normal(v[n].shape)
        t = 1e-5
        diff = (value(dict(v, **{n: v[n] + t * u})) - value(dict(v, **{n: v[n] - t * u}))) / (2 * t)
        got = (to_f64(b[g]) * u).sum()
        # every element of the gradient is off by a bfloat16 rounding, and x in the backward by one of its own
        size = np.sqrt(((np.abs(to_f64(b[g])) * np.abs(u)) ** 2).sum())
        assert abs(got - diff) <= 8 * 2.0 ** -8 * size + 1e-6 * abs(diff), (n, got, diff, size)


def test_captured_graph_replays_and_other_stream():
    M, H, kind = 300, 2048, F.NORM_LAYER
    print("norm graph", flush=True)
    p = _inputs(M, H, kind, 3, 41)
    r = _rand(9)
    dh, dx = r(M, H), r(M, H)
    want = _forward(p, kind, 0.9, 40.0)
    wb = _bwd_buffers(M, H, kind, 3)
    _backward(p, want, wb, dh, dx, kind, 0.9)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _forward(p, kind, 0.9, 40.0, stream=side)
    side.synchronize()
    assert torch.equal(got["h8"], want["h8"]) and torch.equal(got["h"], want["h"])
    gb = _bwd_buffers(M, H, kind, 3)
    sc = torch.tensor([40.0], **F32)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    cap = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=cap):
        F.fp8_norm_residual_fwd(p["o"], p["w_post"], p["b_post"], p["gate"], p["resid"], 0.9, got["x"], got["post"],
                                p["w_pre"], p["b_pre"], got["pre"], got["h"], got["h8"], sc, F.E4M3, got["sinv"], got["amax"],
                                kind=kind, eps=EPS)
        _backward(p, got, gb, dh, dx, kind, 0.9)
    for k in range(3):
        for t in (got["x"], got["h"], gb["d_block"], gb["d_resid"], gb["dgate"], gb["dw_post"]):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for n in ("x", "h", "h8", "post", "pre"):
            assert torch.equal(got[n], want[n]), (k, n)
        for n in wb:
            if n != "ws" and wb[n] is not None:
                assert torch.equal(gb[n], wb[n]), (k, n)


def test_rows_past_2_31_elements():
    M, H = 131080, 16384                      # 2^31 + 131072 elements
    print(f"norm {M}x{H}", flush=True)
    o = torch.zeros(M, H, **BF)
    last = _rand(1)(4, H)
    o[-4:] = last
    w = torch.ones(H, **BF)
    x = torch.empty(M, H, **BF)
    h8 = torch.empty(M, H, **U8)
    F.fp8_norm_residual_fwd(o, w, None, None, None, 1.0, x, None, w, None, None, None, h8, torch.full((1,), 32.0, **F32))
    want, _, _, err = R.norm(to_f64(last), np.ones(H), None, False, EPS)
    _close(to_f64(x[-4:]), want, err, R.BF16, "x")
    assert (x[:2] == 0).all() and (h8[:2] == 0).all()
    h, _, _, herr = R.norm(to_f64(x[-4:]), np.ones(H), None, False, EPS)
    _check_codes(u8_host(h8[-4:]), h, herr, 32.0, F.E4M3)
