"""The experts' FP8 products (fp8_grouped_gemm, fp8_grouped_wgrad): exact where the arithmetic is,
against the float64 product with the GEMM's gate elsewhere; every format pair, ragged experts,
experts without rows, odd sizes, strided operands, bad offsets, graphs."""
import numpy as np
import pytest
import torch

import fp8_delayed_scaling_amd as F
import oracle
from helpers import DEV, gemm_close, to_f64

pytestmark = pytest.mark.gpu

BF = dict(device=DEV, dtype=torch.bfloat16)
F32 = dict(device=DEV, dtype=torch.float32)
U8 = dict(device=DEV, dtype=torch.uint8)
I32 = dict(device=DEV, dtype=torch.int32)


def _codes(rng, shape, fmt, sd):
    return oracle.encode((rng.standard_normal(shape) * sd).astype(np.float32), fmt).reshape(shape)


def _exact_codes(rng, shape, fmt):
    """Codes of 0, +-0.5, +-1, +-2: every float32 partial sum of their products is exact."""
    return oracle.encode(rng.choice(np.float32([0, 0.5, -0.5, 1, -1, 2, -2]), shape), fmt).reshape(shape)


def _offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _scal(v):
    return torch.tensor([v], **F32)


LENS = [[16], [0], [160, 0, 32], [0, 0, 0, 48], [256, 16, 112, 0, 400], [1024, 528], [16] * 70, [0] * 63 + [272] + [0] * 10 + [64, 16]]


def _gemm(A, fa, B, fb, off, cap, dtype, sa=0.5, sb=2.0):
    D = torch.full((cap, B.shape[1]), 7.0, device=DEV, dtype=dtype)
    F.fp8_grouped_gemm(A, fa, _scal(sa), B, fb, _scal(sb), torch.from_numpy(off).to(DEV), D)
    return D


@pytest.mark.parametrize("lens", LENS, ids=lambda v: f"{len(v)}experts{sum(v)}rows")
@pytest.mark.parametrize("N,K", [(16, 16), (130, 144), (256, 256), (384, 400), (72, 1024), (520, 2064)])
def test_gemm_exact(lens, N, K):
    print(f"grouped gemm lens={lens[:5]} N={N} K={K}", flush=True)
    rng = np.random.default_rng(N + K)
    off, E = _offsets(lens), len(lens)
    cap = int(off[-1]) + 48
    A, B = _exact_codes(rng, (cap, K), F.E4M3), _exact_codes(rng, (E, N, K), F.E4M3)
    a, b = oracle.decode(A, 0).astype(np.float64).reshape(A.shape), oracle.decode(B, 0).astype(np.float64).reshape(B.shape)
    At, Bt = torch.from_numpy(A).to(DEV), torch.from_numpy(B).to(DEV)
    for dtype in (torch.float32, torch.bfloat16):
        D = _gemm(At, F.E4M3, Bt, F.E4M3, off, cap, dtype)
        want = np.full((cap, N), 7.0)
        for e in range(E):
            want[off[e]:off[e + 1]] = a[off[e]:off[e + 1]] @ b[e].T
        ref = torch.from_numpy(want).to(dtype)
        assert torch.equal(D.cpu(), ref)


@pytest.mark.parametrize("fa", [F.E4M3, F.E5M2])
@pytest.mark.parametrize("fb", [F.E4M3, F.E5M2])
@pytest.mark.parametrize("N,K", [(640, 1424), (300, 2048), (64, 4096)])
def test_gemm_formats(fa, fb, N, K):
    print(f"grouped gemm fa={fa} fb={fb} N={N} K={K}", flush=True)
    rng = np.random.default_rng(K)
    lens = [304, 0, 16, 512, 80]
    off, E = _offsets(lens), len(lens)
    cap = int(off[-1])
    A, B = _codes(rng, (cap, K), fa, 20.0), _codes(rng, (E, N, K), fb, 10.0)
    a, b = oracle.decode(A, fa).reshape(A.shape).astype(np.float64), oracle.decode(B, fb).reshape(B.shape).astype(np.float64)
    want = np.concatenate([a[off[e]:off[e + 1]] @ b[e].T for e in range(E)]) * 0.25 * 0.125
    At, Bt = torch.from_numpy(A).to(DEV), torch.from_numpy(B).to(DEV)
    for dtype in (torch.bfloat16, torch.float32):
        gemm_close(to_f64(_gemm(At, fa, Bt, fb, off, cap, dtype, 0.25, 0.125)), want, dtype == torch.bfloat16)


@pytest.mark.parametrize("lens", LENS, ids=lambda v: f"{len(v)}experts{sum(v)}rows")
@pytest.mark.parametrize("N,K", [(16, 16), (130, 136), (256, 512), (300, 33), (512, 260)])
def test_wgrad_exact(lens, N, K):
    print(f"grouped wgrad lens={lens[:5]} N={N} K={K}", flush=True)
    rng = np.random.default_rng(N + K + 1)
    off, E = _offsets(lens), len(lens)
    cap = int(off[-1]) + 32
    A, B = _exact_codes(rng, (N, cap), F.E5M2), _exact_codes(rng, (K, cap), F.E4M3)
    a, b = oracle.decode(A, 1).reshape(A.shape).astype(np.float64), oracle.decode(B, 0).reshape(B.shape).astype(np.float64)
    want = np.stack([a[:, off[e]:off[e + 1]] @ b[:, off[e]:off[e + 1]].T for e in range(E)])
    for dtype in (torch.float32, torch.bfloat16):
        dW = torch.full((E, N, K), 7.0, device=DEV, dtype=dtype)
        F.fp8_grouped_wgrad(torch.from_numpy(A).to(DEV), F.E5M2, _scal(0.5), torch.from_numpy(B).to(DEV), F.E4M3, _scal(2.0),
                            torch.from_numpy(off).to(DEV), dW)
        assert torch.equal(dW.cpu(), torch.from_numpy(want).to(dtype))


@pytest.mark.parametrize("fa,fb", [(F.E5M2, F.E4M3), (F.E4M3, F.E4M3), (F.E4M3, F.E5M2), (F.E5M2, F.E5M2)])
def test_wgrad_formats(fa, fb):
    N, K = 768, 528
    print(f"grouped wgrad fa={fa} fb={fb}", flush=True)
    rng = np.random.default_rng(5)
    off = _offsets([1040, 0, 304, 16])
    cap = int(off[-1])
    A, B = _codes(rng, (N, cap), fa, 30.0), _codes(rng, (K, cap), fb, 20.0)
    a, b = oracle.decode(A, fa).reshape(A.shape).astype(np.float64), oracle.decode(B, fb).reshape(B.shape).astype(np.float64)
    for dtype in (torch.bfloat16, torch.float32):
        dW = torch.empty(4, N, K, device=DEV, dtype=dtype)
        F.fp8_grouped_wgrad(torch.from_numpy(A).to(DEV), fa, _scal(0.1), torch.from_numpy(B).to(DEV), fb, _scal(0.3),
                            torch.from_numpy(off).to(DEV), dW)
        for e in range(4):
            s = slice(off[e], off[e + 1])
            gemm_close(to_f64(dW[e]), (a[:, s] @ b[:, s].T) * float(np.float32(0.1)) * float(np.float32(0.3)),
                       dtype == torch.bfloat16)


def test_strided_operands():
    """The weights' transpose as the cast leaves it ([N, E * K] seen as [E, N, K]), rows of A and D
    inside wider buffers, an output that is not 8-byte aligned."""
    print("grouped strided", flush=True)
    rng = np.random.default_rng(9)
    E, N, K = 3, 144, 160
    off = _offsets([32, 48, 16])
    cap = int(off[-1])
    w_t = torch.from_numpy(_exact_codes(rng, (N, E * K), F.E4M3)).to(DEV)
    B = w_t.view(N, E, K).transpose(0, 1)
    wide = torch.from_numpy(_exact_codes(rng, (cap, K + 48), F.E5M2)).to(DEV)
    A = wide[:, 16:16 + K]
    want = _gemm(A.contiguous(), F.E5M2, B.contiguous(), F.E4M3, off, cap, torch.float32)
    for dtype, lead in ((torch.float32, 1), (torch.bfloat16, 3)):
        host = torch.full((cap, N + 9), 7.0, device=DEV, dtype=dtype)
        D = host[:, lead:lead + N]
        F.fp8_grouped_gemm(A, F.E5M2, _scal(0.5), B, F.E4M3, _scal(2.0), torch.from_numpy(off).to(DEV), D)
        assert torch.equal(D, want.to(dtype))
        assert (host[:, :lead] == 7).all() and (host[:, lead + N:] == 7).all()


def test_bad_offsets_stay_in_bounds():
    """Offsets past the buffer, negative, falling or not multiples of 16 are held to the buffer and
    rounded down; what remains well formed is right."""
    print("grouped bad offsets", flush=True)
    rng = np.random.default_rng(2)
    E, N, K, cap = 4, 64, 96, 128
    A, B = torch.from_numpy(_exact_codes(rng, (cap, K), 0)).to(DEV), torch.from_numpy(_exact_codes(rng, (E, N, K), 0)).to(DEV)
    good = _gemm(A, 0, B, 0, np.int32([0, 32, 32, 64, 128]), cap, torch.float32)
    got = _gemm(A, 0, B, 0, np.int32([-50, 40, 33, 64 + 7, 10 ** 9]), cap, torch.float32)
    assert torch.equal(got, good)
    At, Bt = A.t().contiguous(), torch.from_numpy(_exact_codes(rng, (48, cap), 0)).to(DEV)
    out = []
    for off in (np.int32([0, 32, 32, 64, 128]), np.int32([-50, 40, 32, 64 + 7, 10 ** 9]), np.int32([0, 32, 16, 64, 128])):
        dW = torch.empty(E, K, 48, **F32)
        F.fp8_grouped_wgrad(At, 0, _scal(1.0), Bt, 0, _scal(1.0), torch.from_numpy(off).to(DEV), dW)
        out.append(dW)
    assert torch.equal(out[0], out[1])
    # falling: the second expert has no rows, the third starts where the second ended
    assert torch.equal(out[2][[0, 3]], out[0][[0, 3]]) and (out[2][1] == 0).all()


def test_one_expert_equals_the_plain_gemm():
    """One expert over all rows is fp8_gemm_bias without a bias (same products, same gate)."""
    print("grouped one expert", flush=True)
    rng = np.random.default_rng(3)
    M, N, K = 768, 1024, 2048
    A, B = torch.from_numpy(_codes(rng, (M, K), 0, 30.0)).to(DEV), torch.from_numpy(_codes(rng, (1, N, K), 0, 9.0)).to(DEV)
    D = _gemm(A, 0, B, 0, np.int32([0, M]), M, torch.float32, 0.01, 0.02)
    ref = torch.empty(M, N, **F32)
    F.fp8_gemm_bias(A, 0, _scal(0.01), B[0], 0, _scal(0.02), None, ref)
    gemm_close(to_f64(D), to_f64(ref), False)


def test_empty_sizes():
    print("grouped empty", flush=True)
    s = _scal(1.0)
    off = torch.tensor([0, 32], **I32)
    D = torch.full((32, 48), 7.0, **F32)
    F.fp8_grouped_gemm(torch.empty(32, 0, **U8), 0, s, torch.empty(1, 48, 0, **U8), 0, s, off, D)
    assert (D == 0).all()                                     # an empty sum
    F.fp8_grouped_gemm(torch.empty(0, 16, **U8), 0, s, torch.empty(1, 48, 16, **U8), 0, s, off, torch.empty(0, 48, **F32))
    dW = torch.full((2, 16, 32), 7.0, **BF)
    F.fp8_grouped_wgrad(torch.empty(16, 0, **U8), 0, s, torch.empty(32, 0, **U8), 0, s, torch.zeros(3, **I32), dW)
    assert (dW == 0).all()


def test_results_do_not_depend_on_other_experts_and_graph_replays():
    print("grouped graph", flush=True)
    rng = np.random.default_rng(8)
    E, N, K = 6, 512, 768
    cap = 1200
    A, B = torch.from_numpy(_codes(rng, (cap, K), 0, 30.0)).to(DEV), torch.from_numpy(_codes(rng, (E, N, K), 0, 9.0)).to(DEV)
    At = A.t().contiguous()
    G = torch.from_numpy(_codes(rng, (N, cap), 1, 9.0)).to(DEV)
    off = torch.zeros(E + 1, **I32)
    s = _scal(0.01)
    D, dW = torch.zeros(cap, N, **BF), torch.zeros(E, N, K, **BF)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        F.fp8_grouped_gemm(A, 0, s, B, 0, s, off, D)
        F.fp8_grouped_wgrad(G, 1, s, At, 0, s, off, dW)
    first = None
    for lens in ([208, 0, 400, 16, 32, 544], [208, 304, 96, 16, 32, 544], [208, 992, 0, 0, 0, 0]):
        off.copy_(torch.from_numpy(_offsets(lens)))
        D.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = (D.clone(), dW.clone())
        D2, dW2 = torch.zeros_like(D), torch.zeros_like(dW)
        F.fp8_grouped_gemm(A, 0, s, B, 0, s, off, D2)
        F.fp8_grouped_wgrad(G, 1, s, At, 0, s, off, dW2)
        assert torch.equal(got[0], D2) and torch.equal(got[1], dW2)
        if first is None:
            first = (got[0][:208].clone(), got[1][0].clone())
        assert torch.equal(got[0][:208], first[0]) and torch.equal(got[1][0], first[1])
