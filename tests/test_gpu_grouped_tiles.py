"""The experts' FP8 products over every tiling: wide and paired tiles of every height, heights mixed
in one call, more experts than one wave looks at, short and odd contractions, outputs of every
alignment.  Operands are codes of 0, +-0.5, +-1, +-2, so every partial sum is exact in float32 and
the result must be the float32 product's, rounded once."""
import numpy as np
import pytest
import torch

import fp8_delayed_scaling_amd as F
import oracle
from helpers import DEV

pytestmark = pytest.mark.gpu

F32 = dict(device=DEV, dtype=torch.float32)
U8 = dict(device=DEV, dtype=torch.uint8)
VALUES = np.float32([0, 0.5, -0.5, 1, -1, 2, -2])


def _pair(gen, shape, fmt):
    """Codes and their values, both on the GPU."""
    pick = torch.randint(0, len(VALUES), shape, generator=gen, device=DEV)
    codes = torch.from_numpy(oracle.encode(VALUES, fmt)).to(DEV)
    return codes[pick], torch.from_numpy(VALUES).to(DEV)[pick]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device=DEV, dtype=torch.int32)


def _check_gemm(lens, N, K, seed, dtype=torch.bfloat16, pad=0, lead=0, fa=F.E4M3, fb=F.E4M3):
    print(f"tiles gemm experts={len(lens)} rows={sum(lens)} N={N} K={K} pad={pad} lead={lead}", flush=True)
    g = _gen(seed)
    cap = sum(lens) + 32
    A, a = _pair(g, (cap, K), fa)
    B, b = _pair(g, (len(lens), N, K), fb)
    host = torch.full((cap, N + pad + lead), 7.0, device=DEV, dtype=dtype)
    D = host[:, lead:lead + N]
    F.fp8_grouped_gemm(A, fa, torch.full((1,), 0.5, **F32), B, fb, torch.full((1,), 2.0, **F32), _offsets(lens), D)
    at = 0
    for e, n in enumerate(lens):
        want = (a[at:at + n] @ b[e].t().contiguous()).to(dtype)
        assert torch.equal(D[at:at + n], want), f"expert {e} of {n} rows"
        at += n
    assert (D[at:] == 7).all() and (host[:, :lead] == 7).all() and (host[:, lead + N:] == 7).all()


# rows of one expert for every number of 16-row blocks at a tile's end, and for each height of wide tiles
HEIGHTS = [16 * i for i in range(1, 35)] + [0, 784, 1040]


@pytest.mark.parametrize("N,K", [(512, 272), (1040, 640), (264, 1552)])
def test_every_height_paired(N, K):
    _check_gemm(HEIGHTS, N, K, N + K)


@pytest.mark.parametrize("N,K", [(2048, 784), (1288, 400), (1296, 128), (1040, 16), (2048, 1024), (2312, 912)])
def test_wide_tiles(N, K):
    """Enough rows for each expert that tiles of 256 rows are taken: every height in one call."""
    lens = [16 * i for i in range(1, 18)] + [4096, 288, 0, 2064, 528, 1296, 3008, 336, 5008, 4400]
    assert (sum(lens) + 32) // len(lens) >= 192
    lens = lens + [8192] if (sum(lens) // 256) * ((N + 255) // 256) < 520 else lens
    _check_gemm(lens, N, K, N + K)


@pytest.mark.parametrize("fa,fb", [(F.E5M2, F.E4M3), (F.E4M3, F.E5M2), (F.E5M2, F.E5M2)])
def test_wide_formats_and_float32(fa, fb):
    _check_gemm([9008, 0, 8192, 8496, 7504], 1100, 656, 5, torch.float32, fa=fa, fb=fb)


@pytest.mark.parametrize("pad,lead", [(3, 5), (8, 0), (0, 8), (1, 0)])
def test_wide_output_alignment(pad, lead):
    _check_gemm([9008, 16, 8192, 8496, 7504], 1032, 272, 6, pad=pad, lead=lead)
    _check_gemm([9008, 16, 8192, 8496, 7504], 1032, 272, 6, torch.float32, pad=pad, lead=lead)


@pytest.mark.parametrize("E,rows,N,K", [(1024, 16, 64, 144), (1000, 48, 272, 80), (130, 400, 1040, 96), (65, 512, 2048, 64)])
def test_many_experts(E, rows, N, K):
    rng = np.random.default_rng(E)
    lens = [int(v) // 16 * 16 for v in rng.uniform(0, 2 * rows + 15, E)]
    _check_gemm(lens, N, K, E)


@pytest.mark.parametrize("lens", [[16], [32, 0, 16], [0, 64, 0, 272], [512]], ids=str)
@pytest.mark.parametrize("N,K", [(240, 3392), (16, 16), (1000, 128), (8, 4096)])
def test_few_low_tiles(lens, N, K):
    _check_gemm(lens, N, K, N + K + len(lens))
    _check_gemm(lens, N, K, N + K + len(lens), torch.float32, pad=1)


def _check_wgrad(lens, N, K, seed, dtype=torch.bfloat16, lead=0):
    print(f"tiles wgrad experts={len(lens)} rows={sum(lens)} N={N} K={K} lead={lead}", flush=True)
    g = _gen(seed)
    cap = lead + sum(lens) + 32
    A, a = _pair(g, (N, cap), F.E5M2)
    B, b = _pair(g, (K, cap), F.E4M3)
    dW = torch.full((len(lens), N, K), 7.0, device=DEV, dtype=dtype)
    F.fp8_grouped_wgrad(A, F.E5M2, torch.full((1,), 0.5, **F32), B, F.E4M3, torch.full((1,), 2.0, **F32), _offsets(lens) + lead, dW)
    at = lead
    for e, n in enumerate(lens):
        want = (a[:, at:at + n].contiguous() @ b[:, at:at + n].t().contiguous()).to(dtype) if n else torch.zeros_like(dW[e])
        assert torch.equal(dW[e], want), f"expert {e} of {n} rows"
        at += n


# blocks shared in two, three and four groups, in none, and one expert after the other
@pytest.mark.parametrize("N,K", [(2048, 1024), (1024, 4096), (1408, 1024), (512, 1024), (4096, 4096), (130, 264), (1000, 2051)])
def test_wgrad_groups(N, K):
    lens = [272, 0, 16, 1040, 96, 32, 0, 48, 528, 16, 144]
    _check_wgrad(lens, N, K, N + K, lead=16)


def test_wgrad_many_experts_and_a_large_output():
    rng = np.random.default_rng(4)
    _check_wgrad([int(v) // 16 * 16 for v in rng.uniform(0, 80, 700)], 48, 136, 9)
    # past 512 MB: streaming stores
    _check_wgrad([int(v) // 16 * 16 for v in rng.uniform(0, 300, 36)], 2048, 3840, 10)
    _check_wgrad([int(v) // 16 * 16 for v in rng.uniform(0, 300, 20)], 1900, 3600, 11, torch.float32)
