"""The experts' FP8 products whose weights no cache holds: B comes from HBM, later than A, so that a
read of LDS ahead of its load shows.  Operands are codes of 0, +-0.5, +-1, +-2: every partial sum is
exact in float32 and each output must be the float32 product's, rounded once."""
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
    pick = torch.randint(0, len(VALUES), shape, generator=gen, device=DEV, dtype=torch.uint8)
    codes = torch.from_numpy(oracle.encode(VALUES, fmt)).to(DEV)
    values = torch.from_numpy(VALUES).to(DEV)
    out, val = torch.empty(shape, **U8), torch.empty(shape, **F32)
    for i in range(len(VALUES)):
        out[pick == i], val[pick == i] = codes[i], values[i]
    return out, val


# tiles of 256 rows, several to a block: forward (E4M3) and input gradient (E5M2 by E4M3), a
# contraction of whole steps and one that ends inside a step, and one of two steps
@pytest.mark.parametrize("E,N,K,fa,dtype", [
    (72, 2048, 4096, F.E4M3, torch.bfloat16),
    (72, 2048, 4096, F.E4M3, torch.float32),
    (66, 2048, 4112, F.E5M2, torch.bfloat16),
    (128, 16384, 256, F.E4M3, torch.bfloat16),
])
def test_wide_tiles_of_cold_weights(E, N, K, fa, dtype):
    print(f"grouped cold E={E} N={N} K={K} {dtype}", flush=True)
    assert E * N * K >= 512 << 20
    g = torch.Generator(device=DEV).manual_seed(E + K)
    rng = np.random.default_rng(E + K)
    lens = [int(v) // 16 * 16 for v in rng.uniform(0, 900, E)]
    off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device=DEV, dtype=torch.int32)
    cap = sum(lens)
    assert cap // E >= 192 and cap // 256 * ((N + 255) // 256) >= 512
    A, a = _pair(g, (cap, K), fa)
    B, b = _pair(g, (E, N, K), F.E4M3)
    sa, sb = torch.full((1,), 0.5, **F32), torch.full((1,), 2.0, **F32)
    want = torch.empty(cap, N, device=DEV, dtype=dtype)
    at = 0
    for e, n in enumerate(lens):
        want[at:at + n] = (a[at:at + n] @ b[e].t().contiguous()).to(dtype)
        at += n
    del a, b
    other = torch.empty(1 << 30, **U8)
    for i in range(3):
        D = torch.full((cap, N), 7.0, device=DEV, dtype=dtype)
        other.fill_(i)                                    # nothing of the operands stays in a cache
        F.fp8_grouped_gemm(A, fa, sa, B, F.E4M3, sb, off, D)
        assert torch.equal(D, want), f"call {i}: {int((D != want).sum())} of {D.numel()} differ"
