"""The experts' FP8 products of offsets that fall again and again: together the experts then have more
tiles than the rows can give, and the forward's search over them would not be bounded."""
import numpy as np
import pytest
import torch

import fp8_delayed_scaling_amd as F
from helpers import DEV

pytestmark = pytest.mark.gpu

F32 = dict(device=DEV, dtype=torch.float32)
U8 = dict(device=DEV, dtype=torch.uint8)


def _run(off, cap, N, K):
    s = torch.ones(1, **F32)
    E = len(off) - 1
    A, B = torch.full((cap, K), 0x38, **U8), torch.full((E, N, K), 0x38, **U8)          # 1.0
    D = torch.full((cap, N), 7.0, device=DEV, dtype=torch.bfloat16)
    F.fp8_grouped_gemm(A, 0, s, B, 0, s, torch.tensor(np.int32(off), device=DEV), D)
    torch.cuda.synchronize()
    return D


# paired tiles of each height, wide tiles; fewer experts than a wave's lanes, and several waves' worth
@pytest.mark.parametrize("E,cap,N,K", [(40, 512, 64, 32), (64, 4096, 256, 32), (200, 2048, 1024, 48), (64, 16384, 2048, 32)])
def test_falling_offsets_beyond_the_rows_write_nothing(E, cap, N, K):
    print(f"grouped falling E={E} cap={cap} N={N}", flush=True)
    D = _run([0 if e % 2 else cap for e in range(E + 1)], cap, N, K)
    assert (D == 7).all()


def test_rising_offsets_of_the_most_tiles_are_served():
    """Every expert's rows end in a tile of 16: as many tiles as sorted offsets can give."""
    for E, cap, N in ((64, 1024, 64), (65, 65 * 144, 512), (80, 80 * 272, 2048)):
        rows = cap // E
        assert rows % 16 == 0
        D = _run([e * rows for e in range(E + 1)], cap, N, 32)
        assert (D == 32).all()


def test_offsets_that_fall_a_little_keep_the_other_experts_rows():
    D = _run([0, 32, 16, 64, 128], 128, 48, 32)
    assert (D == 32).all()
