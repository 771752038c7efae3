"""The experts' FP8 products without a contraction, whatever the operands' strides, and with operands so
small that a K step reaches past all of them."""
import pytest
import torch

import fp8_delayed_scaling_amd as F
from helpers import DEV

pytestmark = pytest.mark.gpu

F32 = dict(device=DEV, dtype=torch.float32)
U8 = dict(device=DEV, dtype=torch.uint8)
I32 = dict(device=DEV, dtype=torch.int32)


@pytest.mark.parametrize("ld", [1, 1 << 24, 1 << 26, (1 << 28) + 16])
@pytest.mark.parametrize("cap,E,N", [(64, 2, 48), (1024, 3, 600)])
def test_empty_contraction_of_any_stride(ld, cap, E, N):
    print(f"grouped empty ld={ld} cap={cap}", flush=True)
    s = torch.ones(1, **F32)
    none = torch.empty(0, **U8)
    off = torch.tensor([0, *[16 * (e + 1) for e in range(E - 1)], cap], **I32)
    for dtype in (torch.bfloat16, torch.float32):
        D = torch.full((cap, N), 7.0, device=DEV, dtype=dtype)
        F.fp8_grouped_gemm(none.as_strided((cap, 0), (ld, 1)), 0, s, none.as_strided((E, N, 0), (ld, ld, 1)), 0, s, off, D)
        assert (D == 0).all()
        dW = torch.full((E, N, 80), 7.0, device=DEV, dtype=dtype)
        F.fp8_grouped_wgrad(none.as_strided((N, 0), (ld, 1)), 0, s, none.as_strided((80, 0), (ld, 1)), 0, s, off * 0, dW)
        assert (dW == 0).all()


@pytest.mark.parametrize("N", [1, 3, 8, 16])
@pytest.mark.parametrize("K", [16, 32, 144, 272])
def test_operands_smaller_than_a_step(N, K):
    """16 rows by N: a step's K bytes are more than the operand's extent.  Codes of 1.0."""
    print(f"grouped small N={N} K={K}", flush=True)
    s = torch.ones(1, **F32)
    A, B = torch.full((16, K), 0x38, **U8), torch.full((1, N, K), 0x38, **U8)
    D = torch.full((16, N), 7.0, **F32)
    F.fp8_grouped_gemm(A, 0, s, B, 0, s, torch.tensor([0, 16], **I32), D)
    assert (D == K).all()
    dW = torch.full((1, N, 16), 7.0, **F32)
    Bt = torch.full((16, K), 0x38, **U8)
    F.fp8_grouped_wgrad(B[0], 0, s, Bt, 0, s, torch.tensor([0, K], **I32), dW)
    assert (dW == K).all()
