"""The block operators' calls through the native module and through the binding's own marshalling:
the same results for tensors, raw pointers, prepared calls, and every way to name a stream."""
import pytest
import torch

import fp8_delayed_scaling_amd as F
from helpers import DEV

pytestmark = pytest.mark.gpu

BF = dict(device=DEV, dtype=torch.bfloat16)
U8 = dict(device=DEV, dtype=torch.uint8)
I32 = dict(device=DEV, dtype=torch.int32)


def _norm_args(M=6, H=96):
    g = torch.Generator(device=DEV).manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, **BF)  # noqa: E731
    return [r(M, H), r(H), None, None, r(M, H), 0.5, torch.zeros(M, H, **BF), None, r(H), None, None, torch.zeros(M, H, **BF)]


def test_native_calls_are_taken():
    """Arguments as they should be are taken by the native module, which says so."""
    a = _norm_args()
    call = F._native()
    assert call.norm_fwd(*a, None, None, F.E4M3, None, None, F.NORM_RMS, 1e-5, None) is True
    assert call.norm_fwd(*a, None, None, F.E4M3, None, None, F.NORM_RMS, -1.0, None) is False      # the entry point refuses
    assert call.norm_fwd(*[a[0][:, ::2], *a[1:]], None, None, F.E4M3, None, None, F.NORM_RMS, 1e-5, None) is False
    assert call.norm_fwd(*[a[0].float(), *a[1:]], None, None, F.E4M3, None, None, F.NORM_RMS, 1e-5, None) is False
    assert call.norm_fwd(*a) is False


@pytest.mark.parametrize("how", ["default", "stream", "handle", "context", "pointers", "int16"])
def test_every_way_gives_the_same(how):
    a = _norm_args()
    F.fp8_norm_residual_fwd(*a)
    want = a[6].clone(), a[11].clone()
    a[6].zero_(), a[11].zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    if how == "default":
        F.fp8_norm_residual_fwd(*a)
    elif how == "stream":
        F.fp8_norm_residual_fwd(*a, stream=s)
    elif how == "handle":
        F.fp8_norm_residual_fwd(*a, stream=s.cuda_stream)
    elif how == "context":
        with torch.cuda.stream(s):
            F.fp8_norm_residual_fwd(*a)
    elif how == "pointers":                    # a raw device pointer is passed through unchecked
        b = list(a)
        b[1], b[8] = a[1].data_ptr(), a[8].data_ptr()
        F.fp8_norm_residual_fwd(*b)
    else:                                      # bfloat16 bit patterns
        F.fp8_norm_residual_fwd(*[t.view(torch.int16) if torch.is_tensor(t) else t for t in a])
    torch.cuda.synchronize()
    assert torch.equal(a[6], want[0]) and torch.equal(a[11], want[1])


def test_work_is_put_on_the_named_stream():
    """A call on a captured stream is recorded, not run: the native module resolves the current stream."""
    a = _norm_args()
    F.fp8_norm_residual_fwd(*a)
    want = a[11].clone()
    a[11].zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        F.fp8_norm_residual_fwd(*a)
    torch.cuda.synchronize()
    assert (a[11] == 0).all()
    for _ in range(3):
        a[11].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a[11], want)


def test_refusals_name_the_argument_on_the_gpu():
    a = _norm_args()
    with pytest.raises(ValueError, match="resid"):
        F.fp8_norm_residual_fwd(*a[:4], a[4][:-1], *a[5:])
    with pytest.raises(F.Fp8dsError):
        F.fp8_norm_residual_fwd(*a, eps=-1.0)
    T, k, E = 5, 2, 3
    cap = F.fp8_moe_capacity(T, k, E)
    choice, off = torch.zeros(T, k, **I32), torch.zeros(E + 1, **I32)
    src, slot = torch.zeros(cap, **I32), torch.zeros(T, k, **I32)
    with pytest.raises(ValueError, match="offsets"):
        F.fp8_moe_plan(choice, E, 16, off[:-1], src, slot)
    with pytest.raises(F.Fp8dsError):
        F.fp8_moe_plan(choice, E, 8, off, src, slot)
    with pytest.raises(ValueError, match="out"):
        F.fp8_moe_sort_codes(torch.zeros(T, 32, **U8), src, k, torch.zeros(cap, 16, **U8))
