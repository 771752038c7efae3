"""Tokens sorted by expert and back at sizes whose work is more than one launch can number (2^32
threads): many choices of narrow rows, 2^24 wide rows, 2^30 narrow ones.  Values are small whole
numbers, so every result is exact."""
import pytest
import torch

import fp8_delayed_scaling_amd as F
from helpers import DEV

pytestmark = pytest.mark.gpu

BF = dict(device=DEV, dtype=torch.bfloat16)
F32 = dict(device=DEV, dtype=torch.float32)
U8 = dict(device=DEV, dtype=torch.uint8)
I32 = dict(device=DEV, dtype=torch.int32)


@pytest.fixture(autouse=True)
def _room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of free GPU memory")
    yield
    torch.cuda.empty_cache()


def _whole(g, *shape):
    return torch.randint(-2, 3, shape, generator=g, device=DEV).bfloat16()


def _pieces(n, step):
    return [(a, min(n, a + step)) for a in range(0, n, step)]


def test_weight_gradient_of_2_26_choices():
    T, k, H, cap = (1 << 20) + 1, 64, 16, 4096
    print(f"weight gradient choices={T * k}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(1)
    dy, ys = _whole(g, T, H), _whole(g, cap, H)
    slot = torch.randint(-3, cap + 3, (T, k), generator=g, **I32)
    dw = torch.full((T, k), 7.0, **F32)
    F.fp8_moe_weight_grad(dy, ys, slot, dw)
    for a, b in _pieces(T, 1 << 16):
        s = slot[a:b].long()
        live = (s >= 0) & (s < cap)
        dots = dy[a:b].float() @ ys.float().t().contiguous()          # [tokens, cap]
        want = torch.where(live, dots.gather(1, s.clamp(0, cap - 1)), torch.zeros((), device=DEV))
        assert torch.equal(dw[a:b], want), (a, b)


def test_combine_of_2_24_wide_tokens():
    T, H, cap = (1 << 24) + 5, 2048, 64
    print(f"combine tokens={T}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(2)
    ys = _whole(g, cap, H)
    slot = torch.randint(-1, cap + 1, (T, 1), generator=g, **I32)
    y = torch.full((T, H), 7.0, **BF)
    F.fp8_moe_combine(ys, slot, None, y)
    table = torch.cat([torch.zeros(1, H, **BF), ys, torch.zeros(1, H, **BF)])
    for a, b in _pieces(T, 1 << 20):
        assert torch.equal(y[a:b], table[slot[a:b, 0].long() + 1]), (a, b)


@pytest.mark.parametrize("what", ["codes", "bf16"])
def test_sort_of_2_24_wide_rows(what):
    T, cap = 48, (1 << 24) + 16
    H = 4096 if what == "codes" else 2304
    print(f"sort {what} rows={cap}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(3)
    src = torch.randint(-1, T + 1, (cap,), generator=g, **I32)
    if what == "codes":
        x, out = torch.randint(1, 100, (T, H), generator=g, **U8), torch.full((cap, H), 7, **U8)
        F.fp8_moe_sort_codes(x, src, 1, out)
    else:
        x, out = _whole(g, T, H), torch.full((cap, H), 7.0, **BF)
        F.fp8_moe_sort_bf16(x, src, 1, None, out)
    table = torch.cat([torch.zeros_like(x[:1]), x, torch.zeros_like(x[:1])])
    for a, b in _pieces(cap, 1 << 20):
        assert torch.equal(out[a:b], table[src[a:b].long() + 1]), (a, b)


def test_sort_and_transpose_of_2_30_narrow_rows():
    T, H, cap = 48, 16, (1 << 30) + 4112
    print(f"sort + transpose rows={cap}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(4)
    src = torch.randint(-1, T + 1, (cap,), generator=g, **I32)
    x = _whole(g, T, H)
    out, out_t = torch.full((cap, H), 7, **U8), torch.full((H, cap), 7, **U8)
    scale, sinv, amax = torch.full((1,), 4.0, **F32), torch.zeros(1, **F32), torch.zeros(1, **F32)
    F.fp8_moe_sort_cast(x, src, 1, None, scale, F.E4M3, out, out_t, sinv, amax)
    codes = (x.float() * 4).to(torch.float8_e4m3fn).view(torch.uint8)
    table = torch.cat([torch.zeros_like(codes[:1]), codes, torch.zeros_like(codes[:1])])
    for a, b in _pieces(cap, 1 << 25):
        want = table[src[a:b].long() + 1]
        assert torch.equal(out[a:b], want), (a, b)
        assert torch.equal(out_t[:, a:b], want.t()), (a, b)
    assert amax.item() == 2.0 and sinv.item() == 0.25
