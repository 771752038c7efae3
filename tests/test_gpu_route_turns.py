"""The router over more rows than its blocks take in one turn: the next row's loads beside this one's choices, sums and counts
carried on from turn to turn, in both kernels of the forward and in the backward; and that every block of a launch takes rows."""
import math

import pytest
import torch

import fp8_delayed_scaling_amd as F
from test_gpu_route import DEV, U32, backward, check, close, forward_as_given, make, reference_backward, rel_of

pytestmark = pytest.mark.gpu

# one turn: 16384 rows of up to 256 experts, 4096 of more
FORWARD = [(16388, 64, 4), (40000, 256, 8), (33001, 7, 3), (20000, 100, 17), (4099, 300, 8), (9001, 1024, 4), (12500, 512, 66)]
# one turn: 8192 rows
BACKWARD = [(8195, 64, 4), (30011, 200, 8), (17000, 5, 2), (9001, 700, 6), (8200, 1024, 3)]


@pytest.mark.parametrize("case", FORWARD, ids=str)
@pytest.mark.parametrize("bf16", [False, True])
def test_forward(case, bf16):
    T, E, top = case
    check(make(T, E, T + E, bf16), top, normalise=top % 2 == 0)


def test_forward_of_padding_between_turns():
    """Whole turns of padding; rows with few open experts behind and before them."""
    x = make(50000, 40, 3, padded=0.0)
    x[10000:35000] = -math.inf
    x[35000:, 5:] = -math.inf
    got = check(x, 8)
    assert int(got["counts"][-1]) == 25000 and bool((got["experts"][10000:35000] == -1).all())
    assert bool((got["experts"][35000:, 5:] == -1).all())


@pytest.mark.parametrize("case", BACKWARD, ids=str)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("normalise", [False, True])
def test_backward(case, bf16, normalise):
    T, E, top = case
    x = make(T, E, T * 3 + E, bf16)
    g = torch.Generator(device=DEV).manual_seed(T)
    dweights, dloss = torch.randn(T, top, device=DEV, generator=g), torch.full((1,), 3.0, device=DEV)
    want, mag, p = reference_backward(x, top, normalise, dweights, dloss)
    got = backward(x, forward_as_given(x, top, normalise), dweights, dloss, normalise)
    most = rel_of(x, p).max(1, keepdim=True).values
    bound = mag * (3 * most + 2 * U32 * (E + top)) + 1e-37
    close(got, want, bound + (2.0 ** -8 * (want.abs() + bound) if bf16 else 0))


def test_strided_rows_over_turns():
    wide = torch.randn(20000, 90, device=DEV)
    x = wide[:, 7:71]
    got, want = check(x, 4), check(x.contiguous(), 4)
    assert all(torch.equal(got[n], want[n]) for n in got)


@pytest.mark.parametrize("T,E", [(65, 64), (100, 16), (128, 64), (1000, 256), (1000, 40), (8192, 64), (8192, 256), (16384, 8), (20000, 100), (17, 300), (5000, 1024)])
def test_every_block_takes_rows(T, E):
    """The live rows that each block counted lie at the workspace's end: none is zero where no row is padding, and they are T together."""
    size = F.fp8_moe_route_workspace_bytes(T, E)
    blocks = (size - 128) // (4 * (2 * E + 1))
    assert blocks > 1 and size == blocks * 4 * (2 * E + 1) + 128
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
    i32, f32 = dict(dtype=torch.int32, device=DEV), dict(dtype=torch.float32, device=DEV)
    F.fp8_moe_route(torch.randn(T, E, **f32), torch.empty(T, 2, **i32), torch.empty(T, 2, **f32), torch.empty(T, **f32), torch.empty(E + 1, **i32),
                    torch.empty(E, **f32), torch.empty(1, **f32), ws)
    live = ws[-4 * blocks:].view(torch.int32)
    assert int(live.sum()) == T and int(live.min()) > 0
