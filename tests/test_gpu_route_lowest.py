"""The router's gradient where logits are far from zero: rows and experts masked by a lowest value instead of -inf, logits that
float32's lse holds without their digits behind the point; and padding under a gradient that is not finite."""
import math

import pytest
import torch

from test_gpu_route import DEV, backward, close, make, reference_backward, run

pytestmark = pytest.mark.gpu


def check(x, top, normalise, dloss=2.0):
    g = torch.Generator(device=DEV).manual_seed(3)
    dw, dl = torch.randn(x.shape[0], top, device=DEV, generator=g), torch.full((1,), dloss, device=DEV)
    f = run(x, top, normalise)
    near = x.double() - x.double().max(1, keepdim=True).values       # shares are those of the differences, which 64 bits hold
    want, mag, _ = reference_backward(near, top, normalise, dw, dl)
    got = backward(x, f, dw, dl, normalise)
    # a probability is off by float32 roundings of differences below 2^7 and of sums, whatever the logits' size: below 2^-15 of it
    bound = mag * 2.0 ** -15 + 1e-37
    close(got, want, bound + (2.0 ** -8 * (want.abs() + bound) if x.dtype == torch.bfloat16 else 0))
    return f, got


@pytest.mark.parametrize("value", [-1e9, -1e30, None, 2.0 ** 30, -2.0 ** 27])
@pytest.mark.parametrize("E,top", [(5, 2), (64, 4), (100, 6), (256, 8), (1000, 3)])
@pytest.mark.parametrize("bf16", [False, True])
def test_rows_at_one_far_value(value, E, top, bf16):
    """Every expert has the same share of such a row, in the forward and in the gradient."""
    x = make(90, E, E, bf16, padded=0.0)
    value = torch.finfo(x.dtype).min if value is None else value
    x[::3] = value
    for normalise in (False, True):
        f, _ = check(x, top, normalise)
        assert bool((f["weights"][::3] - (1 / top if normalise else 1 / E)).abs().max() <= 2.0 ** -20)
    x[1::3, : E // 2] = value                            # and experts closed to a row that way
    check(x, top, True)
    check(x, top, False)


@pytest.mark.parametrize("power", [10, 16, 20, 22, 24, 26, 27, 28, 29, 30, 31, 60, 100])
@pytest.mark.parametrize("sign", [1, -1])
def test_logits_of_every_magnitude(power, sign):
    """Neighbouring values of 2^power, as far apart as float32 sets them: the others' shares are those of the differences."""
    g = torch.Generator(device=DEV).manual_seed(power)
    step = torch.randint(0, 4, (200, 48), device=DEV, generator=g).float() * 2.0 ** -23
    x = sign * 2.0 ** power * (1 + step)
    for normalise in (False, True):
        check(x, 4, normalise)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("bf16", [False, True])
def test_padding_under_a_gradient_that_is_not_finite(bad, bf16):
    """Padding rows get zeros whatever the gradients are."""
    x = make(100, 40, 1, bf16, padded=0.0)
    x[[0, 7, 99]] = -math.inf
    f = run(x, 4)
    dw = torch.full((100, 4), bad, device=DEV)
    got = backward(x, f, dw, torch.full((1,), bad, device=DEV), True)
    assert bool((got[[0, 7, 99]] == 0).all()) and bool(got[1].isnan().any())
