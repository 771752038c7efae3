"""The amax of attention's output: what it may be off by, which rows are computed again, and where the waves' largest
outputs are more than a thread holds at a time.

The outputs are made of probabilities rounded to bfloat16, each off by up to 2^-8 of itself, so an output is off by up to
2^-8 sum_j p |v|.  The row that proves largest and the one that is may differ by both roundings: 2^-7 of the largest such
sum bounds the amax.  Rows that are computed again are off by float32 roundings only."""
import math

import pytest
import torch

import attention_ref as ref
from test_gpu_attention import DEV, inputs, offsets, run_forward

pytestmark = pytest.mark.gpu


def amax_of(q, k, v, **kw):
    return run_forward(q, k, v, fp8=True, **kw)[2]["amax_slot"].item()


def sizes(q, k, v, **kw):
    """The amax in 64 bits, the largest sum_j p |v|, and what float32 sums and exponentials may be off by there."""
    most, reach, fine = 0.0, 0.0, 0.0
    for _, _, _, _, _, _, _, V, p, _, eps, _ in ref.heads(q, k, v, **kw):
        o, m = p @ V, p @ V.abs()
        most, reach = max(most, o.abs().max().item()), max(reach, m.max().item())
        fine = max(fine, (m * (3 * eps[:, None] + 4 * ref.U32 * (V.shape[0] + 64))).max().item())
    return most, reach, fine


@pytest.mark.parametrize("keys", [2, 3, 16, 200])
@pytest.mark.parametrize("sd", [0.02, 0.3, 2.0])
def test_bound_where_values_cancel(keys, sd):
    """Values of +1 and -1 under probabilities that nearly balance: outputs far below the terms that they are made of."""
    q, k, _, _ = inputs(keys, 600, keys, 4, 2, 64, sd=sd)
    v = torch.ones(keys, 2, 64, device=DEV).bfloat16()
    v[1::2] = -1
    got, (want, reach, fine) = amax_of(q, k, v, causal=False), sizes(q, k, v, causal=False)
    assert abs(got - want) <= 2.0 ** -7 * reach + fine


@pytest.mark.parametrize("seed", range(6))
def test_bound_of_near_rows_of_one_wave(seed):
    """All rows of a wave nearly alike: the one whose rounded output is largest need not be the one whose exact output is."""
    q, k, v, _ = inputs(seed, 1, 40, 4, 2, 64, sd=1.0)
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = (q.float() * (1 + 0.02 * torch.randn(500, 4, 64, device=DEV, generator=g))).bfloat16()
    v = v.abs()
    got, (want, reach, fine) = amax_of(q, k, v, causal=False), sizes(q, k, v, causal=False)
    assert abs(got - want) <= 2.0 ** -7 * reach + fine


def query_for(second):
    """A query element whose score against a key of ones puts the exponential of a key of zeros nearest to `second` of it."""
    a = torch.tensor(-math.log(second) / 0.125).bfloat16()
    return a, math.exp(-a.double().item() * 0.125)


@pytest.mark.parametrize("where", [0, 9, 39])
def test_the_sixteen_largest_are_computed_again(where):
    """40 heads over two keys, of which the second has the value: 39 round its exponential down, one rounds another up to the same.
    That head's 8 waves have the largest rounded outputs, all others the largest exact ones, of more candidates than
    are listed at a time."""
    down, e_down = query_for(254.46 / 256)
    up, e_up = query_for(253.54 / 256)
    r = lambda e: torch.tensor(e).bfloat16().item()  # noqa: E731
    assert r(e_down) == r(e_up) == 254 / 256 and r(e_up) / (1 + e_up) > 1.0015 * r(e_down) / (1 + e_down)
    q = torch.zeros(256, 40, 64, device=DEV).bfloat16()
    k, v = torch.zeros(2, 40, 64, device=DEV).bfloat16(), torch.zeros(2, 40, 64, device=DEV).bfloat16()
    q[:, :, 0], k[0, :, 0], v[1] = down, 1, 1
    q[:, where, 0] = up
    got = amax_of(q, k, v, causal=False)
    # in float32: the score, the exponential, the sum of two, the quotient
    assert abs(got - e_down / (1 + e_down)) <= 16 * 2.0 ** -24


@pytest.mark.parametrize("token", [0, 16383])
def test_many_waves(token):
    """More waves than the threads hold outputs of at a time: the one large output is found in the first and in the last."""
    T, Hq, Hkv = 16384, 32, 8
    q, k, v, _ = inputs(5, T, 8, Hq, Hkv, 64, sd=0.5)
    q[:, :, 0], k[:, :, 0] = -1, 0
    k[7, :, 0], v[7] = 30, 8
    q[token, 17, 0] = 16
    got = amax_of(q, k, v, causal=False)
    one = slice(token, token + 1)
    want, _, fine = sizes(q[one, 16:20], k[:, 4:5], v[:, 4:5], causal=False)
    others = run_forward(q, k, v, causal=False)[0].float().abs()
    others[token, 17] = 0
    assert others.max().item() < 0.9 * want                      # so no other row is a candidate for it
    assert abs(got - want) <= fine


def test_many_waves_alike():
    """Every wave a candidate, more than the threads hold."""
    T = 16384
    q, v = torch.zeros(T, 32, 64, device=DEV).bfloat16(), torch.ones(4, 8, 64, device=DEV).bfloat16()
    assert amax_of(q, torch.zeros_like(v), v, causal=False) == 1.0
    v[:, 5] = 1.0078125
    assert abs(amax_of(q, torch.zeros_like(v), v, causal=False) - 1.0078125) <= 2.0 ** -22


def test_ragged_with_more_candidates_than_are_listed():
    lens = [700, 1, 0, 333, 500]
    q, k, v, _ = inputs(3, sum(lens) + 4, sum(lens) + 4, 24, 24, 64, sd=0.0)
    v[:] = 1 - 2.0 ** -8
    v[705, 11] = 1.0                                             # the only key that the fourth sequence's first row sees
    off = offsets(lens)
    assert abs(amax_of(q, k, v, offsets_q=off, offsets_k=off) - 1.0) <= 2.0 ** -7
