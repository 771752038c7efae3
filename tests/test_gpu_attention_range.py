"""Attention where scores are of any size that float32 holds: rows all of whose keys are masked by a lowest value, scores
that grow or fall by dozens of orders along the keys, of either sign."""
import math

import pytest
import torch

import fp8_delayed_scaling_amd as F
from test_gpu_attention import DEV, U16, inputs, offsets, run_backward, run_forward

pytestmark = pytest.mark.gpu

# (sequences, query tokens, keys, heads, key/value heads, head size): blocks of 128 rows, few rows, either split over the keys
SHAPES = [(1, 300, 300, 4, 2, 128), (2, 150, 150, 8, 8, 64), (1, 200, 333, 4, 1, 96), (2, 3, 200, 4, 2, 64), (1, 1, 5000, 8, 2, 128),
          (1, 200, 5000, 4, 2, 64)]


def make(shape, seed=1):
    """Queries whose first element alone makes the scores: it is 1, the other elements meet zeros in the keys."""
    B, lq, lk, Hq, Hkv, D = shape
    q, k, v, dout = inputs(seed, B * lq, B * lk, Hq, Hkv, D)
    k[:] = 0
    q[:, :, 0] = 1
    return q, k, v, dout


def reference(q, k, v, B, causal, scale):
    """out and lse from scores less their row's largest, so that 64 bits hold the differences."""
    Tq, Hq, D = q.shape
    lq, lk, G = Tq // B, k.shape[0] // B, Hq // k.shape[1]
    out, lse = torch.zeros(Tq, Hq, D, dtype=torch.float64, device=DEV), torch.zeros(Hq, Tq, dtype=torch.float64, device=DEV)
    size = torch.zeros_like(out)
    see = torch.ones(lq, lk, dtype=torch.bool, device=DEV)
    if causal:
        see = torch.arange(lk, device=DEV)[None] <= torch.arange(lq, device=DEV)[:, None] + (lk - lq)
    for b in range(B):
        rows, keys = slice(b * lq, (b + 1) * lq), slice(b * lk, (b + 1) * lk)
        for h in range(Hq):
            s = (q[rows, h, 0].double()[:, None] * k[keys, h // G, 0].double()[None]).masked_fill(~see, -math.inf)
            top = s.max(1, keepdim=True).values
            e = torch.exp((s - top) * scale)
            p = e / e.sum(1, keepdim=True)
            out[rows, h], size[rows, h] = p @ v[keys, h // G].double(), p @ v[keys, h // G].double().abs()
            lse[h, rows] = top[:, 0] * scale + torch.log(e.sum(1))
    return out, lse, size


def check(q, k, v, B, causal=True, scale=0.125):
    out, lse, f = run_forward(q, k, v, batch=B, causal=causal, scale=scale, fp8=True)
    w_out, w_lse, size = reference(q, k, v, B, causal, scale)
    # a probability: the rounding of it as an operand, and 2^-12 for the exponential of a difference below 2^8 and float32 sums
    bound = size * (U16 + 2.0 ** -12)
    bad = ~((out.double() - w_out).abs() <= bound + U16 * (w_out.abs() + bound))
    assert not bad.any(), f"{int(bad.sum())} outputs of {bad.numel()}, first at {bad.nonzero()[0].tolist()}"
    bad = ~((lse.double() - w_lse).abs() <= 2.0 ** -21 * (w_lse.abs() + 16))
    assert not bad.any(), f"{int(bad.sum())} sums of {bad.numel()}, first at {bad.nonzero()[0].tolist()}"
    assert math.isfinite(f["amax_slot"].item())
    return out, lse


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("value", [-1e30, -3e38, -2.0 ** 40, 1e30, 2.0 ** 33])
@pytest.mark.parametrize("causal", [True, False])
def test_every_key_at_one_far_value(shape, value, causal):
    """No key is nearer than another: each counts the same."""
    q, k, v, _ = make(shape)
    k[:, :, 0] = value
    check(q, k, v, shape[0], causal)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("seed", range(3))
def test_far_and_near_keys_in_any_order(shape, seed):
    """Keys at the lowest value, at none, at ordinary and at far values, in runs and one by one; the largest that a row sees counts."""
    q, k, v, _ = make(shape, seed)
    lk = k.shape[0]
    g = torch.Generator(device=DEV).manual_seed(seed)
    values = torch.tensor([-1e30, -2.0 ** 36, -3.0, 0.0, 5.0, 2.0 ** 28, 2.0 ** 34][:7 if seed == 0 else 5], device=DEV)
    at = torch.randint(0, len(values), (lk,), device=DEV, generator=g)
    if seed != 1:                                        # runs of 50 keys: whole tiles at one value
        at = at[torch.arange(lk, device=DEV) // 50 * 50]
    k[:, :, 0] = values[at][:, None].bfloat16()
    check(q, k, v, shape[0])
    k[:, :, 0] = values.sort().values[torch.arange(lk, device=DEV) * len(values) // lk][:, None].bfloat16()      # rising, a step at a time
    check(q, k, v, shape[0])
    k[:, :, 0] = k[:, :, 0].flip(0)
    check(q, k, v, shape[0])


@pytest.mark.parametrize("power", [16, 20, 24, 26, 27, 28, 30, 33, 40, 60, 100])
@pytest.mark.parametrize("scale", [0.125, 0.7, 1.0])
def test_scores_of_every_magnitude(power, scale):
    """Neighbouring bfloat16 values of 2^power, of either sign: beside the largest, the others' weights are those of the differences."""
    for shape in SHAPES[:4]:
        for sign in (1, -1):
            q, k, v, _ = make(shape, power)
            step = (torch.arange(k.shape[0], device=DEV) * 7 % 3).float() * 2.0 ** -8
            k[:, :, 0] = (sign * 2.0 ** power * (1 - step))[:, None].bfloat16()
            check(q, k, v, shape[0], scale=scale)


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[1] == s[2]] + [(1, 200, 333, 4, 1, 96)], ids=str)
@pytest.mark.parametrize("value", [-1e30, -2.0 ** 40, 2.0 ** 33])
def test_gradients_beside_rows_of_far_scores(shape, value):
    """The first keys of each sequence are padding, masked by a far value: rows that see nothing else give no gradient, as their
    probabilities cannot be had from a float32 lse; the other rows' gradients are as without the padding."""
    B, lq, lk, Hq, Hkv, D = shape
    pad, past = 40, lk - lq
    low = value < 0
    q, k, v, dout = inputs(9, B * lq, B * lk, Hq, Hkv, D)
    q[:, :, 0], k[:, :, 0] = 1, 0
    masked = (torch.arange(B * lk, device=DEV) % lk) < pad
    if low:
        k[masked, :, 0] = value
    else:                                                # every key far but the padding's: all rows that see one of them
        k[~masked, :, 0] = value
    out, lse, _ = run_forward(q, k, v, batch=B)
    got = run_backward(dout, q, k, v, out, lse, batch=B)
    assert all(bool(t.isfinite().all()) for t in (out, lse, *got))
    token = torch.arange(B * lq, device=DEV) % lq
    far = (token + past < pad) if low else (token + past >= pad)
    assert bool((lse[:, far].abs() >= 2.0 ** 24).all()) and bool((lse[:, ~far].abs() < 2.0 ** 10).all())
    assert bool((got[0][far] == 0).all())
    # the same rows with their output gradient at zero
    quiet = dout.clone()
    quiet[far] = 0
    for a, b in zip(got, run_backward(quiet, q, k, v, out, lse, batch=B)):
        assert torch.equal(a, b)


def test_ragged_left_padding():
    """Packed sequences that begin with padding masked by a lowest value; a sequence that is padding throughout."""
    lens = [70, 5, 200, 1]
    q, k, v, dout = inputs(4, sum(lens), sum(lens), 4, 2, 64)
    q[:, :, 0], k[:, :, 0] = 1, 0
    start = 0
    for n, pad in zip(lens, (30, 5, 64, 0)):
        k[start:start + pad, :, 0] = torch.finfo(torch.bfloat16).min
        start += n
    off = offsets(lens)
    out, lse, f = run_forward(q, k, v, off, off, fp8=True)
    assert bool(out.isfinite().all()) and bool(lse.isfinite().all()) and bool(f["amax_slot"].isfinite())
    assert torch.equal(out[0], v[0].repeat_interleave(2, 0)) and torch.equal(out[70], v[70].repeat_interleave(2, 0))   # one key: its value
    for t in run_backward(dout, q, k, v, out, lse, off, off):
        assert bool(t.isfinite().all())
    assert F.fp8_attention_bwd_workspace_bytes(276, 276, 4, 4, 2, 64) > 0
