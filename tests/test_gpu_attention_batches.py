"""Batches as servers hold them: caches with a slot for each sequence, and the workspace of either kind of batch."""
import pytest
import torch

import fp8_delayed_scaling_amd as F
from test_gpu_attention import DEV, inputs, offsets, run_backward, run_forward

pytestmark = pytest.mark.gpu


def slots(used, size):
    """Key offsets of sequences in slots of `size` tokens, the unused part of each as a sequence without queries."""
    at = []
    for i, n in enumerate(used):
        at += [i * size, i * size + n]
    return torch.tensor(at + [len(used) * size], dtype=torch.int32, device=DEV)


def queries(new):
    """Their query offsets: an empty sequence behind each."""
    at = [0]
    for n in new:
        at += [at[-1] + n, at[-1] + n]
    return torch.tensor(at, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("new,used,size,Hq,Hkv,D,window", [
    ([1] * 6, [700, 1, 33, 1024, 512, 1000], 1024, 8, 2, 128, 0), ([1] * 3, [4000, 17, 2500], 4096, 8, 2, 128, 0), ([1] * 3, [4000, 17, 2500], 4096, 8, 2, 128, 512),
    ([5, 1, 40], [300, 1, 299], 300, 4, 4, 64, 0), ([200, 130], [3000, 131], 3008, 4, 2, 64, 0)])
def test_a_cache_with_a_slot_for_each_sequence(new, used, size, Hq, Hkv, D, window):
    """As the packed batch, bit for bit where both are split alike, and within the output's rounding anyhow; what lies behind a
    sequence in its slot is not read, and the cache grows without moving."""
    q, k, v, dout = inputs(len(new) + size, sum(new), len(used) * size, Hq, Hkv, D)
    held = torch.cat([torch.arange(n, device=DEV) + i * size for i, n in enumerate(used)])
    behind = torch.ones(len(used) * size, dtype=torch.bool, device=DEV)
    behind[held] = False
    k[behind], v[behind] = torch.nan, torch.nan
    oq, ok = queries(new), slots(used, size)
    out, lse, _ = run_forward(q, k, v, oq, ok, window=window)
    want = run_forward(q, k[held], v[held], offsets(new), offsets(used), window=window)
    # two sums of the same probabilities in other parts: float32, then a rounding to bfloat16 each
    assert bool(((out.float() - want[0].float()).abs() <= 2.0 ** -7 * want[0].float().abs() + 2.0 ** -8 * v[held].abs().max().float()).all())
    assert bool(((lse - want[1]).abs() <= 2.0 ** -18 * (want[1].abs() + 16)).all())
    got = run_backward(dout, q, k, v, want[0], want[1], oq, ok, window=window)
    ref = run_backward(dout, q, k[held], v[held], want[0], want[1], offsets(new), offsets(used), window=window)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1][held], ref[1]) and torch.equal(got[2][held], ref[2])
    for t in got[1:]:                                    # keys of a sequence without queries have no gradient
        assert bool((t[behind] == 0).all())


# (query tokens, keys, sequences, heads, key/value heads, head size): split unlike, or with unlike numbers of waves
EITHER = [(300, 16384, 2, 8, 2, 128), (256, 16384, 1, 8, 2, 128), (200, 40000, 8, 8, 4, 128), (40, 20000, 4, 4, 4, 64), (512, 16384, 4, 4, 1, 128),
          (1024, 1024, 8, 4, 2, 64), (4, 9000, 4, 8, 2, 128)]


@pytest.mark.parametrize("sizes", EITHER, ids=str)
def test_the_workspace_is_enough_for_any_call_of_its_sizes(sizes):
    """Exactly the bytes that were asked for, with offsets and without, with an amax and without: none is refused, and none
    writes past them."""
    Tq, Tk, B, Hq, Hkv, D = sizes
    q, k, v, _ = inputs(Tq, Tq, Tk, Hq, Hkv, D)
    n = F.fp8_attention_workspace_bytes(*sizes)
    room = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
    out8, s, amax = torch.empty(Tq, Hq * D, dtype=torch.uint8, device=DEV), torch.ones(1, device=DEV), torch.zeros(1, device=DEV)
    oq, ok = offsets([Tq // B] * B), offsets([Tk // B] * B)
    refused = 0
    for off in ((None, None), (oq, ok)):
        for kw in ({}, dict(out8=out8, scale=s, amax_slot=amax)):
            out = torch.empty_like(q)
            F.fp8_attention_fwd(q, k, v, out, None, *off, batch=B, workspace=room[:n], **kw)
            torch.cuda.synchronize()
            assert bool((room[n:] == 0x5A).all())
            try:                                         # of some call it is all needed; refused on the host
                F.fp8_attention_fwd(q, k, v, out, None, *off, batch=B, workspace=room[:n - 1], **kw)
            except F.Fp8dsError as e:
                assert e.status == -5
                refused += 1
    torch.cuda.synchronize()
    assert refused > 0
