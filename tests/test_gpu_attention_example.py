"""The attention half of a block over batches of changing lengths."""
import importlib.util
import os

import pytest
import torch

from test_gpu_attention import DEV, offsets

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_a_shorter_batch_after_a_longer_one():
    """Rows past the second batch's last sequence hold nothing of the first's: the step is a new block's first step, bit for bit."""
    m = example()
    args = dict(tokens=256, width=128, heads=4, kv_heads=2, dim=64, seed=2)
    g = torch.Generator(device=DEV).manual_seed(7)
    x, dy = torch.randn(256, 128, device=DEV, generator=g).bfloat16(), torch.randn(256, 128, device=DEV, generator=g).bfloat16()
    short = offsets([90, 60])
    old, new = m.AttentionBlock(**args), m.AttentionBlock(**args)
    old.forward(x, offsets([100, 156]))
    old.backward(dy)
    old.history.zero_()
    for b in (old, new):
        b.forward(x, short)
        b.backward(dy)
    for name in ("y", "dx", "dw_qkv", "dw_o", "history"):
        assert torch.equal(getattr(old, name), getattr(new, name)), name
    assert bool((new.y[150:] == 0).all()) and bool((new.dx[150:] == 0).all())
