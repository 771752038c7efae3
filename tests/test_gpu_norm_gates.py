"""The block norms' backward with more gates than blocks (one gate for each row or for few): every
thread layout, both kinds, even and odd widths, parts left out; and long units of many rows."""
import pytest
import torch

import fp8_delayed_scaling_amd as F
from test_gpu_norm import _backward, _bwd_buffers, _check_backward, _forward, _inputs, _rand

pytestmark = pytest.mark.gpu

# rows, width, gates: past 2048 blocks up to 1024 columns, 1024 up to 2048, 512 up to 4096, 256 beyond
MANY = [(2100, 40, 2100), (2100, 72, 2100), (4206, 520, 2103), (4206, 517, 2103), (1100, 1032, 1100), (1100, 2047, 1100),
        (1560, 2056, 520), (540, 4093, 540), (300, 4104, 300), (300, 8191, 300), (264, 8200, 264), (528, 12281, 264),
        (264, 12296, 264), (264, 16383, 264)]


def _run(M, H, G, kind, seed):
    p = _inputs(M, H, kind, G, seed)
    out = _forward(p, kind, 1.25)
    r = _rand(seed + 1)
    dh, dx = r(M, H, sd=0.1), r(M, H, sd=0.1)
    b = _bwd_buffers(M, H, kind, G)
    _backward(p, out, b, dh, dx, kind, 1.25)
    _check_backward(p, out, b, dh, dx, kind, 1.25)
    again = _bwd_buffers(M, H, kind, G)
    _backward(p, out, again, dh, dx, kind, 1.25)
    for n in b:
        if n != "ws" and b[n] is not None:
            assert torch.equal(b[n], again[n]), f"{n} differs between two runs"


@pytest.mark.parametrize("kind", [F.NORM_RMS, F.NORM_LAYER])
@pytest.mark.parametrize("shape", MANY, ids=str)
def test_more_gates_than_blocks(kind, shape):
    print(f"norm bwd many gates kind={kind} {shape}", flush=True)
    _run(*shape, kind, 41)


@pytest.mark.parametrize("kind", [F.NORM_RMS, F.NORM_LAYER])
@pytest.mark.parametrize("shape", [(2600, 4104, 1), (2600, 8200, 2), (1400, 12296, 1), (1400, 12279, 1), (3000, 1024, 0)], ids=str)
def test_units_of_many_rows(kind, shape):
    print(f"norm bwd long units kind={kind} {shape}", flush=True)
    _run(*shape, kind, 43)


@pytest.mark.parametrize("kind", [F.NORM_RMS, F.NORM_LAYER])
def test_many_gates_without_a_norm_after_the_block(kind):
    M, H = 2100, 136
    print(f"norm bwd many gates, gate alone kind={kind}", flush=True)
    p = _inputs(M, H, kind, M, 47)
    p["w_post"] = p["b_post"] = None
    out = _forward(p, kind, 0.5)
    out["post"] = torch.ones(2 if kind == F.NORM_LAYER else 1, M, device="cuda")
    r = _rand(48)
    dh, dx = r(M, H), r(M, H)
    b = _bwd_buffers(M, H, kind, M)
    b["dw_post"] = b["db_post"] = None
    F.fp8_norm_residual_bwd(dh, dx, p["o"], None, None, p["gate"], 0.5, out["x"], None, p["w_pre"], out["pre"], b["d_block"],
                            b["d_resid"], None, None, b["dgate"], b["dw_pre"], b["db_pre"], b["ws"], kind=kind)
    _check_backward(p, out, b, dh, dx, kind, 0.5)
