"""Layer norms whose rows fill only a part of their threads' columns.  The columns past the width must
not reach a sum: with a large mean and a row that hardly varies, (0 - mean) * rstd is infinite there."""
import numpy as np
import pytest
import torch

import block_ref as R
import fp8_delayed_scaling_amd as F
from helpers import DEV

pytestmark = pytest.mark.gpu

BF = dict(device=DEV, dtype=torch.bfloat16)
F32 = dict(device=DEV, dtype=torch.float32)

BIG = 2.0 ** 100      # a constant row of a power-of-two width: its mean is exact, its deviations are zero
EPS = 1e-20           # rstd 1e10: BIG * rstd is past the float32 range


def _rows(M, H):
    """Constant rows, so that the norm is zero exactly and only the bias is left."""
    sign = torch.tensor([1.0, -1.0], device=DEV).repeat(M)[:M, None]
    return (sign * BIG).expand(M, H).to(torch.bfloat16).contiguous()


WIDTHS = [256, 8, 4, 2, 1]
# the backward is given its means: any width below what its threads hold (512, 1024, 2048, 4096, 8192, 12288, 16384 columns)
ANY = WIDTHS + [300, 503, 520, 1001, 1032, 2041, 2056, 4089, 4104, 4099, 8184, 8200, 8195, 12280, 12281, 12296, 16376, 16383]


@pytest.mark.parametrize("H", WIDTHS)
def test_forward_of_a_row_without_variation(H):
    print(f"norm columns forward H={H}", flush=True)
    M = 6
    g = torch.Generator(device=DEV).manual_seed(H)
    r = lambda *s: torch.randn(*s, generator=g, **BF)  # noqa: E731
    w, b, resid, w2, b2 = r(H), r(H), r(M, H), r(H), r(H)
    x, h = torch.zeros(M, H, **BF), torch.zeros(M, H, **BF)
    post, pre = torch.zeros(2, M, **F32), torch.zeros(2, M, **F32)
    F.fp8_norm_residual_fwd(_rows(M, H), w, b, None, resid, 1.0, x, post, w2, b2, pre, h, kind=F.NORM_LAYER, eps=EPS)
    assert torch.equal(x, (resid.float() + b.float()).bfloat16())
    v = x.cpu().double().numpy()
    want, _, _, err = R.norm(v, w2.cpu().double().numpy(), b2.cpu().double().numpy(), True, EPS)
    got = h.cpu().double().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= err + R.BF16 * np.abs(want)).all()


@pytest.mark.parametrize("H", ANY)
def test_backward_of_a_row_without_variation(H):
    """hat(block_out) is zero: d_block = rstd * (dn w - mean of dn w), dw_post = 0, db_post = sum of dn."""
    print(f"norm columns backward H={H}", flush=True)
    M = 6
    g = torch.Generator(device=DEV).manual_seed(H + 1)
    r = lambda *s: torch.randn(*s, generator=g, **BF)  # noqa: E731
    o, w, b, dx = _rows(M, H), r(H), r(H), r(M, H)
    rstd = 2.0 ** 33                                  # about 1 / sqrt(EPS), exact
    post = torch.stack([torch.full((M,), rstd, **F32), o[:, 0].float()])
    d_block, d_resid = torch.zeros(M, H, **BF), torch.zeros(M, H, **BF)
    dw, db = torch.zeros(H, **F32), torch.zeros(H, **F32)
    ws = torch.empty(F.fp8_norm_residual_workspace_bytes(M, H, 1), device=DEV, dtype=torch.uint8)
    F.fp8_norm_residual_bwd(None, dx, o, w, b, None, 0.5, None, post, None, None, d_block, d_resid, dw, db, None, None, None, ws,
                            kind=F.NORM_LAYER)
    d, wv = dx.cpu().double().numpy(), w.cpu().double().numpy()
    q = d * wv
    want = rstd * (q - q.mean(1, keepdims=True))
    err = R.STEPS * R.U * rstd * (np.abs(q) + np.abs(q).mean(1, keepdims=True))
    got = d_block.cpu().double().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= err + R.BF16 * np.abs(want)).all()
    assert (dw == 0).all()
    assert (np.abs(db.cpu().double().numpy() - d.sum(0)) <= (M + R.STEPS) * R.U * np.abs(d).sum(0)).all()
    assert torch.equal(d_resid, (dx.float() * 0.5).bfloat16())


@pytest.mark.parametrize("H", ANY)
def test_backward_of_the_second_norm(H):
    print(f"norm columns second H={H}", flush=True)
    M = 6
    g = torch.Generator(device=DEV).manual_seed(H + 2)
    r = lambda *s: torch.randn(*s, generator=g, **BF)  # noqa: E731
    x, w, dh = _rows(M, H), r(H), r(M, H)
    rstd = 2.0 ** 33
    pre = torch.stack([torch.full((M,), rstd, **F32), x[:, 0].float()])
    d_resid, dw, db = torch.zeros(M, H, **BF), torch.zeros(H, **F32), torch.zeros(H, **F32)
    ws = torch.empty(F.fp8_norm_residual_workspace_bytes(M, H, 0), device=DEV, dtype=torch.uint8)
    F.fp8_norm_residual_bwd(dh, None, None, None, None, None, 1.0, x, None, w, pre, None, d_resid, None, None, None, dw, db, ws,
                            kind=F.NORM_LAYER)
    q = dh.cpu().double().numpy() * w.cpu().double().numpy()
    want = rstd * (q - q.mean(1, keepdims=True))
    err = R.STEPS * R.U * rstd * (np.abs(q) + np.abs(q).mean(1, keepdims=True))
    got = d_resid.cpu().double().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= err + R.BF16 * np.abs(want)).all()
    assert (dw == 0).all()
