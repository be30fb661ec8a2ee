"""Norm gradients of rows whose mean is far from 0: x - mean is nearly exact, so the gradient depends on the deviations
alone, whichever kernel the rows' alignment and length select."""
import pytest
import torch

import layers_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from bit_gradient_compression_gb300 import loco
    return loco


@pytest.mark.parametrize("rows,cols", [(40, 96), (33, 500), (20, 1024), (9, 2048), (30, 4096), (5, 8000), (6, 12000), (3, 17000)])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("yd", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mean_of", [0.0, 100.0, -10000.0])
def test_gradient(L, rows, cols, pad, yd, mean_of):
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (r(rows, cols + pad) * 0.5 + mean_of)[:, :cols]
    dy, gamma = (r(rows, cols + pad) * 0.1).to(yd)[:, :cols], r(cols)
    mean = x.double().mean(1).float()
    rstd = ((x.double() - mean.double()[:, None]).square().mean(1) + 1e-5).rsqrt().float()
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    want, wdg, wdb = R.norm_backward(dy, xh, rstd, "layer", gamma, None)
    dx, dg, db = torch.empty(rows, cols + pad, device="cuda")[:, :cols], torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(L.loco_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    L.loco_norm_backward(L.make_norm(), dy, gamma, rstd, dx, x=x, mean=mean, dgamma=dg, dbeta=db, workspace=ws)
    # x - mean and its product with rstd are off by u each, relative to the deviation; a sum over the row has at most
    # 64 additions on a chain, and one for every 512 columns beyond
    n = 64 + cols / 512
    gg = (dy.double() * gamma.double()).abs()
    s1, s2 = gg.mean(1, keepdim=True), (gg * xh.abs()).mean(1, keepdim=True)
    tol = (n + 8) * R.U * rstd.double()[:, None] * (gg + s1 + xh.abs() * s2)
    R.close(dx, want, tol + R.out_tol(want, dx.dtype), "dx")
    R.close(dg, wdg, (rows + 64) * R.U * (dy.double() * xh).abs().sum(0) + R.out_tol(wdg, dg.dtype), "dgamma")
    R.close(db, wdb, (rows + 64) * R.U * dy.double().abs().sum(0) + R.out_tol(wdb, db.dtype), "dbeta")
