"""Norm gradients of rows that two CTAs share: more rows than pairs fit at once, and ragged second halves."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import test_layers_gpu as base  # noqa: E402
from test_layers_gpu import BF16, F32, L  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(1, 8193), (2, 8200), (401, 8225), (170, 9001), (250, 12000), (333, 16352), (160, 16383),
                                       (500, 16384)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("source", ["x", "ckpt"])
@pytest.mark.parametrize("xd,yd,gd", [(F32, F32, BF16), (BF16, BF16, F32), (F32, BF16, BF16)])
@pytest.mark.parametrize("pad", [0, 8, 5])
def test_two_ctas_a_row(L, rows, cols, kind, source, xd, yd, gd, pad):  # noqa: F811
    base.test_norm_backward(L, rows, cols, kind, source, xd, yd, gd, pad)


def test_same_bits_every_run(L):  # noqa: F811
    rows, cols = 700, 9003
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randn(rows, cols, device="cuda", generator=gen).to(BF16) for _ in range(2))
    gamma = torch.randn(cols, device="cuda", generator=gen)
    mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
    y = torch.empty_like(x)
    cfg = L.make_norm()
    L.loco_norm_forward(cfg, x, gamma, gamma, y, mean=mean, rstd=rstd)
    ws = torch.empty(L.loco_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    seen = []
    for _ in range(3):
        dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
        L.loco_norm_backward(cfg, dy, gamma, rstd, dx, x=x, mean=mean, residual=dy, dgamma=dg, dbeta=db, workspace=ws)
        seen.append((dx, dg, db))
    for other in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(seen[0], other))
