"""NaN and infinities reach the outputs that read them and no others, in every kernel of the layers."""
import math

import pytest
import torch

import layers_ref as R
from test_layers_gpu import BF16, F32, L, gen, rand  # noqa: F401

pytestmark = pytest.mark.gpu


def bad_is(t, rows=(), cols=()):
    """Exactly these rows and columns of t hold values that are not finite, and they hold nothing else."""
    want = torch.zeros(t.shape, dtype=torch.bool, device=t.device)
    want[list(rows)] = True
    if t.dim() == 2:
        want[:, list(cols)] = True
    assert torch.equal(~torch.isfinite(t), want)


@pytest.mark.parametrize("cols,pad", [(96, 0), (96, 1), (500, 0), (4096, 0), (4095, 0), (9000, 0), (9001, 0), (17000, 0)])
@pytest.mark.parametrize("source", ["x", "ckpt"])
def test_norm_backward(L, cols, pad, source):  # noqa: F811
    rows, g = 12, gen(70)
    x, dy, gamma = rand(g, rows, cols, F32, ld=cols + pad), rand(g, rows, cols, BF16, ld=cols + pad), rand(g, 1, cols, F32)[0]
    m, r, xh, _ = R.norm_forward(x, "layer", 1e-5, None, None)
    dy[2, 5] = math.nan
    dy[7, cols - 1] = -math.inf
    kw = dict(x=x, mean=m.float())
    x[4, 11] = math.inf
    hit = {11}
    if source == "ckpt":
        xh[4, 11] = math.inf
        codes, scales = R.encode(xh)
        kw = dict(codes=codes, scales=scales)
        hit = set(range(0, 32))                          # the block
    dx, dg, db = torch.empty(rows, cols, device="cuda"), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(L.loco_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    L.loco_norm_backward(L.make_norm(), dy, gamma, r.float(), dx, dgamma=dg, dbeta=db, workspace=ws, **kw)
    bad_is(dx, rows=(2, 4, 7))
    bad_is(db, rows=(5, cols - 1))
    bad_is(dg, rows=sorted(hit | {5, cols - 1}))


# the few-row kernel; split k; one CTA a tile; pairs of CTAs; each with operands that TMA takes and that it does not
@pytest.mark.parametrize("T,N,K", [(1, 2440, 264), (2, 2500, 1024), (4, 2432, 520), (16, 300, 2048), (200, 520, 1024), (300, 700, 72),
                                   (1100, 2300, 264)])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("save", [False, True])
def test_linear_forward(L, T, N, K, pad, save):  # noqa: F811
    g = gen(71)
    K8 = -(-K // 8) * 8
    x, w = rand(g, T, K, BF16, ld=K8 + pad), rand(g, N, K, BF16, K ** -0.5, ld=K8 + pad)
    x[T - 1, K - 1] = math.nan
    w[9, 4] = math.inf
    w[N - 1, 0] = math.nan
    rows = {T - 1}
    if T > 2:
        x[0, 3] = -math.inf
        rows.add(0)
    y = torch.empty(T, N, device="cuda")
    codes = scales = None
    if save:
        nb = -(-N // 32)
        codes, scales = torch.empty(T, nb * 32, dtype=torch.int8, device="cuda"), torch.empty(T, nb, dtype=torch.uint8, device="cuda")
    L.loco_linear_forward(x, w, y, codes=codes, scales=scales)
    bad_is(y, rows=rows, cols=(9, N - 1))
    if save:
        want = torch.zeros(scales.shape, dtype=torch.bool, device="cuda")
        want[list(rows)] = True
        want[:, [0, (N - 1) // 32]] = True
        assert torch.equal(scales == 255, want)


@pytest.mark.parametrize("T,N,K", [(512, 256, 264), (64, 300, 520), (300, 1100, 2300), (2048, 64, 130)])
@pytest.mark.parametrize("pad", [0, 1])
def test_linear_backward(L, T, N, K, pad):  # noqa: F811
    g = gen(72)
    K8, N8 = -(-K // 8) * 8, -(-N // 8) * 8
    dy, w = rand(g, T, N, BF16, ld=N8 + pad), rand(g, N, K, BF16, N ** -0.5, ld=K8 + pad)
    x = rand(g, T, K, BF16, ld=K8 + pad)
    z = rand(g, T, K, F32)
    z[5, 40] = math.nan
    codes, scales = R.encode(z)
    dy[3, N - 1] = math.nan
    w[2, K - 1] = math.inf
    dx = torch.empty(T, K, device="cuda")
    L.loco_linear_backward_input(dy, w, dx)
    bad_is(dx, rows=(3,), cols=(K - 1,))
    L.loco_linear_backward_input(dy, w, dx, act=L.LOCO_ACT_GELU, codes=codes, scales=scales)
    want = torch.zeros(T, K, dtype=torch.bool, device="cuda")
    want[3], want[:, K - 1], want[5, 32:64] = True, True, True
    assert torch.equal(~torch.isfinite(dx), want)
    x[T - 1, 1] = math.inf
    dw, db = torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
    L.loco_linear_backward_weight(dy, dw, x=x, db=db)
    bad_is(dw, rows=(N - 1,), cols=(1,))
    bad_is(db, rows=(N - 1,))
