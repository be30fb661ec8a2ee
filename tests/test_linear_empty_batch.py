"""Weight gradients of no rows are zeros, whatever else is given."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
B = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    from bit_gradient_compression_gb300 import loco
    return loco


@pytest.mark.parametrize("source", ["x", "ckpt"])
@pytest.mark.parametrize("worst", [1.0, math.inf, math.nan])
@pytest.mark.parametrize("N,K", [(40, 16), (3, 5), (300, 520)])
def test_weight_gradient(L, source, worst, N, K):
    """gamma and beta are not read with x (and no workspace is needed then), nor without rows."""
    nb = -(-K // 32)
    dy = torch.empty(0, N, dtype=B, device="cuda")
    kw = dict(x=torch.empty(0, K, dtype=B, device="cuda"))
    if source == "ckpt":
        kw = dict(codes=torch.empty(0, nb * 32, dtype=torch.int8, device="cuda"),
                  scales=torch.empty(0, nb, dtype=torch.uint8, device="cuda"))
    gamma, beta = torch.full((K,), worst, device="cuda"), torch.full((K,), worst, device="cuda")
    dw, db = torch.full((N, K), 9.0, device="cuda"), torch.full((N,), 9.0, device="cuda")
    L.loco_linear_backward_weight(dy, dw, gamma=gamma, beta=beta, db=db, **kw)
    assert not dw.any() and not db.any()
