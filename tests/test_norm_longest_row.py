"""A row of as many columns as the library takes: counts of columns and blocks that do not fit 32 bits with their rounding."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [2 ** 31 - 1, 2 ** 31 - 31])
def test_forward(cols):
    """x alternates between 1 and -1: mean 0, deviation 1, every code at its end."""
    from bit_gradient_compression_gb300 import loco as L
    nb = -(-cols // 32)
    x = torch.ones(1, cols, dtype=torch.bfloat16, device="cuda")
    x[:, 1::2] = -1
    y, mean, rstd = torch.zeros_like(x), torch.full((1,), 7.0, device="cuda"), torch.full((1,), 7.0, device="cuda")
    codes = torch.zeros(1, nb * 32, dtype=torch.int8, device="cuda")
    scales = torch.zeros(1, nb, dtype=torch.uint8, device="cuda")
    L.loco_norm_forward(L.make_norm(eps=1e-5), x, None, None, y, mean=mean, rstd=rstd, codes=codes, scales=scales)
    assert abs(float(mean)) <= 2.0 ** -22 and abs(float(rstd) - (1 + 1e-5) ** -0.5) <= 2.0 ** -20
    assert torch.equal(y, x)                          # 0.999995 rounds to 1 in bf16
    assert bool((scales == 120).all())                # steps of 2^-7: the values saturate at 127 of them
    assert bool((codes[0, :cols:2] == 127).all()) and bool((codes[0, 1:cols:2] == -127).all())
    assert not codes[0, cols:].any()
