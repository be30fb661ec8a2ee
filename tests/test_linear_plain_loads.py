"""Linear layers whose operands TMA cannot fetch, read by loader warps as they lie: tiles of every width, and clusters that
share k.  Large ones too, which a call copies to aligned rows first where there is memory for that: here there is none."""
import pytest
import torch

import test_layers_gpu as base
from test_layers_gpu import BF16, F32, L  # noqa: F401

pytestmark = pytest.mark.gpu

LAYOUTS = [("odd", 0), ("even", 1)]
# On 152 SMs, the tile's width and its split of k in the forward, input-gradient and weight-gradient products:
SHAPES = [(1500, 3001, 51),     # 256; 128 in 8; 192 in 8
          (8192, 2000, 16),     # 224; 224 in 4; 128 in 8
          (90, 2999, 1100),     # 64 in 2; 64 in 8; 192
          (81, 4100, 2049),     # 128 in 4; 128 in 8; 256
          (2500, 60, 1500),     # 160 in 8; 224; 64 in 8
          (1400, 1400, 130),    # 128; 160 in 8; 64 in 2
          (1000, 2900, 90)]     # 192; 64 in 8; 64 in 2
LARGE = [(2100, 4500, 320), (1100, 2300, 2056), (2304, 2060, 2500)]   # 160 and 192, split in 2 and 4


@pytest.fixture(autouse=True)
def no_memory_for_copies(monkeypatch, L):  # noqa: F811
    monkeypatch.setattr(L, "_scratch", lambda n: None)


@pytest.mark.parametrize("T,N,K", SHAPES + LARGE)
@pytest.mark.parametrize("layout,off", LAYOUTS)
@pytest.mark.parametrize("variant", [0, 1, 3])
def test_forward(L, T, N, K, layout, off, variant):  # noqa: F811
    base.test_linear_forward(L, T, N, K, layout, off, variant)


@pytest.mark.parametrize("T,N,K", SHAPES + LARGE)
@pytest.mark.parametrize("layout,off", LAYOUTS)
@pytest.mark.parametrize("variant", [0, 4])
def test_backward_input(L, T, N, K, layout, off, variant):  # noqa: F811
    base.test_linear_backward_input(L, T, N, K, layout, off, variant)


@pytest.mark.parametrize("T,N,K", SHAPES + LARGE)
@pytest.mark.parametrize("layout,off", LAYOUTS)
@pytest.mark.parametrize("source,od", [("x", F32), ("both", BF16)])
def test_backward_weight(L, T, N, K, layout, off, source, od):  # noqa: F811
    base.test_linear_backward_weight(L, T, N, K, layout, off, source, od)
