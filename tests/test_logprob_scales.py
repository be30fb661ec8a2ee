"""Scales of logits at both ends: refused where their product with log2(e) is infinite, right up to there."""
import math

import numpy as np
import pytest
import torch

import steps_ref as S
from test_steps_cpu import BAD, L, call  # noqa: F401 (L: a fixture)

LOG2E = np.float32(1.4426950408889634)
# the largest scale whose product with log2(e) is finite in fp32
LARGEST = float(np.float32(np.finfo(np.float32).max / np.float64(LOG2E)))


def test_the_largest_scale():
    with np.errstate(over="ignore"):
        assert np.isfinite(np.float32(LARGEST) * LOG2E)
        assert np.isinf(np.float32(LARGEST * (1 + 2.0 ** -20)) * LOG2E)


@pytest.mark.parametrize("name", ["loco_logprob_forward", "loco_logprob_backward"])
def test_scales_that_have_no_base_two(L, name):  # noqa: F811
    """(z - max) scale log2(e) of the largest logit would be 0 times infinity."""
    for scale in (2.4e38, float(np.finfo(np.float32).max)):
        got, said = call(L, name, scale=scale)
        assert got == BAD and "scale" in said, (got, said)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [LARGEST, 1e30, 1e-30, 1.2e-38, 1e-44])
@pytest.mark.parametrize("vocab", [300, 3000])
def test_scales_at_both_ends(L, scale, vocab):  # noqa: F811
    """A row whose logits are so far apart that one is left or so near that all are alike, and their gradient.

    Scaled logits are 0 or beyond 1e6 (one is left), or below 1e-6 (all alike to 1e-6): p is off by a few u and that."""
    z = torch.full((3, vocab), -5.0, device="cuda")
    z[:, 7], z[2, 9] = 0.0, 0.0
    y = torch.tensor([7, 3, 9], device="cuda")
    f = lambda: torch.empty(3, device="cuda")  # noqa: E731
    logp, lse, h, dz = f(), f(), f(), torch.empty_like(z)
    L.loco_logprob_forward(z, y, logp, lse=lse, entropy=h, scale=scale)
    want = S.logprob(z.double() * float(np.float32(scale)), y, 1)
    for got, w in ((logp, want[1]), (lse, want[0]), (h, want[2])):
        # (-5 scale passes fp32's range at the largest scale)
        assert bool((((got.double() - w).abs() <= 1e-5 * (1 + w.abs())) | (got == w.float())).all())
    d = torch.full((3,), min(1.0, 1.0 / scale), device="cuda")
    L.loco_logprob_backward(z, y, lse, dz, dlogp=d, scale=scale)
    p, one = want[5].exp(), torch.zeros_like(want[5]).scatter_(1, y[:, None], 1.0)
    exact = float(np.float32(scale)) * d.double()[:, None] * (one - p)
    assert bool(torch.isfinite(dz).all())
    assert float((dz.double() - exact).abs().max()) <= 1e-5 * float(scale * d.max()) + math.ldexp(1.0, -149)
