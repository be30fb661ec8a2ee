"""The activations and their slopes relative to their own size, the tails included.

With u = 2^-24 and e the natural exponent that an activation takes (v for SiLU, v^2 / 2 for GELU, 2 sqrt(2/pi)
(v + 0.044715 v^3) for its tanh form), an exponential's relative error is its argument's absolute one: every
rounding on the way to the argument costs |e| u.  SiLU rounds once and has log2(e) to half a unit: 1.5 |e|.  GELU
squares, multiplies and has its constant to a quarter of a unit: 2.25 |e|.  The tanh form has a square, a sum of
products, a product, log2(e) and two constants: 6 |e|.  To that come the hardware's 2^x (4 u), 1 / x (2 u), a sum and
products (4 u), and for GELU what the quotient's error, tripled at most, and a polynomial of eight terms add (16 u).
"""
import math

import pytest
import torch

import layers_ref as R

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -100        # below it a result may come out as 0


@pytest.fixture(scope="module")
def L():
    from bit_gradient_compression_gb300 import loco
    return loco


def code(L, name):
    return getattr(L, "LOCO_ACT_" + name.upper())


def exponent(v, name):
    if name == "silu":
        return v.abs()
    if name == "gelu":
        return v * v / 2
    return 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3).abs()


def rel(v, name):
    per, const = {"silu": (1.5, 10), "gelu": (2.25, 26), "gelu_tanh": (6, 10)}[name]
    return (const + per * exponent(v, name)) * R.U


def cdf(v, name):
    """What the activation multiplies v by, without cancellation in the lower tail."""
    if name == "gelu":
        return 0.5 * torch.special.erfc(-v / math.sqrt(2))
    return torch.sigmoid(v if name == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))


def slope_terms(v, name):
    """The two terms of the slope."""
    p = cdf(v, name)
    if name == "gelu":
        return p, v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    q = torch.sigmoid(-v if name == "silu" else -2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    inner = 1.0 if name == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * v * v)
    return p, v * p * q * inner


def kept(rows):
    """A checkpoint of values from 2^-12 to 13, and they."""
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(-104, 105, (rows, 256), device="cuda", generator=g, dtype=torch.int32).to(torch.int8)
    scales = torch.tensor([124, 124, 124, 123, 123, 121, 119, 115], dtype=torch.uint8, device="cuda").repeat(rows, 1)
    return codes.contiguous(), scales.contiguous(), R.decode(codes, scales, 256)


NAMES = ["gelu", "gelu_tanh", "silu"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_values_of_a_checkpoint(L, name, dtype):
    codes, scales, v = kept(300)
    out = torch.empty(300, 256, dtype=dtype, device="cuda")
    L.loco_ckpt_decode(codes, scales, out, act=code(L, name))
    want = v * cdf(v, name)
    R.close(out, want, rel(v, name) * want.abs() + R.out_tol(want, dtype) + TINY, name)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("rows,cols", [(1, 2432), (5, 300), (300, 2000)])
def test_values_behind_a_product(L, name, rows, cols):
    """z is w's first column in every row."""
    x = torch.zeros(rows, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    w = torch.zeros(cols, 8, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = torch.linspace(-13, 13, cols, device="cuda")
    y = torch.empty(rows, cols, device="cuda")
    L.loco_linear_forward(x, w, y, act=code(L, name))
    v = w[:, 0].double().expand(rows, cols)
    want = v * cdf(v, name)
    R.close(y, want, rel(v, name) * want.abs() + R.out_tol(want, y.dtype) + TINY, name)


@pytest.mark.parametrize("name", NAMES)
def test_slopes(L, name):
    """dy w is 1 everywhere."""
    codes, scales, v = kept(300)
    dy = torch.zeros(300, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")
    dy[:, 0], w[0] = 1, 1
    dx = torch.empty(300, 256, device="cuda")
    L.loco_linear_backward_input(dy, w, dx, act=code(L, name), codes=codes, scales=scales)
    a, b = slope_terms(v, name)
    # the second term has a product or two more, and 1 - s in the place of the upper tail
    tol = 2 * rel(v, name) * (a + b.abs()) + TINY
    R.close(dx, a + b, tol + R.out_tol(a + b, dx.dtype), name)


@pytest.mark.parametrize("name", NAMES)
def test_ends(L, name):
    """Values beyond every tail, infinities and NaN: v or 0, and NaN where the formula has it."""
    x = torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    v = torch.tensor([-3e38, -1e20, -200.0, 200.0, 1e20, 3e38, math.inf, math.nan], device="cuda").to(torch.bfloat16)
    w = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = v
    y = torch.empty(1, 8, device="cuda")
    L.loco_linear_forward(x, w, y, act=code(L, name))
    got = y[0].tolist()
    assert got[:3] == [0, 0, 0] and got[3:6] == v[3:6].float().tolist()
    assert got[6] == math.inf and math.isnan(got[7])
