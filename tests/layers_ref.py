"""The layers' formulas in 64 bits, and the rounding bounds that the GPU tests hold the kernels to.

u = 2^-24 is the relative rounding error of one fp32 operation.  A sum of n terms in fp32 is off by
at most (number of additions on its longest chain) * u * sum |terms|.
"""
import math

import torch

U = 2.0 ** -24
BLOCK = 32


def out_tol(exact, dtype):
    """Half a unit in the last place of the output type."""
    return exact.abs() * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23)


def close(got, want, tol, what=""):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol)
    bad &= ~(torch.isnan(got) & torch.isnan(want))
    if bad.any():
        i = int(bad.flatten().nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at {i}: got "
                             f"{got.flatten()[i].item():.9g} want {want.flatten()[i].item():.9g} tol "
                             f"{torch.broadcast_to(tol, want.shape).flatten()[i].item():.3g}")


# ---------------------------------------------------------------- checkpoints

def encode(v):
    """codes [rows, nb*32] int8, scales [rows, nb] uint8 of the rows v (any float type), by the definition."""
    R, C = v.shape
    nb = -(-C // BLOCK)
    b = torch.zeros(R, nb * BLOCK, dtype=torch.float64, device=v.device)
    b[:, :C] = v.double()
    b = b.view(R, nb, BLOCK)
    a = b.abs().amax(2)                       # NaN where the block holds one
    bad = ~torch.isfinite(a)
    _, ex = torch.frexp(torch.where(bad, torch.ones_like(a), a))
    e = torch.where(a == 0, torch.full_like(ex, -126), (ex - 1 - 6).clamp(min=-126)).double()
    q = torch.round(b / torch.exp2(e)[..., None]).clamp(-127, 127)   # torch.round: halves to even
    q[bad] = 0
    s = torch.where(bad, torch.full_like(e, 255), e + 127)
    return q.to(torch.int8).reshape(R, nb * BLOCK), s.to(torch.uint8)


def decode(codes, scales, cols):
    R, nb = scales.shape
    step = torch.exp2(scales.double() - 127)
    step[scales == 255] = math.nan
    return (codes.view(R, nb, BLOCK).double() * step[..., None]).reshape(R, nb * BLOCK)[:, :cols]


def check_ckpt_of(codes, scales, v, err):
    """Codes and scales stand for rows near v (64 bits, each value known to within err): every value within half
    a step (a whole one where it saturates), every step the block's own."""
    R, C = v.shape
    nb = scales.shape[1]
    step = torch.exp2(scales.double() - 127)
    pad = torch.zeros(R, nb * BLOCK, dtype=torch.float64, device=v.device)
    pad[:, :C] = v
    perr = torch.zeros_like(pad)
    perr[:, :C] = torch.broadcast_to(err, v.shape)
    a, ae = pad.view(R, nb, BLOCK).abs().amax(2), perr.view(R, nb, BLOCK).amax(2)
    some = a > ae
    assert bool((a + ae >= 64 * step)[some & (scales > 1)].all()) and bool((a - ae < 128 * step)[some].all())
    wide = step.repeat_interleave(BLOCK, 1)
    got = codes.view(R, nb * BLOCK).double() * wide
    assert bool((got[:, C:] == 0).all())
    lim = wide * torch.where(pad.abs() + perr >= 127 * wide, 1.0, 0.5) + perr
    assert bool(((got - pad).abs() <= lim).all())
    assert int(codes.min()) >= -127


# ---------------------------------------------------------------- activations

def act(v, name):
    if name == "relu":
        return torch.relu(v)
    if name == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if name == "silu":
        return v / (1 + torch.exp(-v))
    return v


def act_slope(v, name):
    x = v.detach().clone().requires_grad_(True)
    act(x, name).sum().backward()
    return x.grad


# The fp32 activations: erff and __expf are off by at most 2 + |v| * 1.16 units, the quotient by 2, and
# the products by one each: below 2^-19 of |v| for the |v| <= 30 used here, and likewise for the slopes.
ACT_REL = 2.0 ** -19


# ---------------------------------------------------------------- norms

def norm_forward(x, kind, eps, gamma, beta):
    x = x.double()
    m = x.mean(1) if kind == "layer" else torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
    r = ((x - m[:, None]).square().mean(1) + eps).rsqrt()
    xh = (x - m[:, None]) * r[:, None]
    y = xh if gamma is None else xh * gamma.double()
    y = y if beta is None else y + beta.double()
    return m, r, xh, y


def norm_backward(dy, xh, r, kind, gamma, residual):
    dy = dy.double()
    g = dy if gamma is None else dy * gamma.double()
    c1 = g.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(g[:, :1])
    c2 = (g * xh).mean(1, keepdim=True)
    dx = r.double()[:, None] * (g - c1 - xh * c2)
    if residual is not None:
        dx = dx + residual.double()
    return dx, (dy * xh).sum(0), dy.sum(0)


# ---------------------------------------------------------------- products

def mm_tol(a, b):
    """Bound of |fp32 tensor-core a @ b - exact| (a [r, K], b [K, c]): K/16 + 16 accumulations, each of 17
    terms aligned to the largest and cut at 2^-24 of it: below 2^-21 of sum |a||b| each."""
    return (a.shape[1] / 16 + 16) * 2.0 ** -21 * (a.double().abs() @ b.double().abs())
