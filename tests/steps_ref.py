"""Joins, log probabilities and many-tensor optimizer steps by their definitions, and the rounding bounds that the GPU
tests hold the kernels to.

u = 2^-24 is the relative rounding error of one fp32 operation.  A sum of n terms in fp32 is off by at most (additions on
its longest chain) * u * sum |terms|.
"""
import math

import numpy as np
import torch

U = 2.0 ** -24
BLOCK = 256


def out_tol(exact, dtype):
    """Half a step of the output's type, relative to the value."""
    return exact.abs() * (torch.finfo(dtype).eps / 2)


def or64(t, other):
    return other if t is None else t.double()


# ---------------------------------------------------------------- joins

def norm_stats(v, kind, eps):
    """(mean, reciprocal root of the variance) of the rows of v (64 bits)."""
    m = v.mean(1) if kind == "layer" else torch.zeros(v.shape[0], dtype=torch.float64, device=v.device)
    return m, ((v - m[:, None]).square().mean(1) + eps).rsqrt()


def join_forward(x, y, kind, post, eps, a, s, gate=None, row_gate=None, post_gamma=None, post_beta=None):
    """(h, n, yh, m1, r1) in 64 bits."""
    y = y.double()
    if post:
        m1, r1 = norm_stats(y, kind, eps)
    else:
        m1, r1 = torch.zeros_like(y[:, 0]), torch.ones_like(y[:, 0])
    yh = (y - m1[:, None]) * r1[:, None]
    n = yh * or64(post_gamma, 1.0) + or64(post_beta, 0.0)
    w = or64(row_gate, torch.ones_like(m1))[:, None]
    return a * x.double() + s * w * or64(gate, 1.0) * n, n, yh, m1, r1


def through_norm(q, vh, r, kind):
    level = q.mean(1, keepdim=True) if kind == "layer" else 0.0
    return r[:, None] * (q - level - vh * (q * vh).mean(1, keepdim=True))


def join_backward(dh, du, h, y, stats, kind, post, a, s, gate=None, row_gate=None, gamma=None, post_gamma=None,
                  post_beta=None):
    """Every gradient in 64 bits, and what the bounds need."""
    m1, r1, m2, r2 = stats.double().unbind()
    rows, cols = y.shape
    zero = torch.zeros(rows, cols, dtype=torch.float64, device=y.device)
    yh = (y.double() - m1[:, None]) * r1[:, None] if post else y.double()
    hh = (h.double() - m2[:, None]) * r2[:, None] if du is not None else zero
    dud = zero if du is None else du.double()
    q = dud * or64(gamma, 1.0)
    t = or64(dh, zero) + (through_norm(q, hh, r2, kind) if du is not None else 0.0)
    w = or64(row_gate, torch.ones_like(m1))[:, None]
    g, pg = or64(gate, torch.ones(cols, dtype=torch.float64, device=y.device)), or64(post_gamma, 1.0)
    n = yh * pg + or64(post_beta, 0.0)
    c = s * w * g * t
    p = c * pg
    dy = through_norm(p, yh, r1, kind) if post else p
    return dict(dx=a * t, dy=dy, dgamma=(dud * hh).sum(0), dbeta=dud.sum(0), dpost_gamma=(c * yh).sum(0),
                dpost_beta=c.sum(0), dgate=(s * w * t * n).sum(0), drow_gate=(s * g * t * n).sum(1),
                t=t, q=q, hh=hh, yh=yh, n=n, c=c, p=p, w=w, g=g, pg=pg, r1=r1, r2=r2)


# ---------------------------------------------------------------- log probabilities

def logprob(z, targets, top):
    """(lse, logp, entropy, ids, alts, logp of every token) of the rows z (64 bits) by the definition."""
    rows, vocab = z.shape
    # in deviations from the maximum: the log of the sum is not lost beside rows of the type's lowest value
    m = z.amax(1, keepdim=True)
    empty = m[:, 0] == -math.inf
    d = z - torch.where(m == -math.inf, torch.zeros_like(m), m)
    ls = d.exp().sum(1).log()
    lse = torch.where(empty, -math.inf, m[:, 0] + ls)
    lse = torch.where((z == math.inf).any(1), math.nan, lse)
    logp = torch.where(empty[:, None], z, d - ls[:, None])
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
    entropy = torch.where(torch.isnan(lse), lse, entropy)
    at = logp.gather(1, targets.clamp(0, vocab - 1)[:, None])[:, 0]
    at = torch.where(targets < 0, torch.zeros_like(at), torch.where(targets >= vocab, math.nan, at))
    # values in order, the lower column first among equal ones: a stable sort
    order = torch.sort(z + 0.0, dim=1, descending=True, stable=True).indices[:, :top]
    alts = logp.gather(1, order)
    ids = torch.where(alts > -math.inf, order, -1)
    pad = top - order.shape[1]
    ids = torch.nn.functional.pad(ids, (0, pad), value=-1)
    alts = torch.nn.functional.pad(alts, (0, pad), value=-math.inf)
    bad = torch.isnan(lse)
    at = torch.where(bad & (targets >= 0), math.nan, at)
    return lse, at, entropy, torch.where(bad[:, None], -1, ids), torch.where(bad[:, None], math.nan, alts), logp


# ---------------------------------------------------------------- optimizer steps (fp32, in the stated order)

def f32(v):
    return float(np.float32(v))


def mix(x):
    """The hash behind the dither (32 bits in 64-bit integers)."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def random_bits(dither, t, i, n, device):
    e = torch.arange(n, device=device)
    key = mix(mix(mix(torch.tensor(dither, device=device)) ^ (t & 0xFFFFFFFF)) ^ i)
    return mix((e & 0xFFFFFFFF) ^ mix(key ^ (e >> 32)))


def blocks(v, fill=0):
    """[nb, 256] of a flat tensor."""
    return torch.nn.functional.pad(v, (0, -v.numel() % BLOCK), value=fill).view(-1, BLOCK)


def decode(codes, steps, second):
    v = codes.view(-1, BLOCK).float() * steps[:, None]
    return (v * v if second else v).view(-1)


def encode(value, most, bits, byte, least_one):
    """(codes as floats [nb, 256], steps) of the values [n]."""
    b = blocks(value)
    top = b.abs().amax(1, keepdim=True)      # NaN where a block holds one
    bad = ~torch.isfinite(top)
    whole = torch.full_like(top, most)       # (torch divides by a number through its reciprocal)
    inv = whole / top
    ok = ~bad & torch.isfinite(inv)
    x = b * torch.where(ok, inv, torch.zeros_like(inv))
    if bits is not None:
        x = x + (((blocks(bits) >> byte) & 255).float() - 127.5) * (1.0 / 256.0)
    q = torch.round(x)
    if least_one:
        q = torch.where(b > 0, q.clamp(min=1.0), q)
    q = torch.where(ok, q, torch.zeros_like(q))
    q.view(-1)[value.numel():] = 0.0
    step = torch.where(bad, math.nan, torch.where(ok, top / whole, torch.zeros_like(top)))
    return q, step[:, 0]


def adam(p, g, m, v, hp, t, lr_scale=1.0, decay_scale=1.0, grad_scale=None):
    """(p, m, v, sqrt(v)) in fp32 after one step, every product and sum rounded on its own."""
    lr, wd = f32(f32(hp.lr) * f32(lr_scale)), f32(f32(hp.weight_decay) * f32(decay_scale))
    b1, b2 = f32(hp.beta1), f32(hp.beta2)
    n1, n2 = f32(np.float32(1) - np.float32(b1)), f32(np.float32(1) - np.float32(b2))
    c1, c2 = lr, 1.0
    if hp.bias_correction:
        c1 = f32(lr / (1.0 - b1 ** t))
        bc2 = 1.0 - b2 ** t
        c2 = f32(1.0 / bc2) if hp.eps_inside_sqrt else f32(1.0 / math.sqrt(bc2))
    g = g.float()
    if grad_scale is not None:
        g = g * grad_scale
    p = p.float()
    p = p - f32(lr * wd) * p
    m = b1 * m + n1 * g
    v = b2 * v + n2 * (g * g)
    root = torch.sqrt(v)
    den = torch.sqrt(v * c2 + f32(hp.eps)) if hp.eps_inside_sqrt else root * c2 + f32(hp.eps)
    return p - c1 * (m / den), m, v, root


def to_bf16(p, bits=None):
    if bits is None:
        return p.to(torch.bfloat16)
    b = p.contiguous().view(torch.int32).to(torch.int64)
    return ((b + (bits >> 16)) & -65536).to(torch.int32).view(torch.float32).to(torch.bfloat16)
