"""Gradient of logits whose log sum is so far from 0 that its 24 bits do not hold what the row adds to its largest logit,
or that it is infinite: rows of masks only, rows far from 0 (GPU)."""
import math

import pytest
import torch

import layers_ref as R
import steps_ref as S
from test_layers_gpu import F32, BF16, gen, guarded

pytestmark = pytest.mark.gpu
U, INF = S.U, math.inf


@pytest.fixture(scope="module")
def L():
    from bit_gradient_compression_gb300 import loco
    return loco


def far_rows(g, rows, vocab, dtype, ld):
    """Random rows, the first thirteen of which are far from 0 or masked, and their targets."""
    low = torch.finfo(dtype).min
    z = (torch.randn(rows * ld, generator=g, device="cuda") * 2.5).to(dtype).as_strided((rows, vocab), (ld, 1))
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    z[0] = low                      # nothing but the lowest value
    z[1] = low
    y[1] = -1                       # and no token given
    z[2] = low
    z[2, : vocab // 2] = -INF       # beside tokens that cannot come
    z[3] = -1e9
    z[4] = low
    z[4, vocab // 3] = 1.0          # an ordinary row
    for i, off in ((5, 3e4), (6, -5000.0), (7, 900.0), (8, -1100.0)):
        z[i] = (z[i].float() + off).to(dtype)
    z[9] = -INF                     # nothing is left
    z[10] = low / 2
    z[10, vocab - 1] = -low * 0.95
    z[10, 0] = -low * 0.9
    z[11, 1] = math.nan
    z[12] = -low * 0.95             # ties at the upper end
    return z, y


@pytest.mark.parametrize("vocab", [37, 1000, 1500, 33001])
@pytest.mark.parametrize("rows", [13, 700])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [1.0, 0.7, 1.5])
@pytest.mark.parametrize("which", ["both", "logp", "entropy"])
@pytest.mark.parametrize("ld,ldd", [(0, 0), (8, 5)])
def test_backward(L, vocab, rows, dtype, scale, which, ld, ldd):
    """With a scale of 1.5 the log sums of rows 0 to 2, 10 and 12 are infinite in 32 bits.

    Where |lse| is at most 1024, p's exponent is off by the rounding of z scale - lse, as in the tests of ordinary rows;
    else by that of deviations from the row's maximum: u for each of a difference, a product, a sum and a product with
    log2(e), itself off by u; and by that of the sum, vocab / 256 or 32 terms to a thread and 16 joins of terms that are
    off by 4 u and 4 u of their deviation.
    """
    g = gen(51)
    z, y = far_rows(g, rows, vocab, dtype, vocab + ld)
    f = lambda: torch.empty(rows, device="cuda")  # noqa: E731
    lse, h = f(), f()
    L.loco_logprob_forward(z, None, None, lse=lse, entropy=h, scale=scale)
    dlogp = torch.randn(rows, generator=g, device="cuda") if which != "entropy" else None
    dh = torch.randn(rows, generator=g, device="cuda") if which != "logp" else None
    kw = dict(dlogp=dlogp, entropy=h if dh is not None else None, dentropy=dh, scale=scale)
    out, intact = guarded(rows, vocab, dtype, vocab + ldd)
    L.loco_logprob_backward(z, y if dlogp is not None else None, lse, out, **kw)
    assert intact()
    assert torch.isnan(out).all(1).tolist() == [i == 11 for i in range(rows)]
    assert not out[9].any() and (which != "logp" or not out[1].any())

    fine = torch.arange(rows, device="cuda") != 11
    zz = z[fine].double() * scale
    lse64, _, _, _, _, logp = S.logprob(zz, y[fine], 1)
    some, h = lse64 > -INF, h[fine].double()
    p = torch.where(some[:, None], logp.exp(), 0.0)
    none = torch.zeros(len(zz), dtype=torch.float64, device="cuda")
    d = none if dlogp is None else torch.where((y[fine] >= 0) & some, dlogp[fine].double(), 0.0)
    e = none if dh is None else dh[fine].double()
    one = torch.zeros_like(zz).scatter_(1, y[fine].clamp(min=0)[:, None], 1.0)
    inner = torch.where(p > 0, logp + h[:, None], 0.0)
    want = scale * (d[:, None] * (one - p) - e[:, None] * p * inner)
    dev = torch.where(p > 0, -logp, 0.0)        # of the log sum
    far = 6 * U * dev + ((vocab / 256 + 48) * U + 4 * U + 4 * U * (p * dev).sum(1))[:, None]
    near = 3 * U * torch.where(p > 0, zz.abs() + lse64.abs()[:, None], 0.0)
    dt = torch.where((lse64.abs() <= 1025)[:, None], torch.maximum(near, far), far)
    each = p * (d.abs()[:, None] + e.abs()[:, None] * (dev + h.abs()[:, None]))
    tol = scale * ((dt + 12 * U) * each + p * e.abs()[:, None] * dt + 4 * U * one * d.abs()[:, None])
    R.close(out[fine], want, tol + 2 * U * want.abs() + S.out_tol(want, dtype), "dlogits")
    # in place of the logits: the same values
    L.loco_logprob_backward(z, y if dlogp is not None else None, lse, z, **kw)
    assert torch.equal(z.nan_to_num(3.0), out.nan_to_num(3.0))


def test_rows_of_masks_have_no_gradient_of_their_own(L):
    """Padded rows as a training step has them: every logit masked, no token given, entropies weighed alike."""
    for dtype in (F32, BF16):
        for value in (torch.finfo(dtype).min, -1e30, -1e9, -1e4):
            for vocab in (500, 5000):
                z = torch.full((3, vocab), value, device="cuda").to(dtype)
                y = torch.full((3,), -1, device="cuda")
                lse, h, d = torch.empty(3, device="cuda"), torch.empty(3, device="cuda"), torch.ones(3, device="cuda")
                L.loco_logprob_forward(z, None, None, lse=lse, entropy=h)
                out = torch.full_like(z, 7.0)
                L.loco_logprob_backward(z, y, lse, out, dlogp=d, entropy=h, dentropy=d)
                # p (log p + H) of 1/vocab and a difference of two logarithms, each off by a few roundings
                assert float(out.float().abs().max()) <= 64 * U * math.log(vocab) / vocab, (dtype, value, vocab)
