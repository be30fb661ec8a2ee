"""AdamW on many tensors where the second moment is infinite, or its root is: the stated step divides by infinity and
leaves the parameter alone but for its decay, whatever the first moment is (GPU)."""
import math

import pytest
import torch

from test_adam_tensors import expect, same
from test_layers_gpu import F32, BF16, gen

pytestmark = pytest.mark.gpu
INF = math.inf


@pytest.fixture(scope="module")
def L():
    from bit_gradient_compression_gb300 import loco
    return loco


def placed(values, off):
    """The values `off` elements into a buffer (an odd place takes no vectors)."""
    buf = torch.zeros(off + values.numel(), dtype=values.dtype, device="cuda")
    buf[off:] = values
    return buf[off:]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gd", [F32, BF16])
@pytest.mark.parametrize("pd", [F32, BF16])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("beta1", [0.9, 0.95, 0.99])
@pytest.mark.parametrize("correct,inside", [(True, False), (False, False), (True, True)])
def test_squares_that_overflow(L, bits, gd, pd, off, beta1, correct, inside):
    """Finite gradients of 1e18 to 3e20 among ordinary ones, then ordinary ones: every step is the stated one."""
    n = 256 * 5 + 77
    g = gen(61)
    grads = [torch.randn(n, generator=g, device="cuda") for _ in range(40)]
    for i, v in enumerate((1.9e19, -2e19, 3e20, 1e18, 1.85e19)):
        grads[0][i * 7 + 256: i * 7 + 259] = v
    grads[1][600] = -2.5e19
    p, gr = placed(torch.randn(n, generator=g, device="cuda").to(pd), off), placed(grads[0].to(gd), off)
    if bits == 32:
        m, v, kw = placed(torch.zeros(n, device="cuda"), off), placed(torch.zeros(n, device="cuda"), off), {}
    else:
        size = -(-n // 256) * 256
        m, v = torch.zeros(size, dtype=torch.int8, device="cuda"), torch.zeros(size, dtype=torch.uint8, device="cuda")
        kw = dict(m_steps=[torch.zeros(size // 256, device="cuda")], v_steps=[torch.zeros(size // 256, device="cuda")])
    st = dict(p=[p], g=[gr], m=[m], v=[v], ms=kw.get("m_steps"), vs=kw.get("v_steps"), scales=[1.0], decay=[1.0])
    tensors = L.make_adam_tensors([p], [gr], [m], [v], **kw)
    hp = L.make_adam(lr=1e-2, beta1=beta1, beta2=0.95, eps=1e-8, weight_decay=0.1, bias_correction=correct, eps_inside_sqrt=inside)
    for t, values in enumerate(grads, 1):
        gr.copy_(values.to(gd))
        want = expect(st, 0, bits, pd, hp, t, 0, None)
        if t == 1:
            assert bool(torch.isfinite(want["p"].float()).all())     # a NaN in them would be no test
        L.loco_adam_tensors(tensors, hp, t)
        for name in ["p", "m", "v"] + (["ms", "vs"] if bits == 8 else []):
            assert same(st[name][0], want[name]), (t, name)
    if bits == 32:
        assert bool(torch.isfinite(p.float()).all()) and bool(torch.isinf(v).any())


@pytest.mark.parametrize("m0", [0.0, -0.0, 1.0, -3e-5, 2.0 ** -70, 2.0 ** 61, 2.0 ** 59, INF, math.nan])
@pytest.mark.parametrize("v0", [INF, math.nan, 3.4e38, 2.0 ** 120, 2.0 ** 121, 1e38])
def test_states_of_the_upper_end(L, m0, v0):
    """Second moments that are infinite, NaN or near the largest number, with every kind of first moment."""
    n = 700
    p, gr = torch.randn(n, generator=gen(62), device="cuda"), torch.zeros(n, device="cuda")
    m, v = torch.full((n,), m0, device="cuda"), torch.full((n,), v0, device="cuda")
    m[::3], v[1::4] = 0.25, 0.5
    st = dict(p=[p], g=[gr], m=[m], v=[v], scales=[1.0], decay=[1.0])
    hp = L.make_adam(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    tensors = L.make_adam_tensors([p], [gr], [m], [v])
    for t in (5, 6):
        want = expect(st, 0, 32, F32, hp, t, 0, None)
        L.loco_adam_tensors(tensors, hp, t)
        for name in ("p", "m", "v"):
            assert same(st[name][0], want[name]), (t, name)
