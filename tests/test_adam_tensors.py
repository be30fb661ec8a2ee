"""AdamW on many tensors: bit for bit the stated fp32 order, and near the 64-bit update (GPU)."""
import math

import pytest
import torch

import steps_ref as S
from test_layers_gpu import F32, BF16, gen

pytestmark = pytest.mark.gpu
U = S.U


@pytest.fixture(scope="module")
def L():
    from bit_gradient_compression_gb300 import loco
    return loco


def cut(g, n, dtype, sigma, off, positive=False):
    """n values `off` elements into a buffer whose other elements are 7."""
    buf = torch.full((off + n + 16,), 7.0, dtype=dtype, device="cuda")
    v = torch.randn(n, generator=g, device="cuda") * sigma
    buf[off:off + n] = (v * v if positive else v).to(dtype)
    return buf[off:off + n], buf


def same(a, b):
    """Equal bit for bit (NaN like NaN)."""
    a, b = a.reshape(-1), b.reshape(-1)
    if a.dtype.is_floating_point:
        view = torch.int32 if a.dtype == F32 else torch.int16
        return bool(((a.view(view) == b.view(view)) | (torch.isnan(a) & torch.isnan(b))).all())
    return torch.equal(a, b)


def build(L, sizes, bits, pd, gd, copy, dither, off, seed):
    g = gen(seed)
    p, gr, m, v, ms, vs, c, bufs = [], [], [], [], [], [], [], []
    for i, n in enumerate(sizes):
        nb = -(-n // S.BLOCK)
        sigma = 10.0 ** (-4 + i % 3)
        for to, dtype, sg in ((p, pd, 0.02), (gr, gd, sigma)):
            t, buf = cut(g, n, dtype, sg, off)
            to.append(t)
            bufs.append((buf, t))
        if copy:
            t, buf = cut(g, n, BF16, 0.0, off)
            c.append(t)
            bufs.append((buf, t))
        if bits == 32:
            for to, sq in ((m, False), (v, True)):
                t, buf = cut(g, n, F32, sigma, off, sq)
                to.append(t)
                bufs.append((buf, t))
        else:
            mc = torch.randint(-127, 128, (nb * S.BLOCK,), generator=g, device="cuda", dtype=torch.int8)
            vc = torch.randint(0, 256, (nb * S.BLOCK,), generator=g, device="cuda", dtype=torch.uint8)
            mc[n:], vc[n:] = 0, 0
            m.append(mc)
            v.append(vc)
            ms.append(torch.rand(nb, generator=g, device="cuda") * sigma / 127)
            vs.append(torch.rand(nb, generator=g, device="cuda") * sigma / 100)
    scales = [1.0 + i % 2 for i in range(len(sizes))]
    decay = [float(i % 3 != 1) for i in range(len(sizes))]
    eight = bits == 8
    t = L.make_adam_tensors(p, gr, m, v, m_steps=ms if eight else None, v_steps=vs if eight else None,
                            params_bf16=c if copy else None, lr_scales=scales, decay_scales=decay, dither=dither)
    return t, dict(p=p, g=gr, m=m, v=v, ms=ms, vs=vs, c=c, scales=scales, decay=decay, bufs=bufs)


def expect(st, i, bits, pd, hp, t, dither, grad_scale):
    """What tensor i of the list is after the step, from copies taken before it."""
    p, g = st["p"][i], st["g"][i]
    n = p.numel()
    m = st["m"][i] if bits == 32 else S.decode(st["m"][i], st["ms"][i], False)[:n]
    v = st["v"][i] if bits == 32 else S.decode(st["v"][i], st["vs"][i], True)[:n]
    scale = None if grad_scale is None else grad_scale
    p2, m2, v2, root = S.adam(p, g, m, v, hp, t, st["scales"][i], st["decay"][i], scale)
    r = S.random_bits(dither, t, i, n, "cuda") if dither else None
    want = {"p": p2 if pd == F32 else S.to_bf16(p2, r), "c": p2.to(BF16)}
    if bits == 32:
        return {**want, "m": m2, "v": v2}
    q, s = S.encode(m2, 127.0, r, 0, False)
    want["m"], want["ms"] = q.view(-1).to(torch.int8), s
    q, s = S.encode(root, 255.0, r, 8, True)
    want["v"], want["vs"] = q.view(-1).to(torch.uint8), s
    return want


def run_and_compare(L, sizes, bits, pd, gd, copy, dither, off, hp, t, grad_scale, seed=31, steps=2):
    tensors, st = build(L, sizes, bits, pd, gd, copy, dither, off, seed)
    scale = None if grad_scale is None else torch.tensor([grad_scale], device="cuda")
    for k in range(steps):
        want = [expect(st, i, bits, pd, hp, t + k, dither, scale) if n else None for i, n in enumerate(sizes)]
        L.loco_adam_tensors(tensors, hp, t + k, grad_scale=scale)
        for i, n in enumerate(sizes):
            if n == 0:
                continue
            names = ["p", "m", "v"] + (["ms", "vs"] if bits == 8 else []) + (["c"] if copy else [])
            for name in names:
                assert same(st[name][i], want[i][name]), (k, i, n, name)
    for buf, view in st["bufs"]:     # nothing around a tensor was written
        inside = torch.zeros_like(buf, dtype=torch.bool)
        lo = (view.data_ptr() - buf.data_ptr()) // buf.element_size()
        inside[lo:lo + view.numel()] = True
        assert bool((buf[~inside] == 7).all())
    return st


SIZES = [1, 2, 255, 256, 257, 0, 1000, 4096, 70001, 31]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pd,copy", [(F32, True), (F32, False), (BF16, False)])
@pytest.mark.parametrize("gd", [F32, BF16])
@pytest.mark.parametrize("dither", [0, 12345])
@pytest.mark.parametrize("off", [0, 1, 4])
def test_step_is_the_stated_one(L, bits, pd, copy, gd, dither, off):
    hp = L.make_adam(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    run_and_compare(L, SIZES, bits, pd, gd, copy, dither, off, hp, 3, 0.37)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("correct,inside", [(True, True), (False, False), (False, True)])
def test_conventions(L, bits, correct, inside):
    hp = L.make_adam(lr=1e-3, beta1=0.8, beta2=0.999, eps=1e-6, weight_decay=0.0, bias_correction=correct, eps_inside_sqrt=inside)
    run_and_compare(L, SIZES, bits, F32, BF16, True, 9, 0, hp, 1, None)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [24, 25, 384, 385, 900])
def test_many_tensors(L, bits, count):
    """Lists on both sides of what one launch takes, with empty tensors among them."""
    sizes = [(37 * i) % 700 for i in range(count)]
    run_and_compare(L, sizes, bits, F32, BF16, True, 5, 0, L.make_adam(), 2, None, steps=1)


def test_one_large_tensor(L):
    run_and_compare(L, [(1 << 26) + 37, 5], 8, F32, BF16, True, 3, 0, L.make_adam(), 2, None, steps=1)


def test_near_the_64_bit_update(L):
    """p against Algorithm 1's update in 64 bits: the rounding of a dozen operations."""
    g = gen(32)
    n, t = 100003, 5
    p, gr = torch.randn(n, generator=g, device="cuda"), torch.randn(n, generator=g, device="cuda") * 1e-3
    m, v = torch.randn(n, generator=g, device="cuda") * 1e-3, torch.rand(n, generator=g, device="cuda") * 1e-6 + 1e-8
    hp = L.make_adam(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    b1, b2 = S.f32(0.9), S.f32(0.95)
    m64, v64 = b1 * m.double() + (1 - b1) * gr.double(), b2 * v.double() + (1 - b2) * gr.double().square()
    step = S.f32(1e-2) * (m64 / (1 - b1 ** t)) / ((v64 / (1 - b2 ** t)).sqrt() + S.f32(1e-8))
    want = p.double() * (1 - S.f32(1e-2) * S.f32(0.1)) - step
    L.loco_adam_tensors(L.make_adam_tensors([p], [gr], [m], [v]), hp, t)
    # m's two terms may cancel: its error is 3 u of their sizes, which the quotient passes on
    terms = (m64.abs() + 2 * (1 - b1) * gr.double().abs()) / m64.abs().clamp(min=1e-30)
    tol = 3 * U * want.abs() + step.abs() * U * (12 + 4 * terms)
    assert bool(((p.double() - want).abs() <= tol).all())
    assert bool(((v.double() - v64).abs() <= 4 * U * v64).all())


@pytest.mark.parametrize("eps,inside", [(0.0, False), (1e-8, False), (1e-30, True)])
def test_every_root_and_quotient(L, eps, inside):
    """All 2^24 roots of [1, 4), so every denominator of [1, 2), under a numerator each: the IEEE operations' bits."""
    x = (torch.arange(1 << 24, device="cuda", dtype=torch.int32) + 0x3F800000).view(F32)
    hp = L.make_adam(lr=1.0, beta1=0.5, beta2=0.5, eps=eps, bias_correction=False, eps_inside_sqrt=inside)
    for k, scale in ((1, 1.0), (2, 2.0 ** -40), (3, 2.0 ** 40), (4, 2.0 ** -46), (5, 2.0 ** 50)):
        m = torch.rand(x.numel(), generator=gen(k), device="cuda") + 0.5 if k > 1 else torch.full_like(x, 2.0)
        p, z = torch.zeros_like(x), torch.zeros_like(x)
        v = x * (2.0 * scale * scale)       # halved by the step, exactly
        want = S.adam(p, z, m.clone(), v.clone(), hp, 1)
        L.loco_adam_tensors(L.make_adam_tensors([p], [z], [m], [v]), hp, 1)
        assert same(p, want[0]) and same(m, want[1]) and same(v, want[2])


@pytest.mark.parametrize("bits", [32, 8])
def test_every_exponent(L, bits):
    """Parameters, gradients and states of every exponent, subnormal ones and zeros of both signs among them."""
    n = 1 << 20
    g = gen(36)
    rand = lambda lo, hi: torch.ldexp(torch.rand(n, generator=g, device="cuda") + 0.5,  # noqa: E731
                                      torch.randint(lo, hi, (n,), generator=g, device="cuda"))
    sign = lambda: torch.randint(0, 2, (n,), generator=g, device="cuda") * 2.0 - 1.0  # noqa: E731
    p, gr = rand(-20, 3) * sign(), rand(-140, 60) * sign()
    p[::7], gr[::5], gr[1::5] = -0.0, 0.0, -0.0
    hp = L.make_adam(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    if bits == 32:
        m, v, kw = rand(-148, 60) * sign(), rand(-148, 100), {}
        m[::3], v[::3], m[1::9] = 0.0, 0.0, -0.0
    else:
        nb = n // 256
        m = torch.randint(-127, 128, (n,), generator=g, device="cuda", dtype=torch.int8)
        v = torch.randint(0, 256, (n,), generator=g, device="cuda", dtype=torch.uint8)
        kw = dict(m_steps=[rand(-140, 50)[:nb].contiguous()], v_steps=[rand(-74, 40)[:nb].contiguous()])
    for wide in (True, False):
        q, states = p.clone(), [m.clone(), v.clone()]
        steps = {k: [t[0].clone()] for k, t in kw.items()}
        st = dict(p=[q], g=[gr], m=states[:1], v=states[1:], ms=steps.get("m_steps"), vs=steps.get("v_steps"), scales=[1.0], decay=[1.0])
        if not wide:        # an odd place in its buffer
            buf = torch.zeros(n + 1, device="cuda")
            buf[1:] = q
            st["p"] = [buf[1:]]
        want = expect(st, 0, bits, F32, hp, 4, 21, None)
        L.loco_adam_tensors(L.make_adam_tensors(st["p"], [gr], states[:1], states[1:], dither=21, **steps), hp, 4)
        for name in ["p", "m", "v"] + (["ms", "vs"] if bits == 8 else []):
            assert same(st[name][0], want[name]), name


@pytest.mark.parametrize("bits", [32, 8])
def test_zeros_and_values_that_are_not_finite(L, bits):
    """Blocks of zeros stay zeros; a NaN or an infinity stays within its block of 256 of its tensor."""
    n = 256 * 6
    p, gr = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    gr[256] = math.nan
    gr[512] = math.inf
    gr[1024:1280] = 1e-30          # whose square is 0
    gr[1280:] = 1e-3
    if bits == 32:
        m, v, kw = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), {}
    else:
        m, v = torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
        kw = dict(m_steps=[torch.zeros(6, device="cuda")], v_steps=[torch.zeros(6, device="cuda")])
    L.loco_adam_tensors(L.make_adam_tensors([p], [gr], [m], [v], **kw), L.make_adam(lr=0.5), 1)
    zero = torch.ones(256, dtype=torch.bool, device="cuda")
    zero[0] = False
    assert bool((p[:256] == 1).all()) and bool((p[256:512][zero] == 1).all()) and bool((p[768:1024] == 1).all())
    assert bool(torch.isnan(p[256])) and bool(torch.isnan(p[512]))
    # ones step by lr; (1e-30 has m / eps left)
    assert bool(((p[1280:] - 0.5).abs() < 1e-4).all()) and bool(torch.isfinite(p[1024:1280]).all())
    if bits == 8:
        assert torch.isnan(kw["m_steps"][0]).tolist() == [False, True, True, False, False, False]
        assert not m[256:768].any() and not v[256:768].any() and not m[768:1024].any()
        assert bool((m[1280:] == 127).all()) and bool((v[1280:] == 255).all())
        out = torch.empty(n, device="cuda")
        L.loco_adam_state_decode(m, kw["m_steps"][0], out)
        assert bool(torch.isnan(out[256:768]).all()) and not out[:256].any()


def test_dither_is_right_on_average(L):
    """Of a state between two codes the stored values average to it: over many elements and steps within five standard
    errors of a rounding whose spread is at most half a step."""
    n = 1 << 20
    gr = torch.full((n,), 0.3217, device="cuda")
    gr[::256] = 1.0                # sets the step
    p = torch.zeros(n, device="cuda")
    m, v = torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    ms, vs = torch.zeros(n // 256, device="cuda"), torch.zeros(n // 256, device="cuda")
    L.loco_adam_tensors(L.make_adam_tensors([p], [gr], [m], [v], m_steps=[ms], v_steps=[vs], dither=77),
                        L.make_adam(beta1=0.0, beta2=0.0, bias_correction=False), 1)
    for codes, most in ((m, 127), (v, 255)):
        inner = codes.view(-1, 256)[:, 1:].double()
        x = S.f32(0.3217) * most
        assert set(inner.unique().tolist()) == {math.floor(x), math.ceil(x)}
        assert abs(float(inner.mean()) - x) <= 5 * 0.5 / math.sqrt(inner.numel()) + 1 / 512


def test_dither_differs_by_step_tensor_and_seed(L):
    n = 4096
    codes = []
    for seed, t in ((1, 1), (1, 2), (2, 1)):
        gr = [torch.linspace(0.0, 1.0, n, device="cuda") for _ in range(2)]
        z = lambda dtype, k: [torch.zeros(k, dtype=dtype, device="cuda") for _ in range(2)]  # noqa: E731
        m = z(torch.int8, n)
        L.loco_adam_tensors(L.make_adam_tensors(z(F32, n), gr, m, z(torch.uint8, n), m_steps=z(F32, 16), v_steps=z(F32, 16),
                                                dither=seed), L.make_adam(), t)
        codes += m
    for i in range(len(codes)):
        for j in range(i):
            share = float((codes[i] != codes[j]).double().mean())
            assert 0.2 < share < 0.5      # two independent roundings of a uniform fraction differ with probability 1/3


@pytest.mark.parametrize("n", [1, 255, 256, 1000, 70001])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("off", [0, 1])
def test_state_decode(L, n, dtype, off):
    g = gen(33)
    nb = -(-n // 256)
    steps = torch.rand(nb, generator=g, device="cuda")
    for codes in (torch.randint(-127, 128, (nb * 256,), generator=g, device="cuda", dtype=torch.int8),
                  torch.randint(0, 256, (nb * 256,), generator=g, device="cuda", dtype=torch.uint8)):
        buf = torch.full((n + off + 8,), 7.0, dtype=dtype, device="cuda")
        L.loco_adam_state_decode(codes, steps, buf[off:off + n])
        assert same(buf[off:off + n], S.decode(codes, steps, codes.dtype == torch.uint8)[:n].to(dtype))
        assert bool((buf[:off] == 7).all()) and bool((buf[off + n:] == 7).all())


def test_agrees_with_the_fused_step(L):
    """32-bit states on one rank's 8-bit bucket decoded to fp32: the same bits as decode and step in one."""
    n = 100001
    g = gen(34)
    grad = torch.randn(n, generator=g, device="cuda") * 1e-3
    cfg = L.make_config(bits=8, block=256)
    codes = torch.empty(L.loco_code_bytes(n, 8, 256), dtype=torch.uint8, device="cuda")
    scales, mean = torch.empty(L.loco_num_blocks(n, 256), device="cuda"), torch.empty(n, device="cuda")
    L.loco_compress(cfg, grad, torch.zeros(n, device="cuda"), 1, codes, scales)
    L.loco_decode_reduce(cfg, [codes], [scales], n, mean)
    a = [torch.randn(n, generator=g, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")]
    b = [t.clone() for t in a]
    hp = L.make_adam(lr=1e-3, weight_decay=0.1)
    L.loco_adam_step(cfg, [codes], [scales], n, *a, hp, 1)
    L.loco_adam_tensors(L.make_adam_tensors(b[:1], [mean], b[1:2], b[2:]), hp, 1)
    assert all(same(x, y) for x, y in zip(a, b))


def test_graph_replays_the_captured_step(L):
    tensors, st = build(L, [5000, 77], 8, F32, BF16, True, 3, 0, 35)
    hp = L.make_adam()
    L.loco_adam_tensors(tensors, hp, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        L.loco_adam_tensors(tensors, hp, 2)
    want = [expect(st, i, 8, F32, hp, 2, 3, None) for i in range(2)]
    graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        for name in ("p", "m", "v", "ms", "vs", "c"):
            assert same(st[name][i], want[i][name])
