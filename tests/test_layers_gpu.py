"""Norms, linear layers and 8-bit activation checkpoints against their formulas in 64 bits (GPU)."""
import itertools
import math

import pytest
import torch

import layers_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


@pytest.fixture(scope="module")
def L():
    from bit_gradient_compression_gb300 import loco
    return loco


def act_code(L, name):
    return {"none": L.LOCO_ACT_NONE, "relu": L.LOCO_ACT_RELU, "gelu": L.LOCO_ACT_GELU,
            "gelu_tanh": L.LOCO_ACT_GELU_TANH, "silu": L.LOCO_ACT_SILU}[name]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, rows, cols, dtype, sigma=1.0, ld=None, off=0):
    """[rows, cols] with row pitch ld, starting `off` elements into its buffer."""
    ld = ld or cols
    buf = (torch.randn(off + rows * ld + 8, generator=g, device="cuda") * sigma).to(dtype)
    return buf.as_strided((rows, cols), (ld, 1), off)


def guarded(rows, cols, dtype, ld=None, fill=7.0):
    """An output [rows, cols] inside a buffer of `fill`, and a check that nothing around it was written."""
    ld = ld or cols
    buf = torch.full((8 + rows * ld + 8,), fill, dtype=dtype, device="cuda")
    out = buf.as_strided((rows, cols), (ld, 1), 8)

    def intact():
        seen = torch.ones_like(buf, dtype=torch.bool)
        seen.as_strided((rows, cols), (ld, 1), 8).fill_(False)
        return bool((buf[seen] == fill).all())
    return out, intact


def new_ckpt(rows, cols):
    nb = -(-cols // 32)
    return (torch.full((rows, nb * 32), 99, dtype=torch.int8, device="cuda"),
            torch.full((rows, nb), 99, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------ checkpoints

SIZES = [(1, 1), (1, 32), (3, 31), (2, 33), (5, 64), (7, 100), (129, 1001), (64, 4096), (3, 20000)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ld,off", [(0, 0), (1, 0), (8, 0), (0, 1)])
def test_ckpt_round_trip_is_the_definition(L, rows, cols, dtype, ld, off):
    x = rand(gen(1), rows, cols, dtype, 3.0, cols + ld, off)
    if rows > 2:
        x[1] = 0.0
        x[2, : cols // 2] *= 1e-38     # steps at the bottom of the range, subnormal values
        x[0] *= 1e30
    codes, scales = new_ckpt(rows, cols)
    L.loco_ckpt_encode(x, codes, scales)
    wc, ws = R.encode(x)
    assert torch.equal(scales, ws) and torch.equal(codes, wc)
    want = R.decode(wc, ws, cols)
    for out_dtype, pad in itertools.product((F32, BF16), (0, 3)):
        out, intact = guarded(rows, cols, out_dtype, cols + pad)
        L.loco_ckpt_decode(codes, scales, out)
        assert torch.equal(out.double(), want) and intact()


def test_ckpt_rounding_and_saturation(L):
    """Ties go to even, the largest magnitudes saturate at 127 steps, -127 is the lowest code."""
    x = torch.zeros(2, 32, device="cuda")
    x[0, :8] = torch.tensor([64.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 127.0])
    x[1, :3] = torch.tensor([127.75, -127.75, 1.0])
    codes, scales = new_ckpt(2, 32)
    L.loco_ckpt_encode(x, codes, scales)
    assert codes[0, :8].tolist() == [64, 0, 2, 2, 0, -2, -2, 127]
    assert codes[1, :3].tolist() == [127, -127, 1] and scales.flatten().tolist() == [127, 127]


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("ld", [64, 65])
def test_ckpt_marks_blocks_that_are_not_finite(L, bad, ld):
    x = rand(gen(2), 3, 64, F32, 1.0, ld)
    x[1, 40] = bad
    codes, scales = new_ckpt(3, 64)
    L.loco_ckpt_encode(x, codes, scales)
    out = torch.empty(3, 64, device="cuda")
    L.loco_ckpt_decode(codes, scales, out)
    assert int(scales[1, 1]) == 255 and bool((codes[1, 32:] == 0).all())
    nan = torch.isnan(out)
    assert bool(nan[1, 32:].all()) and int(nan.sum()) == 32


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("affine", [None, "gamma", "both"])
def test_ckpt_decode_through_activation(L, name, out_dtype, affine):
    rows, cols = 9, 173
    g = gen(3)
    x = rand(g, rows, cols, F32, 4.0).clamp(-28, 28)
    codes, scales = R.encode(x)
    v = R.decode(codes, scales, cols)
    gamma = rand(g, 1, cols, BF16)[0].clamp(-1, 1) if affine else None
    beta = rand(g, 1, cols, BF16)[0].clamp(-1, 1) if affine == "both" else None
    w = v if gamma is None else v * gamma.double()
    w = w if beta is None else w + beta.double()
    out = torch.empty(rows, cols, dtype=out_dtype, device="cuda")
    L.loco_ckpt_decode(codes, scales, out, act=act_code(L, name), gamma=gamma, beta=beta)
    want = R.act(w, name)
    R.close(out, want, (R.ACT_REL + 4 * R.U) * (w.abs() + v.abs()) + R.out_tol(want, out_dtype), name)


# ------------------------------------------------------------------ norms

NORM_SIZES = [(1, 1), (1, 8), (2, 31), (5, 256), (3, 257), (9, 1000), (300, 1024), (4, 2047), (33, 2048), (17, 4096),
              (2, 5632), (3, 8200), (2, 16384), (2, 17001)]
STRIDES = [0, 1, 8]


def norm_inputs(seed, rows, cols, xd, pad):
    g = gen(seed)
    x = rand(g, rows, cols, xd, 2.0, cols + pad)
    x += 1.5
    if rows > 1:
        x[rows - 1] = 0.0
    return g, x


@pytest.mark.parametrize("rows,cols", NORM_SIZES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("xd,yd,pd", [(F32, F32, F32), (BF16, BF16, BF16), (F32, BF16, BF16), (BF16, F32, F32)])
@pytest.mark.parametrize("pad", STRIDES)
def test_norm_forward(L, rows, cols, kind, xd, yd, pd, pad):
    g, x = norm_inputs(4, rows, cols, xd, pad)
    gamma, beta = rand(g, 1, cols, pd)[0], rand(g, 1, cols, pd)[0]
    eps = 1e-5
    m, r, xh, want = R.norm_forward(x, kind, eps, gamma, beta)
    y, intact = guarded(rows, cols, yd, cols + pad)
    mean, rstd = torch.full((rows,), 5.0, device="cuda"), torch.empty(rows, device="cuda")
    codes, scales = new_ckpt(rows, cols)
    cfg = L.make_norm(L.LOCO_NORM_LAYER if kind == "layer" else L.LOCO_NORM_RMS, eps)
    L.loco_norm_forward(cfg, x, gamma, beta, y, mean=mean, rstd=rstd, codes=codes, scales=scales)
    # at most 64 additions lie on a chain of either sum (long rows: one per 512 columns and 10)
    n = 64 + cols / 512
    top = x.double().abs().amax(1)
    if kind == "layer":
        R.close(mean, m, n * R.U * top, "mean")
    else:
        assert bool((mean == 5.0).all())          # not written
    # the mean's error moves every x - m alike, which is second order in the variance
    rel = n * R.U + (n * R.U * top * r) ** 2 + 4 * R.U * top * r
    R.close(rstd, r, rel * r, "rstd")
    err = (n * R.U * top * r + rel * xh.abs().amax(1))[:, None]
    tol = err * gamma.double().abs() + 4 * R.U * (want.abs() + beta.double().abs())
    R.close(y, want, tol + R.out_tol(want, yd), "y")
    assert intact()
    R.check_ckpt_of(codes, scales, xh, err)
    # without parameters, statistics and checkpoint
    y2, intact = guarded(rows, cols, yd, cols + pad)
    L.loco_norm_forward(cfg, x, None, None, y2)
    R.close(y2, xh, err + R.out_tol(xh, yd), "plain y")
    assert intact()


@pytest.mark.parametrize("rows,cols", NORM_SIZES + [(700, 96), (1300, 64)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("source", ["x", "ckpt"])
@pytest.mark.parametrize("xd,yd,gd", [(F32, F32, F32), (BF16, BF16, BF16), (F32, BF16, BF16)])
@pytest.mark.parametrize("pad", STRIDES)
def test_norm_backward(L, rows, cols, kind, source, xd, yd, gd, pad):
    g, x = norm_inputs(5, rows, cols, xd, pad)
    gamma = rand(g, 1, cols, BF16)[0]
    dy = rand(g, rows, cols, yd, 0.1, cols + pad)
    residual = rand(g, rows, cols, xd, 0.1, cols + pad) if pad != 8 else None
    m, r, xh, _ = R.norm_forward(x, kind, 1e-5, None, None)
    mean, rstd = m.float(), r.float()
    codes = scales = None
    if source == "ckpt":
        codes, scales = R.encode(xh)
        xh = R.decode(codes, scales, cols)
        amp = xh.abs().amax(1, keepdim=True)
    else:
        mm = mean.double()[:, None] if kind == "layer" else 0.0
        xh = (x.double() - mm) * rstd.double()[:, None]
        amp = (x.double().abs().amax(1) * r)[:, None]
    want, wdg, wdb = R.norm_backward(dy, xh, rstd, kind, gamma, residual)
    cfg = L.make_norm(L.LOCO_NORM_LAYER if kind == "layer" else L.LOCO_NORM_RMS, 1e-5)
    dx, intact = guarded(rows, cols, xd, cols + pad)
    dgamma, dbeta = torch.empty(cols, dtype=gd, device="cuda"), torch.empty(cols, dtype=gd, device="cuda")
    ws = torch.empty(L.loco_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    kw = dict(x=x if source == "x" else None, mean=mean if kind == "layer" else None, codes=codes, scales=scales)
    L.loco_norm_backward(cfg, dy, gamma, rstd, dx, residual=residual, dgamma=dgamma, dbeta=dbeta, workspace=ws, **kw)
    gg = (dy.double() * gamma.double()).abs()
    s1, s2 = gg.mean(1, keepdim=True), (gg * xh.abs()).mean(1, keepdim=True)
    n = 64 + cols / 512
    tol = n * R.U * rstd.double()[:, None] * (gg + s1 + (xh.abs() + amp) * (s2 + amp * s1))
    R.close(dx, want, tol + 4 * R.U * want.abs() + R.out_tol(want, xd), "dx")
    assert intact()
    both = (dy.double().abs() * (xh.abs() + 4 * R.U * amp)).sum(0)
    R.close(dgamma, wdg, (rows + 64) * R.U * both + 4 * R.U * (dy.double().abs() * amp).sum(0) + R.out_tol(wdg, gd), "dgamma")
    R.close(dbeta, wdb, (rows + 64) * R.U * dy.double().abs().sum(0) + R.out_tol(wdb, gd), "dbeta")
    # dx over the residual, without the parameters' gradients; the same values
    if residual is not None:
        again = residual.clone() if pad == 0 else residual
        L.loco_norm_backward(cfg, dy, gamma, rstd, again, residual=again, **kw)
        assert torch.equal(again, dx)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradient_against_differences(L, kind):
    """<dx, v> is the directional difference quotient of the 64-bit loss sum(y * c); likewise gamma and beta."""
    rows, cols = 11, 75
    g = gen(6)
    x, gamma, beta, c, v = (rand(g, r, cols, F32) for r in (rows, 1, 1, rows, rows))
    vg, vb = rand(g, 1, cols, F32), rand(g, 1, cols, F32)
    loss = lambda t: float((R.norm_forward(x.double() + t * v.double(), kind, 1e-5, gamma[0].double() + t * vg[0].double(),
                                           beta[0].double() + t * vb[0].double())[3] * c.double()).sum())
    h = 1e-5
    want = (loss(h) - loss(-h)) / (2 * h)
    cfg = L.make_norm(L.LOCO_NORM_LAYER if kind == "layer" else L.LOCO_NORM_RMS, 1e-5)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd, dg, db = (torch.empty(n, device="cuda") for n in (rows, rows, cols, cols))
    ws = torch.empty(L.loco_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    L.loco_norm_forward(cfg, x, gamma[0], beta[0], y, mean=mean, rstd=rstd)
    L.loco_norm_backward(cfg, c, gamma[0], rstd, dx, x=x, mean=mean if kind == "layer" else None, dgamma=dg, dbeta=db,
                         workspace=ws)
    got = float((dx.double() * v.double()).sum() + (dg.double() * vg[0].double()).sum() + (db.double() * vb[0].double()).sum())
    scale = float((dx.double() * v.double()).abs().sum() + (dg.double() * vg[0].double()).abs().sum())
    assert abs(got - want) <= 1e-5 * scale


def test_norm_empty_batch(L):
    cfg = L.make_norm()
    e = torch.empty(0, 40, device="cuda")
    r = torch.empty(0, device="cuda")
    L.loco_norm_forward(cfg, e, None, None, torch.empty(0, 40, device="cuda"), rstd=r)
    dg, db = torch.ones(40, device="cuda"), torch.ones(40, device="cuda")
    L.loco_norm_backward(cfg, e, None, r, torch.empty(0, 40, device="cuda"), x=e, mean=r, dgamma=dg, dbeta=db)
    assert not dg.any() and not db.any()


@pytest.mark.parametrize("cols,pad", [(96, 0), (96, 1), (4096, 0)])
def test_norm_nan_stays_in_its_row(L, cols, pad):
    g, x = norm_inputs(7, 6, cols, F32, pad)
    x[2, 5] = math.nan
    y = torch.empty(6, cols, device="cuda")
    codes, scales = new_ckpt(6, cols)
    L.loco_norm_forward(L.make_norm(), x, None, None, y, codes=codes, scales=scales)
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isfinite(y[[0, 1, 3, 4, 5]]).all())
    assert bool((scales[2] == 255).all()) and not bool((scales[[0, 1, 3, 4, 5]] == 255).any())


# ------------------------------------------------------------------ linear layers

LIN = [(1, 1, 1), (3, 7, 5), (1, 130, 64), (16, 128, 64), (17, 129, 65), (33, 257, 200), (64, 96, 72), (5, 4100, 512),
       (130, 384, 1024), (200, 31, 2049), (512, 256, 2048), (1000, 520, 136), (2100, 4500, 320)]
# products long enough in every direction for pairs of CTAs, several tiles each, ragged at every edge
LIN_FEW = [(1, 4096, 520), (2, 2500, 1027), (4, 2432, 264), (5, 4100, 40), (8, 3000, 512), (7, 2440, 9), (9, 4096, 520)]
LIN_LARGE = [(1100, 2300, 2056), (2304, 2060, 2500)]
# row pitches beyond the width, offset of the first element: TMA takes the first, plain loads the rest
LAYOUTS = [("even", 0), ("odd", 0), ("even", 1)]


def pitch(cols, layout):
    return -(-cols // 8) * 8 + (0 if layout == "even" else 1 if cols % 2 else 3)


def linear_forward_ref(x, w, bias, name, residual):
    z = x.double() @ w.double().t()
    tol = R.mm_tol(x, w.t())
    if bias is not None:
        z = z + bias.double()
        tol = tol + 2 * R.U * z.abs()
    y = R.act(z, name)
    ytol = 1.2 * tol + R.ACT_REL * z.abs() * (name not in ("none", "relu"))
    if residual is not None:
        y = y + residual.double()
        ytol = ytol + 2 * R.U * y.abs()
    return z, tol, y, ytol


@pytest.mark.parametrize("T,N,K", LIN + LIN_FEW + LIN_LARGE)
@pytest.mark.parametrize("layout,off", LAYOUTS)
@pytest.mark.parametrize("variant", range(5))
def test_linear_forward(L, T, N, K, layout, off, variant):
    g = gen(8 + variant)
    name = ACTS[variant]
    od = (F32, BF16)[variant % 2]
    x = rand(g, T, K, BF16, 1.0, pitch(K, layout), off)
    w = rand(g, N, K, BF16, K ** -0.5, pitch(K, layout), off)
    bias = rand(g, 1, N, (BF16, F32)[variant % 2])[0] if variant != 1 else None
    residual = rand(g, T, N, od, 1.0, N + off) if variant in (1, 2, 4) else None
    save = variant != 3
    codes, scales = new_ckpt(T, N) if save else (None, None)
    y, intact = guarded(T, N, od, N + (3 if layout == "odd" else 0))
    L.loco_linear_forward(x, w, y, act=act_code(L, name), bias=bias, residual=residual, codes=codes, scales=scales)
    z, tol, want, ytol = linear_forward_ref(x, w, bias, name, residual)
    R.close(y, want, ytol + R.out_tol(want, od), "y")
    assert intact()
    if save:
        R.check_ckpt_of(codes, scales, z, tol)
    if residual is not None:   # over the residual
        buf = residual.clone() if off == 0 else residual
        L.loco_linear_forward(x, w, buf, act=act_code(L, name), bias=bias, residual=buf)
        assert torch.equal(buf, y)
    assert L.loco_linear_timeouts() == 0


@pytest.mark.parametrize("T,N,K", LIN + LIN_LARGE)
@pytest.mark.parametrize("layout,off", LAYOUTS)
@pytest.mark.parametrize("variant", range(5))
def test_linear_backward_input(L, T, N, K, layout, off, variant):
    g = gen(20 + variant)
    name = ACTS[variant]
    od = (F32, BF16)[variant % 2]
    dy = rand(g, T, N, BF16, 1.0, pitch(N, layout), off)
    w = rand(g, N, K, BF16, K ** -0.5, pitch(K, layout), off)
    residual = rand(g, T, K, od, 1.0, K + off) if variant in (1, 2, 4) else None
    codes = scales = None
    slope = 1.0
    if name != "none":
        codes, scales = R.encode(rand(g, T, K, F32, 2.0).clamp(-25, 25))
        slope = R.act_slope(R.decode(codes, scales, K), name)
    dx, intact = guarded(T, K, od, K + (3 if layout == "odd" else 0))
    L.loco_linear_backward_input(dy, w, dx, act=act_code(L, name), codes=codes, scales=scales, residual=residual)
    p = dy.double() @ w.double()
    want = p * slope
    tol = R.mm_tol(dy, w) * 1.2 + 30 * R.ACT_REL * p.abs() * (name not in ("none", "relu"))
    if residual is not None:
        want = want + residual.double()
        tol = tol + 2 * R.U * want.abs()
    R.close(dx, want, tol + R.out_tol(want, od), "dx")
    assert intact()
    if residual is not None:
        buf = residual.clone() if off == 0 else residual
        L.loco_linear_backward_input(dy, w, buf, act=act_code(L, name), codes=codes, scales=scales, residual=buf)
        assert torch.equal(buf, dx)
    assert L.loco_linear_timeouts() == 0


@pytest.mark.parametrize("T,N,K", LIN + LIN_LARGE)
@pytest.mark.parametrize("layout,off", LAYOUTS)
@pytest.mark.parametrize("source", ["x", "ckpt", "gamma", "beta", "both"])
@pytest.mark.parametrize("od", [F32, BF16])
def test_linear_backward_weight(L, T, N, K, layout, off, source, od):
    g = gen(30)
    dy = rand(g, T, N, BF16, 1.0, pitch(N, layout), off)
    codes = scales = x = None
    gamma = rand(g, 1, K, F32)[0] if source in ("gamma", "both") else None
    beta = rand(g, 1, K, F32)[0] if source in ("beta", "both") else None
    if source == "x":
        x = rand(g, T, K, BF16, 1.0, pitch(K, layout), off)
        v = x.double()
    else:
        codes, scales = R.encode(rand(g, T, K, F32))
        v = R.decode(codes, scales, K)
    dw, intact = guarded(N, K, od, K + (3 if layout == "odd" else 0))
    db, db_intact = guarded(1, N, od)
    ws = torch.empty(L.loco_linear_workspace_bytes(N), dtype=torch.uint8, device="cuda")
    L.loco_linear_backward_weight(dy, dw, x=x, codes=codes, scales=scales, gamma=gamma, beta=beta, db=db[0], workspace=ws)
    s = dy.double().sum(0)
    stol = (T / 16 + 64) * R.U * dy.double().abs().sum(0)
    want, tol = dy.double().t() @ v, R.mm_tol(dy.t(), v)
    if gamma is not None:
        want, tol = want * gamma.double(), tol * gamma.double().abs()
    if beta is not None:
        want = want + s[:, None] * beta.double()
        tol = tol + stol[:, None] * beta.double().abs()
    R.close(dw, want, tol + 4 * R.U * (want.abs() + tol) + R.out_tol(want, od), "dw")
    R.close(db[0], s, stol + R.out_tol(s, od), "db")
    assert intact() and db_intact()
    assert L.loco_linear_timeouts() == 0


def test_linear_gradient_against_differences(L):
    """Difference quotients of the 64-bit loss sum(silu(x w^T + b) * c) along a direction of x, w and b."""
    T, N, K = 37, 50, 61
    g = gen(40)
    x, w = rand(g, T, K, BF16), rand(g, N, K, BF16, K ** -0.5)
    b, vb = rand(g, 1, N, F32)[0], rand(g, 1, N, F32)[0]
    c, vx, vw = rand(g, T, N, F32), rand(g, T, K, F32), rand(g, N, K, F32, K ** -0.5)
    loss = lambda t: float((R.act((x.double() + t * vx.double()) @ (w.double() + t * vw.double()).t() + b.double() +
                                  t * vb.double(), "silu") * c.double()).sum())
    h = 1e-5
    want = (loss(h) - loss(-h)) / (2 * h)
    # dz by the formula from the 64-bit z, rounded to the bf16 that the kernels take
    z = x.double() @ w.double().t() + b.double()
    dz64 = c.double() * R.act_slope(z, "silu")
    dz = dz64.to(BF16)
    dx, dw, db = torch.empty(T, K, device="cuda"), torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
    L.loco_linear_backward_input(dz, w, dx)
    L.loco_linear_backward_weight(dz, dw, x=x, db=db)
    terms = [(dx.double() * vx.double()), (dw.double() * vw.double()), (db.double() * vb.double())]
    got = sum(float(t.sum()) for t in terms)
    # rounding dz moves <dz, dz/dt> by at most 2^-9 of the sum of its terms' magnitudes
    dzdt = vx.double() @ w.double().t() + x.double() @ vw.double().t() + vb.double()
    assert abs(got - want) <= 2.0 ** -9 * float((dz64 * dzdt).abs().sum()) + 1e-6 * abs(want)


def test_linear_slope_against_differences(L):
    """The activation slope in the input gradient is the difference quotient of the activation at the kept values."""
    T, K = 40, 96
    g = gen(41)
    codes, scales = R.encode(rand(g, T, K, F32, 2.0))
    z = R.decode(codes, scales, K)
    dy = torch.eye(K, device="cuda")[:T].to(BF16).contiguous()      # dy w = the first T rows of w
    w = torch.ones(K, K, dtype=BF16, device="cuda")
    for name in ("gelu", "gelu_tanh", "silu"):
        dx = torch.empty(T, K, device="cuda")
        L.loco_linear_backward_input(dy, w, dx, act=act_code(L, name), codes=codes, scales=scales)
        want = (R.act(z + 1e-6, name) - R.act(z - 1e-6, name)) / 2e-6
        R.close(dx, want, torch.full_like(want, 2e-5), name)


def test_linear_empty(L):
    one = lambda *s: torch.ones(*s, dtype=BF16, device="cuda")
    y = torch.full((4, 40), 9.0, device="cuda")
    L.loco_linear_forward(one(4, 0), one(40, 0), y, act=L.LOCO_ACT_RELU, bias=one(40))      # K = 0: act(bias)
    assert bool((y == 1).all())
    L.loco_linear_forward(one(0, 16), one(40, 16), torch.empty(0, 40, device="cuda"))
    dx = torch.full((4, 16), 9.0, device="cuda")
    L.loco_linear_backward_input(one(4, 0), one(0, 16), dx)
    assert not dx.any()
    dw, db = torch.full((40, 16), 9.0, device="cuda"), torch.full((40,), 9.0, device="cuda")
    L.loco_linear_backward_weight(one(0, 40), dw, x=one(0, 16), db=db)
    assert not dw.any() and not db.any()
    dw.fill_(9.0)
    c, s = torch.empty(0, 32, dtype=torch.int8, device="cuda"), torch.empty(0, 1, dtype=torch.uint8, device="cuda")
    ws = torch.empty(L.loco_linear_workspace_bytes(40), dtype=torch.uint8, device="cuda")
    L.loco_linear_backward_weight(one(0, 40), dw, codes=c, scales=s, gamma=one(16), beta=one(16), db=db, workspace=ws)
    assert not dw.any()


@pytest.mark.parametrize("K", [64, 65])
def test_linear_nan_reaches_only_what_reads_it(L, K):
    g = gen(42)
    x, w = rand(g, 20, K, BF16), rand(g, 70, K, BF16)
    x[3, 1] = math.nan
    x[5, 2] = math.inf
    w[9, 4] = math.nan
    y = torch.empty(20, 70, device="cuda")
    L.loco_linear_forward(x, w, y)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[3] = want[5] = True
    want[:, 9] = True
    assert torch.equal(bad, want)
    # a bad block of a checkpoint: its 32 columns of dw
    v = rand(g, 20, 70, F32)
    v[7, 33] = math.inf
    codes, scales = R.encode(v)
    dw = torch.empty(K, 70, device="cuda")
    dy = rand(g, 20, K, BF16)
    L.loco_linear_backward_weight(dy, dw, codes=codes, scales=scales)
    nan = torch.isnan(dw)
    assert bool(nan[:, 32:64].all()) and not bool(nan[:, :32].any()) and not bool(nan[:, 64:].any())


def test_outputs_into_slices_of_a_bucket(L):
    """Gradients written at odd offsets of one flat bf16 bucket, as a data-parallel step keeps them."""
    T, N, K = 48, 37, 53
    g = gen(43)
    dy, x = rand(g, T, N, BF16), rand(g, T, K, BF16)
    bucket = torch.full((3 + N + N * K + 5,), 7.0, dtype=BF16, device="cuda")
    db, dw = bucket[3:3 + N], bucket[3 + N:3 + N + N * K].view(N, K)
    L.loco_linear_backward_weight(dy, dw, x=x, db=db)
    ref_dw, ref_db = torch.empty(N, K, dtype=BF16, device="cuda"), torch.empty(N, dtype=BF16, device="cuda")
    L.loco_linear_backward_weight(dy, ref_dw, x=x, db=ref_db)
    assert torch.equal(dw, ref_dw) and torch.equal(db, ref_db)
    assert bool((bucket[:3] == 7).all()) and bool((bucket[-5:] == 7).all())


def test_column_views_of_one_buffer(L):
    """Input and output side by side in a wider matrix do not overlap; crossing columns are refused."""
    buf = torch.randn(6, 96, device="cuda")
    x, y = buf[:, :40], buf[:, 48:88]
    want = R.norm_forward(x.clone(), "layer", 1e-5, None, None)[3]
    L.loco_norm_forward(L.make_norm(), x, None, None, y)
    R.close(y, want, 1e-4 + 0 * want)
    with pytest.raises(L.LocoError) as e:
        L.loco_norm_forward(L.make_norm(), x, None, None, buf[:, 39:79])
    assert e.value.status == L.LOCO_ERR_INVALID_ARG


def step_all(L, st):
    cfg = L.make_norm(L.LOCO_NORM_LAYER)
    L.loco_norm_forward(cfg, st["x"], st["gamma"], st["beta"], st["y"], mean=st["mean"], rstd=st["rstd"],
                        codes=st["c1"], scales=st["s1"])
    L.loco_linear_forward(st["y"], st["w"], st["h"], act=L.LOCO_ACT_GELU, bias=st["b"], codes=st["c2"], scales=st["s2"])
    L.loco_ckpt_decode(st["c2"], st["s2"], st["h2"], act=L.LOCO_ACT_GELU)
    L.loco_linear_backward_input(st["dout"], st["w2"], st["dz"], act=L.LOCO_ACT_GELU, codes=st["c2"], scales=st["s2"])
    L.loco_linear_backward_weight(st["dz"], st["dw"], codes=st["c1"], scales=st["s1"], gamma=st["gamma"],
                                  beta=st["beta"], db=st["db"], workspace=st["ws"])
    L.loco_linear_backward_input(st["dz"], st["w"], st["dy"])
    L.loco_norm_backward(cfg, st["dy"], st["gamma"], st["rstd"], st["dx"], codes=st["c1"], scales=st["s1"],
                         residual=st["dout"], dgamma=st["dgamma"], dbeta=st["dbeta"], workspace=st["ws2"])
    return {k: st[k] for k in ("h", "h2", "dw", "db", "dx", "dgamma", "dbeta", "c1", "s1", "c2", "s2")}


def step_state(L, T=300, K=200, N=456, seed=50):
    g = gen(seed)
    e = lambda *s, d=BF16: torch.empty(*s, dtype=d, device="cuda")
    st = dict(x=rand(g, T, K, BF16), gamma=rand(g, 1, K, BF16)[0], beta=rand(g, 1, K, BF16)[0],
              w=rand(g, N, K, BF16, K ** -0.5), b=rand(g, 1, N, BF16)[0], w2=rand(g, K, N, BF16, N ** -0.5),
              dout=rand(g, T, K, BF16))
    st["c1"], st["s1"] = new_ckpt(T, K)
    st["c2"], st["s2"] = new_ckpt(T, N)
    st.update(y=e(T, K), mean=e(T, d=F32), rstd=e(T, d=F32), h=e(T, N), h2=e(T, N), dz=e(T, N), dw=e(N, K), db=e(N),
              dy=e(T, K), dx=e(T, K), dgamma=e(K), dbeta=e(K), ws=e(L.loco_linear_workspace_bytes(N), d=torch.uint8),
              ws2=e(L.loco_norm_workspace_bytes(T, K), d=torch.uint8))
    return st


def test_runs_agree_on_streams_and_in_a_graph(L):
    """The same bits on the default stream, on another stream and replayed from a captured graph."""
    st = step_state(L)
    want = {k: v.clone() for k, v in step_all(L, st).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        st2 = step_state(L)
        got = step_all(L, st2)
    side.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step_all(L, st2)
    for k in want:
        if got[k].dtype.is_floating_point:
            got[k].zero_()
    graph.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k
