"""Joins of a block with the residual stream and the next norm, against their formulas in 64 bits (GPU)."""
import math

import pytest
import torch

import layers_ref as R
import steps_ref as S
from test_layers_gpu import F32, BF16, gen, guarded, rand

pytestmark = pytest.mark.gpu
U = S.U


@pytest.fixture(scope="module")
def L():
    from bit_gradient_compression_gb300 import loco
    return loco


def cfg_of(L, kind, post, a=1.0, s=1.0, eps=1e-5):
    return L.make_join(L.LOCO_NORM_LAYER if kind == "layer" else L.LOCO_NORM_RMS, eps, post, a, s)


SIZES = [(1, 1), (1, 8), (2, 31), (5, 256), (3, 257), (9, 1000), (300, 1024), (4, 2047), (33, 2048), (17, 4096),
         (3, 4097), (2, 5632), (700, 96), (2, 16384), (3, 33000), (2, 32761)]
TYPES = [(F32, F32, F32), (BF16, BF16, BF16), (F32, BF16, BF16), (BF16, F32, F32)]
#: what is given: (post, gate, row gate, gammas, betas)
GIVEN = [(True, True, True, True, True), (True, False, False, True, False), (False, True, False, False, False),
         (False, False, True, True, True), (True, True, False, False, False)]


def inputs(seed, rows, cols, xd, yd, pd, pad, given):
    post, gate, row_gate, gammas, betas = given
    g = gen(seed)
    x, y = rand(g, rows, cols, xd, 2.0, cols + pad), rand(g, rows, cols, yd, 1.5, cols + pad)
    x += 1.0
    y += 0.75
    if rows > 1:
        x[rows - 1] = 0.0
        y[rows - 1] = 0.0
    vec = lambda on: rand(g, 1, cols, pd)[0] if on else None  # noqa: E731
    p = dict(gate=vec(gate), gamma=vec(gammas), beta=vec(betas), post_gamma=vec(gammas), post_beta=vec(betas))
    p["row_gate"] = torch.rand(rows, generator=g, device="cuda") if row_gate else None
    return g, x, y, p


def chain(cols):
    """Additions on the longest chain of a sum over a row: 8 of a thread's, 5 + 9 of warps and CTAs; long rows, one per 1024."""
    return 32 + cols / 1024


def stats_close(got, v, kind, eps, what):
    """Mean and reciprocal root within their bounds; the bound of a normalised value comes back."""
    m, r = S.norm_stats(v.double(), kind, eps)
    n, top = chain(v.shape[1]), v.double().abs().amax(1)
    R.close(got[0], m, n * U * top if kind == "layer" else torch.zeros_like(m), what + " mean")
    # the mean's error moves every value alike, which is second order in the variance
    rel = n * U + (n * U * top * r) ** 2 + 4 * U * top * r
    R.close(got[1], r, rel * r, what + " rstd")
    vh = (v.double() - m[:, None]) * r[:, None]
    return vh, (n * U * top * r + rel * vh.abs().amax(1))[:, None]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("xd,yd,pd", TYPES)
@pytest.mark.parametrize("given", GIVEN)
@pytest.mark.parametrize("pad", [0, 1])
def test_forward(L, rows, cols, kind, xd, yd, pd, given, pad):
    g, x, y, p = inputs(11, rows, cols, xd, yd, pd, pad, given)
    post, a, s, eps = given[0], 0.75, -0.5, 1e-5
    h, h_intact = guarded(rows, cols, xd, cols + pad)
    u, u_intact = guarded(rows, cols, yd, cols + pad)
    stats = torch.empty(4, rows, device="cuda")
    L.loco_join_forward(cfg_of(L, kind, post, a, s, eps), x, y, h, u, stats=stats, **p)
    want, n, yh, m1, r1 = S.join_forward(x, y, kind, post, eps, a, s, p["gate"], p["row_gate"], p["post_gamma"], p["post_beta"])
    if post:
        _, err = stats_close(stats[:2], y, kind, eps, "post")
    else:
        assert bool((stats[0] == 0).all()) and bool((stats[1] == 1).all())
        err = torch.zeros_like(m1)[:, None]
    weight = (s * S.or64(p["gate"], 1.0) * S.or64(p["row_gate"], torch.ones_like(m1))[:, None]).abs()
    tol = weight * (err * S.or64(p["post_gamma"], torch.ones(1, device="cuda")).abs() + 4 * U * (n.abs() + yh.abs()))
    tol = tol + 6 * U * ((a * x.double()).abs() + weight * (n.abs() + S.or64(p["post_beta"], torch.zeros(1, device="cuda")).abs()))
    R.close(h, want, tol + S.out_tol(want, xd), "h")
    # the second norm is that of the stream as it was written
    hh, err = stats_close(stats[2:], h, kind, eps, "pre")
    wu = hh * S.or64(p["gamma"], 1.0) + S.or64(p["beta"], 0.0)
    tol = err * S.or64(p["gamma"], torch.ones(1, device="cuda")).abs() + 4 * U * (wu.abs() + S.or64(p["beta"], torch.zeros(1, device="cuda")).abs())
    R.close(u, wu, tol + S.out_tol(wu, yd), "u")
    assert h_intact() and u_intact()
    # over x, and without the second norm and the statistics: the same h
    again, _ = guarded(rows, cols, xd, cols + pad)
    again.copy_(x)
    L.loco_join_forward(cfg_of(L, kind, post, a, s, eps), again, y, again, **p)
    assert torch.equal(again, h)


@pytest.mark.parametrize("rows,cols", SIZES + [(1300, 64), (2000, 512)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("xd,yd,gd", [(F32, F32, F32), (BF16, BF16, BF16), (F32, BF16, BF16)])
@pytest.mark.parametrize("given", GIVEN)
@pytest.mark.parametrize("pad", [0, 1])
def test_backward(L, rows, cols, kind, xd, yd, gd, given, pad):
    g, x, y, p = inputs(12, rows, cols, xd, yd, BF16, pad, given)
    post, a, s, eps = given[0], 0.75, -0.5, 1e-5
    h, m1, r1 = (lambda r: (r[0].to(xd), r[3], r[4]))(S.join_forward(
        x, y, kind, post, eps, a, s, p["gate"], p["row_gate"], p["post_gamma"], p["post_beta"]))
    stats = torch.stack([m1, r1, *S.norm_stats(h.double(), kind, eps)]).float()
    dh, du = rand(g, rows, cols, xd, 0.1, cols + pad), rand(g, rows, cols, yd, 0.1, cols + pad)
    beta = p.pop("beta")
    want = S.join_backward(dh, du, h, y, stats, kind, post, a, s, **p)
    dx, dx_intact = guarded(rows, cols, xd, cols + pad)
    dy, dy_intact = guarded(rows, cols, yd, cols + pad)
    names = [k for k, on in (("dgamma", True), ("dbeta", beta is not None), ("dpost_gamma", True),
                             ("dpost_beta", beta is not None), ("dgate", p["gate"] is not None)) if on]
    out = {k: torch.empty(cols, dtype=gd, device="cuda") for k in names}
    row = torch.empty(rows, device="cuda") if p["row_gate"] is not None else None
    ws = torch.empty(L.loco_join_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    cfg = cfg_of(L, kind, post, a, s, eps)
    L.loco_join_backward(cfg, dh, du, h, y, stats, dx, dy, drow_gate=row, workspace=ws, **p, **out)

    n, n_rows = chain(cols), rows + 64
    mean = lambda v: v.mean(1, keepdim=True)  # noqa: E731
    k = want
    r1, r2 = k["r1"][:, None], k["r2"][:, None]
    hh, yh, q = k["hh"].abs(), k["yh"].abs(), k["q"].abs()
    # (h - m2) r2 is off by 4 u of its terms, |h| r2 and |hh|
    amp2 = h.double().abs().amax(1, keepdim=True) * r2
    amp1 = y.double().abs().amax(1, keepdim=True) * r1
    tol_t = n * U * r2 * (q + mean(q) + (hh + amp2) * (mean(q * hh) + amp2 * mean(q))) + 4 * U * (k["t"].abs() + S.or64(dh, 0.0).abs())
    R.close(dx, k["dx"], abs(a) * tol_t + 2 * U * k["dx"].abs() + S.out_tol(k["dx"], xd), "dx")
    gs = (s * k["g"] * k["pg"]).abs()                       # p / (t w)
    tol_p, pp = gs * tol_t + 4 * U * gs * k["t"].abs(), gs * k["t"].abs()
    if post:
        tol = tol_p + mean(tol_p) + yh * mean(tol_p * yh)
        tol = tol + n * U * (pp + mean(pp) + (yh + amp1) * (mean(pp * yh) + amp1 * mean(pp)))
        tol = k["w"].abs() * r1 * tol
    else:
        tol = k["w"].abs() * tol_p
    R.close(dy, k["dy"], tol + 4 * U * k["dy"].abs() + S.out_tol(k["dy"], yd), "dy")
    assert dx_intact() and dy_intact()

    dud = du.double().abs()
    sums = {"dgamma": (dud * (4 * U * (hh + amp2))).sum(0) + n_rows * U * (dud * (hh + U * amp2)).sum(0),
            "dbeta": n_rows * U * dud.sum(0)}
    c, tol_c = k["w"].abs() * k["t"].abs(), k["w"].abs() * (tol_t + U * k["t"].abs())
    v0 = (tol_c * yh + c * 4 * U * (yh + amp1)).sum(0) + n_rows * U * (c * yh).sum(0)
    v1 = tol_c.sum(0) + n_rows * U * c.sum(0)
    sg = (s * k["g"]).abs()
    pg, pb = k["pg"] if torch.is_tensor(k["pg"]) else torch.ones(cols, device="cuda").double(), S.or64(p["post_beta"], torch.zeros(cols, device="cuda")).abs()
    sums["dpost_gamma"], sums["dpost_beta"] = sg * v0, sg * v1
    sums["dgate"] = abs(s) * (pg.abs() * v0 + pb * v1) + 4 * U * abs(s) * (pg.abs() * (c * yh).sum(0) + pb * c.sum(0))
    for name in names:
        R.close(out[name], want[name], sums[name] + 4 * U * want[name].abs() + S.out_tol(want[name], gd), name)
    if row is not None:
        terms = k["t"].abs() * (yh * pg.abs() + pb)
        tol = (sg * (tol_t * (yh * pg.abs() + pb) + k["t"].abs() * pg.abs() * 4 * U * (yh + amp1)) + n * U * sg * terms).sum(1)
        R.close(row, want["drow_gate"], tol + 8 * U * (sg * terms).sum(1), "drow_gate")
    # dx over dh, without the parameters' gradients: the same values
    (again, _), (dy2, _) = guarded(rows, cols, xd, cols + pad), guarded(rows, cols, yd, cols + pad)
    again.copy_(dh)
    L.loco_join_backward(cfg, again, du, h, y, stats, again, dy2, **p)
    assert torch.equal(again, dx) and torch.equal(dy2, dy)


@pytest.mark.parametrize("rows,cols,pad", [(40, 96, 0), (40, 97, 0), (9, 4096, 0), (3, 9001, 0)])
@pytest.mark.parametrize("post", [True, False])
def test_backward_of_one_side(L, rows, cols, pad, post):
    """Without du only the stream's gradient comes back (h is not read), without dh only that of the next norm."""
    g, x, y, p = inputs(13, rows, cols, F32, BF16, BF16, pad, (post, True, True, True, True))
    p.pop("beta")
    stats = torch.stack([*S.norm_stats(y.double(), "layer", 1e-5), *S.norm_stats(x.double(), "layer", 1e-5)]).float()
    if not post:
        stats[0], stats[1] = 0.0, 1.0
    cfg = cfg_of(L, "layer", post, 0.5, 2.0)
    dh, du = rand(g, rows, cols, F32, 0.1), rand(g, rows, cols, BF16, 0.1)
    ws = torch.empty(L.loco_join_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    new = lambda: (torch.empty(rows, cols, device="cuda"), torch.empty(rows, cols, dtype=BF16, device="cuda"))  # noqa: E731
    zh, zu = torch.zeros_like(dh), torch.zeros_like(du)
    for one, both in (((dh, None), (dh, zu)), ((None, du), (zh, du)), ((None, None), (zh, zu))):
        got = []
        for a, b in (one, both):
            dx, dy = new()
            v = {k: torch.empty(cols, device="cuda") for k in ("dgamma", "dbeta", "dpost_gamma", "dpost_beta", "dgate")}
            dr = torch.empty(rows, device="cuda")
            L.loco_join_backward(cfg, a, b, None if b is None else x, y, stats, dx, dy, workspace=ws, drow_gate=dr, **p, **v)
            got.append([dx, dy, dr, *v.values()])
        for u, v in zip(*got):
            assert torch.equal(u, v)


def test_block_output_not_needed(L):
    """Without a norm behind the block and without its gradients, y is not read."""
    rows, cols = 7, 64
    g = gen(14)
    dh = rand(g, rows, cols, BF16, 1.0)
    gate = rand(g, 1, cols, BF16)[0]
    dx, dy = torch.empty_like(dh), torch.empty_like(dh)
    L.loco_join_backward(cfg_of(L, "rms", False, 1.0, 0.5), dh, None, None, None, None, dx, dy, gate=gate)
    assert torch.equal(dx, dh)
    R.close(dy, 0.5 * gate.double() * dh.double(), S.out_tol(0.5 * gate.double() * dh.double(), BF16) * 1.001, "dy")


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("cols", [75, 4200])
def test_gradient_against_differences(L, kind, post, cols):
    """The gradients along a direction of every input are the difference quotient of the 64-bit loss <h, c> + <u, e>."""
    rows, eps, a, s = 6, 1e-5, 0.8, 0.6
    g = gen(15)
    x, y, c, e, dx_, dy_ = (rand(g, rows, cols, F32) for _ in range(6))
    names = ("gate", "post_gamma", "post_beta", "gamma", "beta")
    p = {k: rand(g, 1, cols, F32)[0] for k in names}
    d = {k: rand(g, 1, cols, F32)[0] for k in names}
    w, dw = torch.rand(rows, device="cuda", generator=g), torch.rand(rows, device="cuda", generator=g)

    def loss(t):
        q = {k: p[k].double() + t * d[k].double() for k in names}
        h = S.join_forward(x.double() + t * dx_.double(), y.double() + t * dy_.double(), kind, post, eps, a, s, q["gate"],
                           w.double() + t * dw.double(), q["post_gamma"], q["post_beta"])[0]
        m, r = S.norm_stats(h, kind, eps)
        u = (h - m[:, None]) * r[:, None] * q["gamma"] + q["beta"]
        return float((h * c.double()).sum() + (u * e.double()).sum())
    step = 1e-5
    want = (loss(step) - loss(-step)) / (2 * step)
    h, u, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(4, rows, device="cuda")
    cfg = cfg_of(L, kind, post, a, s, eps)
    L.loco_join_forward(cfg, x, y, h, u, row_gate=w, stats=stats, **p)
    dx, dy, dr = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
    v = {"d" + k: torch.empty(cols, device="cuda") for k in names}
    ws = torch.empty(L.loco_join_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    q = {k: p[k] for k in names if k != "beta"}
    L.loco_join_backward(cfg, c, e, h, y, stats, dx, dy, row_gate=w, drow_gate=dr, workspace=ws, **q, **v)
    pairs = [(dx, dx_), (dy, dy_), (dr, dw)] + [(v["d" + k], d[k]) for k in names]
    got = sum(float((u.double() * t.double()).sum()) for u, t in pairs)
    scale = sum(float((u.double() * t.double()).abs().sum()) for u, t in pairs)
    assert abs(got - want) <= 1e-6 * scale + 1e-8 * abs(loss(0.0))


@pytest.mark.parametrize("cols,pad", [(96, 0), (96, 1), (4096, 0), (5000, 0), (40000, 0)])
def test_nan_stays_in_its_row(L, cols, pad):
    g, x, y, p = inputs(16, 6, cols, F32, F32, F32, pad, (True, True, True, True, True))
    y[2, 5] = math.nan
    x[4, 7] = math.inf
    h, u = torch.empty(6, cols, device="cuda"), torch.empty(6, cols, device="cuda")
    L.loco_join_forward(cfg_of(L, "layer", True), x, y, h, u, **p)
    bad = torch.isnan(u).any(1)
    assert bad.tolist() == [False, False, True, False, True, False] and bool(torch.isnan(u[2]).all())
    assert bool(torch.isfinite(h[[0, 1, 3, 5]]).all())


@pytest.mark.parametrize("far", [1e2, 1e4])
@pytest.mark.parametrize("cols,pad", [(96, 0), (1001, 0), (4096, 0), (8192, 0), (33000, 0)])
def test_rows_far_from_zero(L, far, cols, pad):
    """Rows whose mean is 10^2 and 10^4 of their spread: a deviation loses only what the value itself had lost."""
    rows = 5
    g = gen(17)
    y = (rand(g, rows, cols, F32) + far)
    x = torch.zeros_like(y)
    h = torch.empty_like(y)
    L.loco_join_forward(cfg_of(L, "layer", True), x, y, h)
    want = S.join_forward(x, y, "layer", True, 1e-5, 1.0, 1.0)[0]
    # the mean is off by at most the last place of `far` times the chain's rounding of deviations, the variance by their square
    n = chain(cols)
    tol = 2 * U * far * (1 + n / 8) + n * U * want.abs() + 8 * U * want.abs()
    assert bool(((h.double() - want).abs() <= tol).all()), float(((h.double() - want).abs() / tol).max())


def test_results_do_not_change_and_graphs_replay(L):
    """The same from call to call; a captured forward and backward pass replays on new values, beside an eager one."""
    rows, cols = 333, 2048
    g, x, y, p = inputs(18, rows, cols, BF16, BF16, BF16, 0, (True, True, True, True, True))
    cfg = cfg_of(L, "layer", True, 1.0, 0.5)
    beta = p["beta"]
    h, u, stats = torch.empty_like(x), torch.empty_like(y), torch.empty(4, rows, device="cuda")
    dx, dy, dr = torch.empty_like(x), torch.empty_like(y), torch.empty(rows, device="cuda")
    v = {k: torch.empty(cols, device="cuda") for k in ("dgamma", "dbeta", "dpost_gamma", "dpost_beta", "dgate")}
    ws = torch.empty(L.loco_join_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    q = {k: t for k, t in p.items() if k != "beta"}

    def both():
        L.loco_join_forward(cfg, x, y, h, u, stats=stats, **p)
        L.loco_join_backward(cfg, h, u, h, y, stats, dx, dy, drow_gate=dr, workspace=ws, **q, **v)
    both()
    first = [t.clone() for t in (h, u, stats, dx, dy, dr, *v.values())]
    both()
    assert all(torch.equal(a, b) for a, b in zip(first, (h, u, stats, dx, dy, dr, *v.values())))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both()
    x.copy_(rand(g, rows, cols, BF16))
    beta.copy_(rand(g, 1, cols, BF16)[0])
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in (h, u, stats, dx, dy, dr, *v.values())]
    assert not torch.equal(replayed[0], first[0])
    both()
    assert all(torch.equal(a, b) for a, b in zip(replayed, (h, u, stats, dx, dy, dr, *v.values())))


@pytest.mark.parametrize("cols,ld", [(1, 1), (2, 2), (3, 3), (5, 5), (3, 4), (9, 9), (23, 23), (25, 25)])
@pytest.mark.parametrize("xd,yd", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("rows", [1, 7, 300])
def test_narrow_rows_without_gaps(L, cols, ld, xd, yd, rows):
    """Matrices narrower than a piece, packed, from an odd element of a buffer to its last one: every value arrives and
    leaves at its place.  Without norms an output is two products and a sum, each off by half a step."""
    g = gen(19)
    cfg, a, s = cfg_of(L, "layer", False, 0.75, -0.5), 0.75, -0.5

    def place(dtype, v):
        t = torch.empty(1 + (rows - 1) * ld + cols, dtype=dtype, device="cuda").as_strided((rows, cols), (ld, 1), 1)
        return t.copy_(v)
    x, dh = (place(xd, rand(g, rows, cols, xd)) for _ in range(2))
    y = place(yd, rand(g, rows, cols, yd))
    h, dx, dy = place(xd, torch.zeros_like(x)), place(xd, torch.zeros_like(x)), place(yd, torch.zeros_like(y))
    L.loco_join_forward(cfg, x, y, h)
    want = a * x.double() + s * y.double()
    R.close(h, want, 3 * U * (a * x.double().abs() + 0.5 * y.double().abs()) + S.out_tol(want, xd), "h")
    dgate = torch.empty(cols, device="cuda")
    ws = torch.empty(L.loco_join_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    L.loco_join_backward(cfg, dh, None, None, y, None, dx, dy, dgate=dgate, workspace=ws)
    d = dh.double()
    R.close(dx, a * d, 2 * U * d.abs() + S.out_tol(a * d, xd), "dx")
    R.close(dy, s * d, 2 * U * d.abs() + S.out_tol(s * d, yd), "dy")
    terms = (d * y.double()).abs().sum(0)
    R.close(dgate, s * (d * y.double()).sum(0), (rows + 4) * U * terms, "dgate")


def test_empty_batch(L):
    cfg = cfg_of(L, "layer", True)
    e = torch.empty(0, 40, device="cuda")
    L.loco_join_forward(cfg, e, e, torch.empty(0, 40, device="cuda"), torch.empty(0, 40, device="cuda"))
    v = {k: torch.ones(40, device="cuda") for k in ("dgamma", "dbeta", "dpost_gamma", "dpost_beta", "dgate")}
    gate = torch.full((40,), math.nan, device="cuda")
    L.loco_join_backward(cfg, e, e, e, e, None, torch.empty(0, 40, device="cuda"), torch.empty(0, 40, device="cuda"),
                         gate=gate, **v)
    assert not any(t.any() for t in v.values())


@pytest.mark.parametrize("rows,cols", [(1, 5), (2, 15), (3, 37), (4, 256), (5, 300), (3, 1025), (2, 4099), (3, 9001), (2, 24577)])
@pytest.mark.parametrize("xd,yd", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_rows_that_lie_anywhere(L, rows, cols, xd, yd):
    """Every matrix at its own place and pitch: the same bits as with some at an odd place, and nothing around the
    outputs is written.  The inputs fill their memory to its last element."""
    g = gen(19)
    _, x, y, p = inputs(19, rows, cols, xd, yd, BF16, 0, (True, True, True, True, True))
    dh, du = rand(g, rows, cols, xd, 0.1), rand(g, rows, cols, yd, 0.1)
    cfg = cfg_of(L, "layer", True, 0.75, 0.5)
    q = {k: t for k, t in p.items() if k != "beta"}
    ws = torch.empty(L.loco_join_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")

    def placed(t, off, pad):
        rows_, ld = t.shape[0], cols + pad
        buf = torch.full((off + (rows_ - 1) * ld + cols,), 3.0, dtype=t.dtype, device="cuda")
        out = buf.as_strided((rows_, cols), (ld, 1), off)
        out.copy_(t)
        return out

    def run(place):
        outs, checks = [], []

        def out(d, i):
            off, pad = place(i)
            buf = torch.full((off + rows * (cols + pad) + 16,), 7.0, dtype=d, device="cuda")
            t = buf.as_strided((rows, cols), (cols + pad, 1), off)
            outs.append(t)
            checks.append((buf, off, pad))
            return t
        a, b, c, d = (placed(t, *place(i)) for i, t in enumerate((x, y, dh, du)))
        h, u, stats = out(xd, 4), out(yd, 5), torch.empty(4, rows, device="cuda")
        L.loco_join_forward(cfg, a, b, h, u, stats=stats, **p)
        dx, dy = out(xd, 6), out(yd, 7)
        v = {k: torch.empty(cols, device="cuda") for k in ("dgamma", "dbeta", "dpost_gamma", "dpost_beta", "dgate")}
        dr = torch.empty(rows, device="cuda")
        L.loco_join_backward(cfg, c, d, h, b, stats, dx, dy, drow_gate=dr, workspace=ws, **q, **v)
        for buf, off, pad in checks:
            seen = torch.ones_like(buf, dtype=torch.bool)
            seen.as_strided((rows, cols), (cols + pad, 1), off).fill_(False)
            assert bool((buf[seen] == 7).all())
        return [t.clone() for t in outs] + [stats, dr, *v.values()]
    want = run(lambda i: (1, 0) if i in (0, 4, 2) else (0, -cols % 8))
    for shift in range(4):
        got = run(lambda i: ((3 * i + shift) % 9, (5 * i + 2 * shift + 1) % 11))
        for k, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (shift, k)
