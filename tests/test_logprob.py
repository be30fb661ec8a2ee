"""Log probabilities, entropies, alternatives and the gradient of the logits against 64 bits (GPU)."""
import math

import pytest
import torch

import layers_ref as R
import steps_ref as S
from test_layers_gpu import F32, BF16, gen, guarded

pytestmark = pytest.mark.gpu
U, INF = S.U, math.inf
NEG = {F32: torch.finfo(F32).min, BF16: torch.finfo(BF16).min}


@pytest.fixture(scope="module")
def L():
    from bit_gradient_compression_gb300 import loco
    return loco


def logits(g, rows, vocab, dtype, ld, off=0, sigma=2.5):
    buf = (torch.randn(off + rows * ld + 16, generator=g, device="cuda") * sigma).to(dtype)
    return buf.as_strided((rows, vocab), (ld, 1), off)


def bounds(z, want):
    """Bounds of the log sum, of a log probability and of the entropy, where z is the rows' logits times the scale."""
    lse, logp = want[0], want[5]
    m = z.amax(1)
    p = torch.where(logp > -INF, logp.exp(), torch.zeros_like(logp))
    d = torch.where(p > 0, (m[:, None] - z), torch.zeros_like(z))       # deviations from the maximum
    mean_d, ls = (p * d).sum(1), (lse - m)
    # a thread adds 16 terms of a tile, two at a time, and its tiles, of vocab / 512 at most (where a warp has the row),
    # then 13 joins; a term's exponent is off by 4 u of its deviation, 2^x by 4 u
    n = z.shape[1] / 512 + 32 + 16
    rel = n * U + 4 * U + 4 * U * mean_d
    t_lse = rel + 3 * U * (m.abs() + lse.abs() + ls)
    t_logp = rel[:, None] + 4 * U * (d + ls[:, None] + logp.abs())
    t_h = rel * (1 + mean_d) + n * U * mean_d + 6 * U * (ls + mean_d) + 4 * U * (p * d * d).sum(1)
    return t_lse, t_logp, t_h


def check_forward(L, z, targets, top, scale):
    rows, vocab = z.shape
    new = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    logp, lse, h, alts = new(rows), new(rows), new(rows), new(rows, top)
    ids = torch.full((rows, top), 77, dtype=torch.int64, device="cuda")
    kw = dict(top_ids=ids, top_logp=alts) if top else {}
    L.loco_logprob_forward(z, targets, logp, lse=lse, entropy=h, scale=scale, **kw)
    zz = z.double() * scale
    want = S.logprob(zz, targets, top)
    t_lse, t_logp, t_h = bounds(zz, want)
    fine = torch.isfinite(want[0])
    for got, w, tol, what in ((lse, want[0], t_lse, "lse"), (h, want[2], t_h, "entropy")):
        R.close(got[fine], w[fine], tol[fine], what)
        assert torch.equal(got[~fine].nan_to_num(3.0), w[~fine].float().nan_to_num(3.0)), what
    at = t_logp.gather(1, targets.clamp(0, vocab - 1)[:, None])[:, 0]
    ok = fine & torch.isfinite(want[1])
    R.close(logp[ok], want[1][ok], at[ok], "logp")
    assert torch.equal(logp[~ok].nan_to_num(3.0, None, -5.0), want[1][~ok].float().nan_to_num(3.0, None, -5.0))
    if top:
        assert torch.equal(ids, want[3])
        listed = ids >= 0
        tol = t_logp.gather(1, ids.clamp(min=0))
        R.close(alts[listed], want[4][listed], tol[listed], "alternatives")
        assert torch.equal(alts[~listed].nan_to_num(3.0, None, -5.0), want[4][~listed].float().nan_to_num(3.0, None, -5.0))
    return lse, h


SHAPES = [(1, 1), (3, 2), (5, 7), (9, 33), (17, 256), (2, 1000), (8, 1023), (40, 1024), (3, 1025), (700, 1031), (1, 4096),
          (2, 32000), (33, 32003), (1, 128001), (300, 50001), (2000, 5000)]


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("top", [0, 1, 5, 20, 32])
@pytest.mark.parametrize("ld,off", [(0, 0), (5, 3)])
def test_forward(L, rows, vocab, dtype, top, ld, off):
    g = gen(21)
    z = logits(g, rows, vocab, dtype, vocab + ld, off)
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    if rows > 2:
        y[1], y[2] = -100, vocab       # none given; one that does not exist
    check_forward(L, z, y, top, 1.0 if top % 2 else 0.7)


@pytest.mark.parametrize("vocab", [40, 900, 1500, 33000])
@pytest.mark.parametrize("rows", [9, 700])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("top", [1, 8, 32])
def test_masks(L, vocab, rows, dtype, top):
    """Tokens that cannot come, rows of which few, one or none is left, the type's lowest value as a mask, infinities, NaN."""
    g = gen(22)
    z = logits(g, rows, vocab, dtype, vocab + 8)
    z[:, torch.rand(vocab, generator=g, device="cuda") < 0.5] = -INF
    z[0] = -INF                                   # nothing is left
    z[1] = -INF
    z[1, vocab // 2] = 3.0                        # one token
    z[2] = NEG[dtype]                             # every token alike, at the lowest value
    z[3] = NEG[dtype]
    z[3, vocab - 1] = -1.0
    z[4, 3] = math.nan
    z[5, vocab - 2] = INF
    z[6] = -INF
    z[6, vocab // 3: vocab // 3 + 7] = torch.tensor([0.0, -0.0, 1.0, 1.0, -0.0, 0.0, 2.0], device="cuda").to(dtype)
    z[7] = 0.0                                    # ties everywhere
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    y[1], y[3] = vocab // 2, 0
    check_forward(L, z, y, top, 1.0)


@pytest.mark.parametrize("order", ["up", "down", "steps", "constant"])
@pytest.mark.parametrize("vocab", [1000, 20000, 70001])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_alternatives_in_ordered_rows(L, order, vocab, dtype):
    """Rows in which every value is a candidate, and rows full of ties."""
    v = torch.arange(vocab, device="cuda", dtype=torch.float64)
    v = {"up": v / vocab, "down": -v / vocab, "steps": torch.floor(v / 97) % 5, "constant": v * 0 + 0.5}[order]
    z = v.to(dtype).repeat(3, 1)
    y = torch.tensor([0, vocab - 1, vocab // 2], device="cuda")
    check_forward(L, z, y, 32, 1.0)


@pytest.mark.parametrize("rows,vocab", [(700, 1500), (1300, 4001), (2500, 20003), (2440, 32768)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("top", [0, 3, 32])
@pytest.mark.parametrize("order", ["random", "up"])
def test_many_long_rows(L, rows, vocab, dtype, top, order):
    """So many rows that a warp takes one, with rows in which every value is a candidate and rows that are masked."""
    g = gen(27)
    z = logits(g, rows, vocab, dtype, vocab + 3)
    if order == "up":
        z.copy_(z.sort(1)[0])
    z[5] = -INF
    z[6, : vocab - 2] = -INF
    z[7, 0] = math.nan
    z[8] = 1.0
    check_forward(L, z, torch.randint(0, vocab, (rows,), generator=g, device="cuda"), top, 1.0)


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ld,ldd", [(0, 0), (5, 0), (8, 16)])
@pytest.mark.parametrize("which", ["both", "logp", "entropy"])
def test_backward(L, rows, vocab, dtype, ld, ldd, which):
    g = gen(23)
    scale = 0.7
    z = logits(g, rows, vocab, dtype, vocab + ld)
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    if rows > 4:
        y[1] = -1
        z[2] = -INF
        z[3, : vocab // 2] = -INF
        z[4] = NEG[dtype]
        z[4, vocab - 1] = 1.0
    zz = z.double() * scale
    lse64, _, h64, _, _, _ = S.logprob(zz, y, 1)
    lse, h = lse64.float(), h64.float()
    dlogp = torch.randn(rows, generator=g, device="cuda") if which != "entropy" else None
    dh = torch.randn(rows, generator=g, device="cuda") if which != "logp" else None
    out, intact = guarded(rows, vocab, dtype, vocab + ldd)
    L.loco_logprob_backward(z, y if dlogp is not None else None, lse, out, dlogp=dlogp, entropy=h if dh is not None else None,
                            dentropy=dh, scale=scale)
    some = torch.isfinite(lse)
    logp = zz - torch.where(some, lse, torch.zeros_like(lse)).double()[:, None]
    p = torch.where(some[:, None], logp.exp(), torch.zeros_like(zz))
    d = torch.zeros(rows, device="cuda").double() if dlogp is None else torch.where((y >= 0) & some, dlogp.double(), 0.0)
    e = torch.zeros(rows, device="cuda").double() if dh is None else dh.double()
    inner = torch.where(p > 0, logp + h.double()[:, None], torch.zeros_like(zz))
    one = torch.zeros_like(zz).scatter_(1, y.clamp(min=0)[:, None], 1.0)
    want = scale * (d[:, None] * (one - p) - e[:, None] * p * inner)
    # p's exponent z c - lse log2(e): each product off by 2 u of itself, 2^x by 4 u
    size = torch.where(p > 0, zz.abs() + torch.where(some, lse, torch.zeros_like(lse)).double().abs()[:, None], torch.zeros_like(zz))
    dt = 3 * U * size
    each = p * (d.abs()[:, None] + e.abs()[:, None] * (torch.where(p > 0, logp.abs(), torch.zeros_like(p)) + h.double().abs()[:, None]))
    tol = scale * ((dt + 12 * U) * each + p * e.abs()[:, None] * dt + 4 * U * one * d.abs()[:, None])
    R.close(out, want, tol + 2 * U * want.abs() + S.out_tol(want, dtype), "dlogits")
    assert intact()
    # in place of the logits: the same values
    L.loco_logprob_backward(z, y if dlogp is not None else None, lse, z, dlogp=dlogp, entropy=h if dh is not None else None,
                            dentropy=dh, scale=scale)
    assert torch.equal(z, out)


@pytest.mark.parametrize("vocab", [100, 3000])
def test_backward_of_bad_rows(L, vocab):
    """NaN where a row's log sum is, and where the given token does not exist; nothing of it in other rows."""
    g = gen(24)
    z = logits(g, 5, vocab, F32, vocab)
    z[1, 3] = math.nan
    y = torch.tensor([0, 1, vocab, 2, -1], device="cuda")
    lse, out, d = torch.empty(5, device="cuda"), torch.empty(5, vocab, device="cuda"), torch.ones(5, device="cuda")
    L.loco_logprob_forward(z, y, torch.empty(5, device="cuda"), lse=lse)
    L.loco_logprob_backward(z, y, lse, out, dlogp=d)
    assert torch.isnan(out).all(1).tolist() == [False, True, True, False, False]
    assert bool(torch.isfinite(out[[0, 3, 4]]).all()) and not out[4].any()


def test_gradient_against_differences(L):
    """The gradient along a direction is the difference quotient of the 64-bit sum of dlogp logp + dentropy entropy."""
    rows, vocab, scale, step = 7, 1500, 0.8, 1e-5
    g = gen(25)
    z, v = logits(g, rows, vocab, F32, vocab), logits(g, rows, vocab, F32, vocab)
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    y[3] = -1
    a, b = torch.randn(rows, generator=g, device="cuda"), torch.randn(rows, generator=g, device="cuda")

    def loss(t):
        lse, logp, h, _, _, _ = S.logprob((z.double() + t * v.double()) * scale, y, 1)
        return float((logp * a.double()).sum() + (h * b.double()).sum())
    want = (loss(step) - loss(-step)) / (2 * step)
    logp, lse, h, dz = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(z)
    L.loco_logprob_forward(z, y, logp, lse=lse, entropy=h, scale=scale)
    L.loco_logprob_backward(z, y, lse, dz, dlogp=a, entropy=h, dentropy=b, scale=scale)
    got, size = float((dz.double() * v.double()).sum()), float((dz.double() * v.double()).abs().sum())
    assert abs(got - want) <= 1e-5 * size


def test_results_do_not_change_and_graphs_replay(L):
    rows, vocab, top = 3, 40001, 20     # shared by several CTAs
    g = gen(26)
    z, y = logits(g, rows, vocab, BF16, vocab), torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    logp, lse, h, alts = (torch.empty(s, device="cuda") for s in ((rows,), (rows,), (rows,), (rows, top)))
    ids, dz, one = torch.empty(rows, top, dtype=torch.int64, device="cuda"), torch.empty_like(z), torch.ones(rows, device="cuda")

    def both():
        L.loco_logprob_forward(z, y, logp, lse=lse, entropy=h, top_ids=ids, top_logp=alts)
        L.loco_logprob_backward(z, y, lse, dz, dlogp=one, entropy=h, dentropy=one)
    outs = (logp, lse, h, alts, ids, dz)
    both()
    first = [t.clone() for t in outs]
    for _ in range(3):
        both()
        assert all(torch.equal(a, b) for a, b in zip(first, outs))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both()
    z.copy_(logits(g, rows, vocab, BF16, vocab))
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in outs]
    both()
    assert all(torch.equal(a, b) for a, b in zip(replayed, outs)) and not torch.equal(replayed[0], first[0])


def test_only_what_is_asked_for(L):
    """Each output alone is what it is among the others; nothing at all is a call too."""
    g = gen(27)
    z, y = logits(g, 50, 3000, F32, 3000), torch.randint(0, 3000, (50,), generator=g, device="cuda")
    f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    logp, lse, h, alts, ids = f(50), f(50), f(50), f(50, 4), torch.empty(50, 4, dtype=torch.int64, device="cuda")
    L.loco_logprob_forward(z, y, logp, lse=lse, entropy=h, top_ids=ids, top_logp=alts)
    a, b, c, d, e = f(50), f(50), f(50), f(50, 4), torch.empty(50, 4, dtype=torch.int64, device="cuda")
    L.loco_logprob_forward(z, y, a)
    L.loco_logprob_forward(z, None, None, lse=b)
    L.loco_logprob_forward(z, None, None, entropy=c)
    L.loco_logprob_forward(z, None, None, top_logp=d)
    L.loco_logprob_forward(z, None, None, top_ids=e)
    L.loco_logprob_forward(z, None, None)
    for u, v in ((a, logp), (b, lse), (c, h), (d, alts), (e, ids)):
        assert torch.equal(u, v)
    L.loco_logprob_forward(z[:0], y[:0], f(0))
