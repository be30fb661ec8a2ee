"""Joins, log probabilities and AdamW behind 2^31 and 2^32 elements, and calls on streams of their own (GPU)."""
import pytest
import torch

import steps_ref as S
import test_adam_tensors as A
from test_join import cfg_of, inputs, rand
from test_layers_gpu import BF16, F32, gen
from test_logprob import bounds

pytestmark = pytest.mark.gpu
U = S.U


@pytest.fixture(scope="module")
def L():
    from bit_gradient_compression_gb300 import loco
    return loco


@pytest.fixture(autouse=True)
def room():
    """These tests hold up to 45 GB: what others left in torch's allocator goes first, and theirs afterwards."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("less than 60 GB of free device memory")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,vocab,ld", [(4, 5000, (1 << 30) + 8), (68000, 32000, 32001)])
def test_logits_behind_two_billion(L, rows, vocab, ld):
    """Rows far apart and many rows: the last ones against 64 bits, with a gradient that goes over the logits."""
    g = gen(51)
    z = torch.empty(rows * ld, dtype=BF16, device="cuda").as_strided((rows, vocab), (ld, 1))
    last = torch.arange(rows - 2, rows, device="cuda")
    z.zero_()
    z[last] = (torch.randn(2, vocab, generator=g, device="cuda") * 2.5).to(BF16)
    zz = z[last].double()
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    logp, lse, h = (torch.empty(rows, device="cuda") for _ in range(3))
    ids, alts = torch.empty(rows, 5, dtype=torch.int64, device="cuda"), torch.empty(rows, 5, device="cuda")
    L.loco_logprob_forward(z, y, logp, lse=lse, entropy=h, top_ids=ids, top_logp=alts)
    want = S.logprob(zz, y[last], 5)
    t_lse, t_logp, t_h = bounds(zz, want)
    assert torch.equal(ids[last], want[3])
    assert bool(((lse[last].double() - want[0]).abs() <= t_lse).all())
    assert bool(((h[last].double() - want[2]).abs() <= t_h).all())
    assert bool(((logp[last].double() - want[1]).abs() <= t_logp.gather(1, y[last][:, None])[:, 0]).all())
    if rows > 2:  # the others' logits are all 0
        assert bool(((lse[:-2].double() - torch.log(torch.tensor(float(vocab)))).abs() <= 2.0 ** -24 * 4 * 11).all())
        assert torch.equal(ids[:-2], torch.arange(5, device="cuda").expand(rows - 2, 5))
    one = torch.ones(rows, device="cuda")
    L.loco_logprob_backward(z, y, lse, z, dlogp=one)
    p = torch.softmax(zz, 1)
    exact = -p
    exact.scatter_add_(1, y[last][:, None], torch.ones(2, 1, dtype=torch.float64, device="cuda"))
    # a probability: the exponent's roundings (4 u of up to 30) and the log sum's; then its rounding to bf16
    assert bool(((z[last].double() - exact).abs() <= 40 * 4 * U * p + 2.0 ** -8 * exact.abs() + 1e-30).all())


def test_longest_row(L):
    """A row of LOCO_MAX_DIM logits, 0 but for three: its log sum in closed form, and alternatives from both of its ends."""
    vocab = (1 << 31) - 1
    z = torch.zeros(1, vocab, dtype=BF16, device="cuda")
    z[0, 0], z[0, vocab - 1], z[0, vocab // 2] = 1.0, 2.0, -float("inf")
    y = torch.tensor([vocab - 1], device="cuda")
    logp, lse, h = (torch.empty(1, device="cuda") for _ in range(3))
    ids, alts = torch.empty(1, 3, dtype=torch.int64, device="cuda"), torch.empty(1, 3, device="cuda")
    L.loco_logprob_forward(z, y, logp, lse=lse, entropy=h, top_ids=ids, top_logp=alts)
    e = torch.tensor([1.0, 2.0], dtype=torch.float64).exp()
    total = (vocab - 3) + float(e.sum())
    want = float(torch.log(torch.tensor(total, dtype=torch.float64)))
    entropy = want - float((e * torch.tensor([1.0, 2.0], dtype=torch.float64)).sum()) / total
    # eight CTAs of 256 threads: 16 terms of a tile two at a time, 2^31 / 65536 tiles, 13 joins; then 4 u of the log sum
    tol = (32768 + 32 + 13) * U + 8 * U * want
    assert abs(float(lse) - want) <= tol and abs(float(logp) - (2.0 - want)) <= tol and abs(float(h) - entropy) <= 4 * tol
    assert ids.tolist() == [[vocab - 1, 0, 1]]
    L.loco_logprob_backward(z, y, lse, z, dlogp=torch.ones(1, device="cuda"))
    assert abs(float(z[0, vocab - 1]) - 1.0) <= 2.0 ** -8 and float(z[0, vocab // 2]) == 0.0
    p = torch.tensor(-1.0 / total)
    assert abs(float(z[0, 12345]) - float(p)) <= (2.0 ** -8 + tol) * abs(float(p))


def test_streams_behind_two_billion(L):
    """The last rows of a join of 2.2e9 elements are those of the same rows alone, forward and backward."""
    rows, cols, few = 530000, 4096, 3
    g, x, y, p = inputs(52, few, cols, BF16, BF16, BF16, 0, (True, False, True, False, True))
    beta, row_gate = p.pop("beta"), p.pop("row_gate")
    cfg = cfg_of(L, "rms", True, 0.75, -0.5)

    def run(x, y, dh, du, rows):
        h, u, stats = torch.empty_like(x), torch.empty_like(y), torch.empty(4, rows, device="cuda")
        dx, dy, gates = torch.empty_like(x), torch.empty_like(y), torch.ones(rows, device="cuda")
        gates[-few:] = row_gate
        v = {k: torch.empty(cols, device="cuda") for k in ("dgamma", "dpost_gamma", "dgate")}
        ws = torch.empty(L.loco_join_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        L.loco_join_forward(cfg, x, y, h, u, stats=stats, beta=beta, row_gate=gates, **p)
        L.loco_join_backward(cfg, dh, du, h, y, stats, dx, dy, workspace=ws, row_gate=gates, **p, **v)
        return [t[-few:].clone() for t in (h, u, dx, dy)] + [stats[:, -few:].clone()], v
    dh, du = rand(g, few, cols, BF16, 0.1), rand(g, few, cols, BF16, 0.1)
    alone, v1 = run(x.contiguous(), y.contiguous(), dh.contiguous(), du.contiguous(), few)
    big = [torch.zeros(rows, cols, dtype=BF16, device="cuda") for _ in range(4)]
    for to, t in zip(big, (x, y, dh, du)):
        to[-few:] = t
    rows_of, v2 = run(*big, rows)
    assert all(torch.equal(a, b) for a, b in zip(alone, rows_of))
    # the other rows add nothing to the parameters' gradients; the three terms may be added in another order
    for k in v1:
        size = sum(t.abs() for t in (v1[k], v2[k])) + v1[k].abs().max()
        assert bool(((v1[k] - v2[k]).abs() <= 8 * U * size * few).all()), k


@pytest.mark.parametrize("bits,n", [(8, (1 << 32) + 300), (32, (1 << 31) + 700)])
def test_tensors_behind_four_billion(L, bits, n, monkeypatch):
    """The last elements of a tensor of more than 2^32 (2^31) elements: bit for bit the stated step, dither included."""
    g, nb, few = gen(53), -(-n // S.BLOCK), 2 * S.BLOCK + n % S.BLOCK
    lo = n - few
    p, gr = (torch.zeros(n, dtype=BF16, device="cuda") for _ in range(2))
    if bits == 8:
        m, v = torch.zeros(nb * S.BLOCK, dtype=torch.int8, device="cuda"), torch.zeros(nb * S.BLOCK, dtype=torch.uint8, device="cuda")
        ms, vs = (torch.zeros(nb, device="cuda") for _ in range(2))
    else:
        m, v, ms, vs = (*(torch.zeros(n, device="cuda") for _ in range(2)), None, None)
    p[lo:], gr[lo:] = (torch.randn(few, generator=g, device="cuda").to(BF16) for _ in range(2))
    # a second tensor behind the large one is a list's later one
    other = [torch.randn(1000, generator=g, device="cuda").to(BF16) for _ in range(2)]
    om = [torch.zeros(1024 if bits == 8 else 1000, dtype=t, device="cuda") for t in ((torch.int8, torch.uint8) if bits == 8 else (F32, F32))]
    os = [torch.zeros(4, device="cuda") for _ in range(2)]
    tail = dict(p=[p[lo:].clone(), other[0].clone()], g=[gr[lo:].clone(), other[1]], scales=[1.0, 1.0], decay=[1.0, 1.0])
    if bits == 8:
        tail.update(m=[m[lo:lo + 3 * S.BLOCK].clone(), om[0].clone()], v=[v[lo:lo + 3 * S.BLOCK].clone(), om[1].clone()],
                    ms=[ms[-3:].clone(), os[0].clone()], vs=[vs[-3:].clone(), os[1].clone()])
    else:
        tail.update(m=[m[lo:].clone(), om[0].clone()], v=[v[lo:].clone(), om[1].clone()])
    hp = L.make_adam(lr=1e-2, weight_decay=0.1)
    tensors = L.make_adam_tensors([p, other[0]], [gr, other[1]], [m, om[0]], [v, om[1]], m_steps=[ms, os[0]] if bits == 8 else None,
                                  v_steps=[vs, os[1]] if bits == 8 else None, dither=77)

    def bits_of(dither, t, i, count, device):
        e = torch.arange(count, device=device) + (lo if i == 0 else 0)
        key = S.mix(S.mix(S.mix(torch.tensor(dither, device=device)) ^ t) ^ i)
        return S.mix((e & 0xFFFFFFFF) ^ S.mix(key ^ (e >> 32)))
    monkeypatch.setattr(S, "random_bits", bits_of)
    want = [A.expect(tail, i, bits, BF16, hp, 4, 77, None) for i in range(2)]
    L.loco_adam_tensors(tensors, hp, 4)
    got = [dict(p=p[lo:], m=m[lo:], v=v[lo:]), dict(p=other[0], m=om[0], v=om[1])]
    if bits == 8:
        got[0].update(ms=ms[-3:], vs=vs[-3:])
        got[1].update(ms=os[0], vs=os[1])
    for a, b in zip(got, want):
        for k in a:
            assert A.same(a[k], b[k]), k
    assert not bool(p[:1 << 20].any()) and not bool(p[lo - (1 << 20):lo].any())
    if bits == 8:  # the values again, from the last codes
        out = torch.empty(n, dtype=BF16, device="cuda")
        L.loco_adam_state_decode(m, ms, out)
        assert torch.equal(out[lo:], S.decode(m[lo:], ms[-3:], False)[:few].to(BF16))


def test_calls_on_streams_of_their_own(L):
    """Two streams at once, each with its workspace, given by `stream` or as the current one: the same as one after the other."""
    rows, cols, vocab = 700, 5000, 9000
    cfg = cfg_of(L, "layer", True, 1.0, 0.5)

    def make(seed):
        g, x, y, p = inputs(seed, rows, cols, BF16, BF16, BF16, 0, (True, True, True, True, True))
        z = torch.randn(rows, vocab, generator=g, device="cuda").to(BF16)
        w = torch.randn(100000, generator=g, device="cuda")
        st = dict(x=x, y=y, p=p, z=z, t=torch.randint(0, vocab, (rows,), generator=g, device="cuda"), w=w,
                  wg=torch.randn(100000, generator=g, device="cuda"),
                  ws=torch.empty(L.loco_join_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda"))
        new = lambda *s, like=F32: torch.empty(s, dtype=like, device="cuda")  # noqa: E731
        st.update(h=new(rows, cols, like=BF16), u=new(rows, cols, like=BF16), stats=new(4, rows), dx=new(rows, cols, like=BF16),
                  dy=new(rows, cols, like=BF16), dg=new(cols), lp=new(rows), lse=new(rows), dz=new(rows, vocab, like=BF16),
                  ids=new(rows, 9, like=torch.int64), alts=new(rows, 9), m=torch.zeros(100000, device="cuda"),
                  v=torch.zeros(100000, device="cuda"), one=torch.ones(rows, device="cuda"))
        st["list"] = L.make_adam_tensors([w], [st["wg"]], [st["m"]], [st["v"]])
        return st

    def run(st, stream):
        q = {k: t for k, t in st["p"].items() if k != "beta"}
        L.loco_join_forward(cfg, st["x"], st["y"], st["h"], st["u"], stats=st["stats"], stream=stream, **st["p"])
        L.loco_join_backward(cfg, st["h"], st["u"], st["h"], st["y"], st["stats"], st["dx"], st["dy"], dgamma=st["dg"],
                             workspace=st["ws"], stream=stream, **q)
        L.loco_logprob_forward(st["z"], st["t"], st["lp"], lse=st["lse"], top_ids=st["ids"], top_logp=st["alts"], stream=stream)
        L.loco_logprob_backward(st["z"], st["t"], st["lse"], st["dz"], dlogp=st["one"], stream=stream)
        L.loco_adam_tensors(st["list"], L.make_adam(), 1, stream=stream)
    outs = ("h", "u", "stats", "dx", "dy", "dg", "lp", "lse", "ids", "alts", "dz", "w", "m", "v")
    alone = []
    for seed in (61, 62):
        st = make(seed)
        run(st, None)
        alone.append([st[k].clone() for k in outs])
    states, streams = [make(61), make(62)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    run(states[0], streams[0])
    with torch.cuda.stream(streams[1]):
        run(states[1], None)
    torch.cuda.synchronize()
    for st, want in zip(states, alone):
        for k, b in zip(outs, want):
            assert torch.equal(st[k], b), k
