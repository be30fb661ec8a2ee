"""Operands of linear layers copied to aligned rows: the copy itself, and the products that make it."""
import types

import pytest

torch = pytest.importorskip("torch")

from bit_gradient_compression_gb300 import loco as L  # noqa: E402

B = torch.bfloat16


def test_refusals():
    call = lambda src=0x10000, lds=40, rows=4, cols=33, dst=0x20000, ldd=40: (  # noqa: E731
        L.lib.loco_linear_align(src, lds, rows, cols, dst, ldd, 0))
    big = L.LOCO_MAX_DIM + 1
    for bad in (dict(src=0), dict(dst=0), dict(lds=32), dict(ldd=32), dict(ldd=41), dict(ldd=44), dict(rows=-1),
                dict(cols=-1), dict(rows=big), dict(cols=big), dict(ldd=big + 7), dict(dst=0x10000),
                dict(dst=0x10000 + 2 * 3 * 40 + 2 * 32 - 2 * 32)):
        assert call(**bad) == L.LOCO_ERR_INVALID_ARG, bad
        assert L.lib.loco_last_error() != b""
    for bad in (dict(src=0x10001), dict(dst=0x20008), dict(dst=0x20002)):
        assert call(**bad) == L.LOCO_ERR_MISALIGNED, bad
    assert call(rows=0, src=0, dst=0) == L.LOCO_OK and call(cols=0, src=0, dst=0) == L.LOCO_OK
    if not torch.cuda.is_available():
        assert call() == L.LOCO_ERR_INVALID_ARG                # nobody's device memory
    t = lambda *s, d=B: torch.zeros(*s, dtype=d)  # noqa: E731
    for src, dst, text in ((t(4, 33, d=torch.float32), t(4, 40), "bfloat16"), (t(4, 33), t(4, 40), "dst must be"),
                           (t(33), t(4, 40), "two-dimensional")):
        with pytest.raises(ValueError, match=text):
            L.loco_linear_align(src, dst, stream=0)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,pitch,start", [
    (1, 1, 1, 0), (1, 1, 1, 3), (1, 7, 7, 1), (3, 5, 5, 0), (5, 8, 9, 0), (5, 16, 16, 0), (7, 17, 17, 5), (2, 15, 31, 7),
    (33, 255, 255, 0), (9, 1023, 1025, 1), (9, 1024, 1025, 0), (5, 1025, 1025, 6), (4, 4099, 4101, 2), (300, 33, 35, 4),
    (2000, 3, 3, 1)])
def test_copy(rows, cols, pitch, start):
    """Every value, the zeros behind them, and nothing else; rows that start on any two-byte boundary."""
    buf = torch.arange(start + rows * pitch + 8, device="cuda").remainder(30011).add(1).to(torch.int16).view(B)
    src = buf[start:start + rows * pitch].view(rows, pitch)[:, :cols]
    ldd = (cols + 7) // 8 * 8 + 8
    whole = torch.full((rows * ldd + 16,), -7, dtype=torch.int16, device="cuda")
    dst = whole[8:8 + rows * ldd].view(rows, ldd)
    L.loco_linear_align(src, dst.view(B)[:, :cols])
    want = torch.full((rows, ldd), -7, dtype=torch.int16, device="cuda")
    want[:, :ldd - 8] = 0
    want[:, :cols] = src.view(torch.int16)
    assert torch.equal(dst, want) and bool((whole[:8] == -7).all()) and bool((whole[8 + rows * ldd:] == -7).all())


def products(T, N, K, pads, stream=None):
    """The three products of one layer, of operands with pads[i] columns behind them, and of aligned copies."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda rows, cols, pad: torch.randn(rows, cols + pad, device="cuda", generator=gen).to(B)[:, :cols]  # noqa: E731
    x, w, dy = r(T, K, pads[0]), r(N, K, pads[1]), r(T, N, pads[2])
    xb = x.contiguous()
    nb = -(-K // 32)
    codes, scales = torch.empty(T, nb * 32, dtype=torch.int8, device="cuda"), torch.empty(T, nb, dtype=torch.uint8, device="cuda")
    L.loco_ckpt_encode(xb, codes, scales)

    def run(x, w, dy):
        o = [torch.empty(s, dtype=d, device="cuda") for s, d in (((T, N), B), ((T, K), torch.float32), ((N, K), B),
                                                                  ((N, K), torch.float32), ((N,), B))]
        L.loco_linear_forward(x, w, o[0], act=L.LOCO_ACT_SILU, stream=stream)
        L.loco_linear_backward_input(dy, w, o[1], stream=stream)
        L.loco_linear_backward_weight(dy, o[2], x=x, db=o[4], stream=stream)
        L.loco_linear_backward_weight(dy, o[3], codes=codes, scales=scales, stream=stream)
        return o

    def aligned(t):
        c = torch.zeros(t.shape[0], (t.shape[1] + 7) // 8 * 8, dtype=B, device="cuda")[:, :t.shape[1]]
        return c.copy_(t)

    return run, (x, w, dy), tuple(aligned(t) for t in (x, w, dy)), (xb, w, dy)


SHAPES = [(333, 1407, 1031, (0, 0, 0)), (96, 2000, 2040, (1, 3, 0)), (1000, 600, 640, (0, 0, 1)), (130, 1511, 2000, (8, 0, 0))]


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K,pads", SHAPES)
@pytest.mark.parametrize("path", ["c", "python", "stream"])
def test_products(monkeypatch, T, N, K, pads, path):
    """The bits of the same product of operands that were aligned by hand."""
    assert T * N * K >= L.ALIGN_WORK and T >= L.ALIGN_ROWS
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if path == "stream" else None
    run, given, aligned, _ = products(T, N, K, pads, stream)
    torch.cuda.synchronize()
    copies = []
    real = L.lib.loco_linear_align
    if path != "c":
        L._dtypes()
        none = {n: lambda *a: None for n in dir(L._marshal) if n.startswith(("norm", "linear"))}
        if path == "python":
            monkeypatch.setattr(L, "_marshal", types.SimpleNamespace(**none))
        monkeypatch.setattr(L.lib, "loco_linear_align", lambda *a: copies.append(a) or real(*a))
    got = run(*given)
    if path != "c":
        assert copies
    del copies[:]
    want = run(*aligned)
    assert not copies
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_no_memory_and_small_products(monkeypatch):
    """Without memory for the copies, and below the sizes at which they pay, the operands are read as they lie."""
    T, N, K, pads = SHAPES[0]
    run, given, _, (x, w, dy) = products(T, N, K, pads)
    asked = []
    monkeypatch.setattr(L, "_scratch", lambda n: asked.append(n))
    got = run(*given)
    assert asked and not any(asked[i] <= 0 for i in range(len(asked)))
    z = x.double() @ w.double().t()
    want = z / (1 + torch.exp(-z))
    # bf16 outputs: half a unit in the last place, and fp32 sums of K products
    assert (got[0].double() - want).abs().max() <= 2 ** -8 * want.abs().max()
    want = dy.double() @ w.double()
    assert (got[1].double() - want).abs().max() <= N * 2 ** -23 * (dy.double().abs() @ w.double().abs()).max()
    del asked[:]
    small, given, _, _ = products(L.ALIGN_ROWS - 1, N, K, pads)
    small(*given)
    assert not asked


@pytest.mark.gpu
def test_in_a_graph():
    T, N, K, pads = SHAPES[0]
    run, given, aligned, _ = products(T, N, K, pads)
    want = run(*aligned)
    run(*given)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(*given)
    for o in got:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
