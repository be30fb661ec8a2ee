"""The binding's marshalling in C: it gives up on whatever is not as an entry point wants it, and gives the
entry points what the marshalling in Python gives them."""
import types

import pytest

torch = pytest.importorskip("torch")

from bit_gradient_compression_gb300 import loco as L  # noqa: E402

marshal = pytest.importorskip("bit_gradient_compression_gb300._marshal", reason="built without Python's headers")
B = torch.bfloat16
NAMES = ("ckpt_encode", "ckpt_decode", "norm_forward", "norm_backward", "linear_forward", "linear_backward_input",
         "linear_backward_weight")


def t(*shape, d=torch.float32):
    return torch.zeros(*shape, dtype=d)


def test_same_functions():
    L._dtypes()
    assert all(getattr(L, "loco_" + name) and getattr(marshal, name) for name in NAMES)
    for name in NAMES:
        with pytest.raises(TypeError):
            getattr(marshal, name)(None)


@pytest.mark.parametrize("call", [
    lambda c, s: marshal.ckpt_encode(None, c, s, 0),
    lambda c, s: marshal.ckpt_encode(t(4, 64), c, s, "stream"),
    lambda c, s: marshal.ckpt_encode(t(4, 64), c.float(), s, 0),
    lambda c, s: marshal.ckpt_encode(t(4, 64), s, c, 0),
    lambda c, s: marshal.ckpt_encode(t(4, 64), c.t(), s, 0),
    lambda c, s: marshal.ckpt_encode(t(8, 64), c, s, 0),
    lambda c, s: marshal.ckpt_encode(t(4, 64, d=torch.float64), c, s, 0),
    lambda c, s: marshal.ckpt_encode(t(64, 4).t(), c, s, 0),
    lambda c, s: marshal.ckpt_encode(t(1, 4, 64), c, s, 0),
    lambda c, s: marshal.ckpt_encode([[0.0]], c, s, 0),
    lambda c, s: marshal.ckpt_decode(c, s, t(4, 64), 0, t(64), t(64, d=B), 0),
    lambda c, s: marshal.ckpt_decode(c, s, t(4, 64), "act", None, None, 0),
    lambda c, s: marshal.ckpt_decode(c, s, t(4, 64), 0, t(128)[::2], None, 0),
    lambda c, s: marshal.norm_forward(0, 1e-5, t(4, 64), None, None, t(4, 64), t(5), None, None, None, 0),
    lambda c, s: marshal.norm_forward(0, 1e-5, t(4, 64), None, None, t(4, 64), t(4, d=B), None, None, None, 0),
    lambda c, s: marshal.norm_forward(0, "eps", t(4, 64), None, None, t(4, 64), None, None, None, None, 0),
    # x, residual and dx: any two of them unlike, whichever the third is
    lambda c, s: marshal.norm_backward(0, 1e-5, t(4, 64), None, t(4), t(4, 64), t(4, 64, d=B), t(4), None, None, None,
                                       None, None, None, 0),
    lambda c, s: marshal.norm_backward(0, 1e-5, t(4, 64), None, t(4), t(4, 64), t(4, 64, d=B), t(4), None, None,
                                       t(4, 64), None, None, None, 0),
    lambda c, s: marshal.norm_backward(0, 1e-5, t(4, 64), None, t(4), t(4, 64), t(4, 64), t(4), None, None,
                                       t(4, 64, d=B), None, None, None, 0),
    lambda c, s: marshal.norm_backward(0, 1e-5, t(4, 64), None, t(4), t(4, 64), None, t(4), c, s, t(4, 64, d=B), None,
                                       None, None, 0),
    lambda c, s: marshal.norm_backward(0, 1e-5, t(4, 64), None, t(4), t(4, 64), t(4, 64), t(4), None, None, None, None,
                                       None, t(64), 0),
    lambda c, s: marshal.linear_forward(t(4, 32), t(64, 32, d=B), t(4, 64), 0, None, None, None, None, 0, None),
    lambda c, s: marshal.linear_forward(t(4, 32, d=B), t(64, 32, d=B), t(4, 64), 0, None, t(4, 64, d=B), None, None, 0,
                                        None),
    lambda c, s: marshal.linear_backward_input(t(4, 32, d=B), t(31, 64, d=B), t(4, 64), 0, c, s, None, 0, None),
    lambda c, s: marshal.linear_backward_weight(t(4, 32, d=B), t(32, 64), t(4, 64), None, None, None, None, None, None,
                                                0, None),
    lambda c, s: marshal.linear_backward_weight(t(4, 32, d=B), t(32, 64), None, c, s, None, None, t(32, d=B), None, 0,
                                                None),
])
def test_gives_up(call):
    L._dtypes()
    c, s = t(4, 64, d=torch.int8), t(4, 2, d=torch.uint8)
    assert call(c, s) is None


def both(monkeypatch, run):
    """run() with the marshalling in C, and without it."""
    L._dtypes()
    seen = []
    spy = types.SimpleNamespace(**{n: (lambda f: lambda *a: seen.append(f(*a)) or seen[-1])(getattr(marshal, n))
                                   for n in NAMES})
    monkeypatch.setattr(L, "_marshal", spy)
    first = run()
    assert seen and all(v == L.LOCO_OK for v in seen)          # none of them fell back
    monkeypatch.setattr(L, "_marshal", types.SimpleNamespace(**{n: lambda *a: None for n in NAMES}))
    return first, run()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,pad", [(1, 256, 0), (5, 100, 0), (37, 96, 8)])
def test_same_results(monkeypatch, rows, cols, pad):
    gen = torch.Generator(device="cuda").manual_seed(7)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    wide = lambda n, d: torch.zeros(rows, n + pad, device="cuda", dtype=d)[:, :n]  # noqa: E731
    x, dy = wide(cols, B).copy_(r(rows, cols)), wide(cols, B).copy_(r(rows, cols))
    w, gamma, beta = r(64, cols).to(B), r(cols), r(cols)
    nb = -(-cols // 32)

    def run():
        y, dx, z, dz = wide(cols, B), wide(cols, B), wide(64, torch.float32), wide(cols, torch.float32)
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        codes = torch.zeros(rows, nb * 32, dtype=torch.int8, device="cuda")
        scales = torch.zeros(rows, nb, dtype=torch.uint8, device="cuda")
        dg, db, dw = torch.empty_like(gamma), torch.empty_like(beta), torch.empty(64, cols, device="cuda")
        ws = torch.empty(L.loco_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        cfg = L.make_norm()
        L.loco_norm_forward(cfg, x, gamma, beta, y, mean=mean, rstd=rstd, codes=codes, scales=scales)
        L.loco_norm_backward(cfg, dy, gamma, rstd, dx, x=x, mean=mean, residual=x, dgamma=dg, dbeta=db, workspace=ws)
        out = wide(cols, torch.float32)
        L.loco_ckpt_decode(codes, scales, out, act=L.LOCO_ACT_SILU, gamma=gamma, beta=beta)
        c2, s2 = torch.zeros_like(codes), torch.zeros_like(scales)
        L.loco_ckpt_encode(out, c2, s2)
        L.loco_linear_forward(y, w, z, act=L.LOCO_ACT_RELU, bias=r(64).zero_())
        dzb = z.to(B)
        L.loco_linear_backward_input(dzb, w, dz, act=L.LOCO_ACT_SILU, codes=c2, scales=s2)
        L.loco_linear_backward_weight(dzb, dw, codes=codes, scales=scales, gamma=gamma, beta=beta,
                                      workspace=ws.new_empty(L.loco_linear_workspace_bytes(64)))
        return y, dx, mean, rstd, codes, scales, dg, db, out, c2, s2, z, dz, dw

    for a, b in zip(*both(monkeypatch, run)):
        assert torch.equal(a, b)
