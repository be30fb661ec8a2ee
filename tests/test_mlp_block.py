"""The MLP block over the layer entry points: its gradients against 64-bit autograd, and training with it."""
import pytest
import torch

import layers_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    from bit_gradient_compression_gb300 import mlp_block
    return mlp_block


@pytest.mark.parametrize("T,H,F,kind,act", [(160, 128, 352, "layer", "gelu_tanh"), (33, 72, 200, "rms", "silu"),
                                            (1, 64, 96, "layer", "gelu"), (512, 256, 688, "layer", "relu")])
def test_gradients(M, T, H, F, kind, act):
    """Every gradient within 3 % (2-norm) of the 64-bit network's on the same parameters.

    Kept values are off by a step's twelfth root of variance, a step being 1/64 to 1/128 of a block's largest
    value: at most 2.5 / 64 / sqrt(12) = 1.1 % of their own size for the normal values here; bf16
    activations and gradients add 2^-9 each (0.2 %, four of them in a row)."""
    L = M.L
    block = M.MlpBlock(H, F, act=getattr(L, "LOCO_ACT_" + act.upper()),
                       kind=L.LOCO_NORM_LAYER if kind == "layer" else L.LOCO_NORM_RMS, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    for name in ("gamma", "beta", "b1", "b2"):
        v = block.view(block.param, name)
        v += (0.2 * torch.randn(v.shape, generator=g, device="cuda")).to(v.dtype)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    c = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    out, kept = block.forward(x)
    dx = block.backward(c, kept)

    p = {k: block.view(block.param, k).double().requires_grad_(True) for k in block.slices}
    x64 = x.double().requires_grad_(True)
    m = x64.mean(1, keepdim=True) if kind == "layer" else 0.0
    xh = (x64 - m) * ((x64 - m).square().mean(1, keepdim=True) + 1e-5).rsqrt()
    z = (xh * p["gamma"] + p["beta"]) @ p["w1"].t() + p["b1"]
    h = R.act(z, act)
    if act == "relu":
        # its slope is a step, and the backward pass takes it at the kept values: those below half a step are
        # kept as 0 and have slope 0
        codes, scales = kept["pre"]
        slope = (R.decode(codes, scales, F) > 0).double()
        h = h.detach() + slope * (z - z.detach())
    want = x64 + h @ p["w2"].t() + p["b2"]
    (want * c.double()).sum().backward()
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert rel(out, want.detach()) < 0.01
    assert rel(dx, x64.grad) < 0.03
    for k in block.slices:
        assert rel(block.view(block.grad, k), p[k].grad) < 0.03, k


def test_training_reduces_the_loss(M):
    losses = M.train(steps=120, tokens=256, hidden=128, ffn=344)
    assert all(v == v for v in losses)
    assert sum(losses[-10:]) < 0.5 * sum(losses[:10])


def test_two_ranks_average(M):
    """Two ranks' packed buckets step both replicas to the same parameters."""
    a, b = M.MlpBlock(64, 96, seed=5), M.MlpBlock(64, 96, seed=5)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    hp = M.L.make_adam(lr=1e-3)
    for _ in range(3):
        packed = []
        for blk in (a, b):
            x = torch.randn(40, 64, generator=g, device="cuda").to(torch.bfloat16)
            out, kept = blk.forward(x)
            blk.backward((out.float() * 1e-3).to(torch.bfloat16), kept)
            packed.append(blk.compress())
        codes, scales = [p[0] for p in packed], [p[1] for p in packed]
        for blk in (a, b):
            blk.step(codes, scales, hp)
        assert torch.equal(a.param, b.param) and torch.equal(a.master, b.master)
