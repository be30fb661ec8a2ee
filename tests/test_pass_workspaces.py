"""Workspaces of the models' backward passes: each pass has its own, so that what a captured pass or one on another stream
writes to is not given back, or to another pass, while it may still be written."""
import pytest
import torch


def make(kind, device):
    """(model, one forward and backward pass on T rows that returns the gradients it made)."""
    if kind == "token":
        from bit_gradient_compression_gb300 import token_model as M
        model = M.TokenModel(300, 64, 96, 2, device=device, kind=M.L.LOCO_NORM_LAYER)

        def run(x):
            logp, _, kept = model.forward(x, torch.arange(len(x), device=device) % 300)
            return model.backward(kept, torch.full_like(logp, 1e-2))
    else:
        from bit_gradient_compression_gb300 import mlp_block as M
        model = M.MlpBlock(64, 96, device=device)

        def run(x):
            out, kept = model.forward(x)
            return model.backward(torch.full_like(out, 1e-2), kept)
    return M.L, model, run


@pytest.mark.parametrize("kind", ["token", "mlp"])
def test_every_pass_has_its_own(monkeypatch, kind):
    """On the CPU, with the calls themselves left out: the workspaces that two passes hand over share no memory."""
    from bit_gradient_compression_gb300 import build
    build.build()
    L, _, run = make(kind, "cpu")
    seen = []
    for name in L.EXPORTS:
        if name.split("_")[1] in ("norm", "join", "linear", "logprob", "ckpt") and not name.endswith("_bytes"):
            monkeypatch.setattr(L, name, lambda *a, workspace=None, **k: seen.append(workspace))
    passes = []
    for T in (8, 8, 700, 8):
        seen.clear()
        run(torch.zeros(T, 64, dtype=torch.bfloat16))
        passes.append([w for w in seen if w is not None and w.numel() > 0])    # (held: their memory is not used again)
        assert passes[-1]
    spans = [{(w.data_ptr(), w.data_ptr() + w.numel()) for w in p} for p in passes]
    for i, a in enumerate(spans):
        for b in spans[:i]:
            assert all(x[1] <= y[0] or y[1] <= x[0] for x in a for y in b)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["token", "mlp"])
def test_captured_before_a_larger_batch(kind):
    """A graph captured at few rows, then a pass at more, then replays: the gradients of few rows, and memory that was
    handed out in between is as it was."""
    L, model, run = make(kind, "cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    x = torch.randn(40, 64, generator=g, device="cuda").to(torch.bfloat16)
    grads = lambda: list(model.grad.values()) if kind == "token" else [model.grad]  # noqa: E731
    want = [run(x).clone()] + [v.clone() for v in grads()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx = run(x)
    run(torch.randn(700, 64, generator=g, device="cuda").to(torch.bfloat16))
    sizes = {L.loco_join_workspace_bytes(40, 64), L.loco_norm_workspace_bytes(40, 64), L.loco_linear_workspace_bytes(96)}
    others = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(8)]
    for _ in range(2):
        for v in grads():
            v.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, [dx, *grads()]))
        assert all(bool((o == 0x5A).all()) for o in others)
