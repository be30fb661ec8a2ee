"""The token model: joins, log probabilities and AdamW on many tensors run together with the layer calls."""
import pytest
import torch

import layers_ref as R

pytestmark = pytest.mark.gpu
rel = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())  # noqa: E731


@pytest.fixture(scope="module")
def M():
    from bit_gradient_compression_gb300 import token_model
    return token_model


def make(M, kind="rms", vocab=1000, hidden=128, ffn=352, layers=2, T=160, seed=3):
    """A model whose vectors are not all alike, rows for it, and targets of which some are missing."""
    model = M.TokenModel(vocab, hidden, ffn, layers, seed=seed, kind=M.L.LOCO_NORM_RMS if kind == "rms" else M.L.LOCO_NORM_LAYER)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    for k, v in model.master.items():
        if v.dim() == 1:
            v += 0.2 * torch.randn(v.shape, generator=g, device="cuda")
        model.param[k].copy_(v)
    x = torch.randn(T, hidden, generator=g, device="cuda").to(torch.bfloat16)
    targets = torch.randint(vocab, (T,), generator=g, device="cuda")
    targets[::7] = -1
    return model, x, targets, g


def network(p, x, targets, kind, layers):
    """log probabilities and entropies of the model with parameters p, in the type of p."""
    def norm(v, gamma, beta):
        m = v.mean(1, keepdim=True) if kind == "layer" else 0.0
        return (v - m) * ((v - m).square().mean(1, keepdim=True) + 1e-5).rsqrt() * gamma + (0.0 if beta is None else beta)
    h, u = x, norm(x, p["gamma0"], p.get("beta0"))
    for i in range(layers):
        y = R.act(u @ p[f"w1.{i}"].t(), "silu") @ p[f"w2.{i}"].t()
        h = h + p[f"gate.{i}"] * norm(y, p[f"post_gamma.{i}"], p.get(f"post_beta.{i}"))
        u = norm(h, p[f"gamma.{i}"], p.get(f"beta.{i}"))
    logp = torch.log_softmax(u @ p["head"].t(), 1)
    entropy = -(logp.exp() * logp).sum(1)
    given = logp.gather(1, targets.clamp_min(0)[:, None])[:, 0]
    return torch.where(targets >= 0, given, torch.zeros_like(given)), entropy


@pytest.mark.parametrize("kind,vocab,hidden,ffn,layers,T", [("rms", 1000, 128, 352, 2, 160), ("layer", 1001, 72, 200, 1, 33),
                                                            ("rms", 2048, 64, 96, 2, 1), ("layer", 512, 256, 688, 2, 300)])
def test_gradients(M, kind, vocab, hidden, ffn, layers, T):
    """Every gradient within 2.5 % a block and 1.5 % of the 64-bit network's on the same parameters (2-norms).

    A block's kept pre-activations are off by at most 1.1 % of their size (a step of 1/64 of a block's largest value,
    2.5 times the usual one, over sqrt(12)), and seven bf16 roundings of 2^-9 (0.2 %) stand between two blocks.  In
    front of the blocks: the logits' rounding, 2^-9 of values of up to 4 (0.8 % of a probability), the gradient of
    the logits', of u's and the parameters' own, 0.2 % each.
    """
    model, x, targets, g = make(M, kind, vocab, hidden, ffn, layers, T, seed=5)
    targets[0] = 3
    logp, entropy, kept = model.forward(x, targets)
    dlogp = torch.randn(T, generator=g, device="cuda")
    dentropy = 0.1 * torch.randn(T, generator=g, device="cuda")
    dx = model.backward(kept, dlogp, dentropy)

    p = {k: v.double().requires_grad_(True) for k, v in model.param.items()}
    x64 = x.double().requires_grad_(True)
    want, want_h = network(p, x64, targets, kind, layers)
    (want * dlogp.double() + want_h * dentropy.double()).sum().backward()
    # a log probability: 2^-9 of the logits, and eight roundings of 2^-9 of rows of H values of size 1 on the way to them
    tol = 2.0 ** -9 * 4 * 2 + 8 * layers * 2.0 ** -9 * 2
    assert float((logp.double() - want.detach()).abs().max()) < tol
    assert float((entropy.double() - want_h.detach()).abs().max()) < tol
    bound = 0.015 + 0.025 * layers
    assert rel(dx, x64.grad) < bound
    for k in p:
        assert rel(model.grad[k], p[k].grad) < bound, k


def test_gradients_against_differences(M):
    """The loss's change along the gradient is what the gradient says.

    The step is taken both ways, so its square drops out; logits move by up to 0.3, of which the cube is a hundredth; the
    gradient is off by 6.5 % (above); and the loss by the logits' rounding, 2^-9 of up to 4 in 160 rows of random sign,
    6e-4, of a change of 0.1 or more: 9 % in all.
    """
    model, x, targets, _ = make(M)
    n = (targets >= 0).sum()
    mean = lambda: float(model.forward(x, targets)[0].double().sum() / n)  # noqa: E731
    logp, _, kept = model.forward(x, targets)
    model.backward(kept, torch.full_like(logp, 1.0) / n)
    size = sum(float(v.double().square().sum()) for v in model.grad.values()) ** 0.5
    reach, said, at = 0.06 / size, 0.0, []  # each way 0.06 by the gradient
    start = {k: v.clone() for k, v in model.master.items()}
    ends = []
    for sign in (1.0, -1.0):
        for k, v in model.param.items():
            v.copy_(start[k] + sign * reach / size * model.grad[k].float())
        ends.append({k: v.double() for k, v in model.param.items()})
        at.append(mean())
    # the parameters are rounded to bf16: where they really went
    for k in start:
        said += float(((ends[0][k] - ends[1][k]) * model.grad[k].double()).sum())
    assert said > 0.1 and abs(at[0] - at[1] - said) < 0.09 * said


def test_steps_follow_the_formula(M):
    """Three steps of the model against its own gradients and moments in 64 bits, states in 8 bits read back each time."""
    model, x, targets, _ = make(M, layers=1)
    L, hp = M.L, M.L.make_adam(lr=1e-3, beta1=0.9, beta2=0.95, weight_decay=0.1)
    scale = torch.tensor([0.5], device="cuda")
    _, _, ms, vs, m_steps, v_steps, _ = model.tensors.tensors
    for t in (1, 2, 3):
        logp, _, kept = model.forward(x, targets)
        model.backward(kept, torch.full_like(logp, -1.0 / logp.numel()))
        before, moments = {k: v.double() for k, v in model.master.items()}, []
        for i, v in enumerate(model.master.values()):
            pair = [torch.empty(v.numel(), device="cuda") for _ in range(2)]
            L.loco_adam_state_decode(ms[i], m_steps[i], pair[0])
            L.loco_adam_state_decode(vs[i], v_steps[i], pair[1])
            moments.append([q.double().view(v.shape) for q in pair])
        model.step(hp, scale)
        for (k, p), (m, v) in zip(before.items(), moments):
            g = 0.5 * model.grad[k].double()
            m, v = 0.9 * m + 0.1 * g, 0.95 * v + 0.05 * g * g
            p = p * (1.0 - (1e-4 if p.dim() == 2 else 0.0))
            step = 1e-3 * (m / (1 - 0.9 ** t)) / ((v / (1 - 0.95 ** t)).sqrt() + 1e-8)
            # the constants beta and lr are fp32 (2^-24 of each), a dozen roundings to 2^-24 follow
            tol = 2.0 ** -20 * step.abs() + 4 * 2.0 ** -24 * p.abs() + 1e-12
            # and where m's two terms cancel, theirs
            tol += 2.0 ** -20 * 1e-3 * (g.abs() * 0.1 + m.abs()) / (1 - 0.9 ** t) / ((v / (1 - 0.95 ** t)).sqrt() + 1e-8)
            assert bool(((model.master[k].double() - (p - step)).abs() <= tol).all()), k
            # (the copy of an fp32 parameter is its nearest bf16 value, with dither too)
            assert torch.equal(model.param[k], model.master[k].to(torch.bfloat16)), k


def test_same_twice_and_captured(M):
    """The same passes give the same bits: twice, on another stream, and replayed from two graphs that share the workspace."""
    model, x, targets, _ = make(M, T=300)

    def passes():
        logp, entropy, kept = model.forward(x, targets)
        dx = model.backward(kept, torch.full_like(logp, -1.0 / 300), torch.full_like(logp, 1e-3))
        return logp, entropy, dx
    first = [v.clone() for v in passes()] + [v.clone() for v in model.grad.values()]
    same = lambda out: all(torch.equal(a, b) for a, b in zip(first, [*out, *model.grad.values()]))  # noqa: E731
    assert same(passes())
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        out = passes()
    torch.cuda.current_stream().wait_stream(other)
    assert same(out)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = passes()
        graphs.append((graph, out))
    for graph, out in graphs + graphs[::-1]:
        for v in (*out, *model.grad.values()):
            v.zero_()
        graph.replay()
        assert same(out)


@pytest.mark.parametrize("T", [1, 37])
def test_likely_tokens(M, T):
    """The list is the logits' own, in order; a temperature changes the log probabilities, not the order."""
    model, x, _, _ = make(M, T=T)
    logits, _ = model.logits(x)
    ids, logp = model.likely(x, 5, temperature=2.0)
    want = torch.log_softmax(logits.double() / 2.0, 1)
    order = torch.argsort(logits.double(), dim=1, descending=True, stable=True)[:, :5]
    assert torch.equal(ids, order)
    # as for the operator itself: the exponent's roundings (2^-24 of a hundred) and the sum's
    assert float((logp.double() - want.gather(1, ids)).abs().max()) < 2e-5


def test_training_runs(M):
    losses = M.train(steps=6, tokens=64, vocab=100, hidden=64, ffn=96)
    assert len(losses) == 6 and all(v == v and abs(v) < 100 for v in losses)
    assert M.L.loco_linear_timeouts() == 0
