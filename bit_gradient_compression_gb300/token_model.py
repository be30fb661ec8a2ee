"""A stack of residual MLP blocks that predicts tokens, trained on one device with 8-bit optimizer states.

    h_0 = x,  u_0 = norm(h_0)
    y_l = w2_l act(w1_l u_l),  h_{l+1} = h_l + gate_l norm(y_l),  u_{l+1} = norm(h_{l+1})
    logits = head u_layers

over the library's entry points, with each parameter in a tensor of its own:

* forward: ``loco_norm_forward`` (u_0), for every block ``loco_linear_forward`` twice (the pre-activation kept in
  8 bits) and ``loco_join_forward`` (the block's output normalised, gated and added to the stream, and the sum
  normalised for the next block, in one pass), ``loco_linear_forward`` (the logits) and ``loco_logprob_forward``
  (log probabilities of the given tokens, entropies, the most likely tokens).
* backward: ``loco_logprob_backward`` (the gradient takes the logits' place), ``loco_linear_backward_weight`` and
  ``loco_linear_backward_input``, for every block ``loco_join_backward`` (both of its norms, the gate and the
  stream) and the products again, ``loco_norm_backward``.
* step: ``loco_adam_tensors`` on all parameters, two bytes of moments for each, which also writes the bf16
  parameters that the next forward pass reads.

The input rows are what lies in front of the stack (``backward`` returns their gradient).

    python -m bit_gradient_compression_gb300.token_model

trains it to predict the successor of every token of a fixed random cycle and prints the loss.
"""
from __future__ import annotations

import torch

from bit_gradient_compression_gb300 import loco as L

BF16, F32 = torch.bfloat16, torch.float32


class TokenModel:
    """The stack's parameters, their gradients and moments, on one device."""

    def __init__(self, vocab: int, hidden: int, ffn: int, layers: int, *, act: int = L.LOCO_ACT_SILU,
                 kind: int = L.LOCO_NORM_RMS, eps: float = 1e-5, dither: int = 1, device="cuda", seed: int = 0):
        self.V, self.H, self.F, self.layers, self.act = vocab, hidden, ffn, layers, act
        self.norm = L.make_norm(kind, eps)
        self.join = L.make_join(kind, eps, post=True)
        shapes = {"gamma0": (hidden,), "head": (vocab, hidden)}
        for i in range(layers):
            shapes |= {f"w1.{i}": (ffn, hidden), f"w2.{i}": (hidden, ffn), f"post_gamma.{i}": (hidden,),
                       f"gate.{i}": (hidden,), f"gamma.{i}": (hidden,)}
            if kind == L.LOCO_NORM_LAYER:
                shapes |= {f"post_beta.{i}": (hidden,), f"beta.{i}": (hidden,)}
        if kind == L.LOCO_NORM_LAYER:
            shapes["beta0"] = (hidden,)
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        dev = torch.device(device)
        self.master = {}
        for name, shape in shapes.items():
            if len(shape) == 2:
                self.master[name] = torch.randn(shape, generator=g, device=dev) * shape[1] ** -0.5
            else:
                self.master[name] = torch.full(shape, 0.0 if "beta" in name else 0.5 if "gate" in name else 1.0, device=dev)
        self.param = {k: v.to(BF16) for k, v in self.master.items()}         # what the passes read
        self.grad = {k: torch.zeros_like(v) for k, v in self.param.items()}  # what the passes write
        blocks = {k: -(-v.numel() // L.LOCO_STATE_BLOCK) for k, v in self.master.items()}
        codes = lambda dtype: [torch.zeros(n * L.LOCO_STATE_BLOCK, dtype=dtype, device=dev) for n in blocks.values()]  # noqa: E731
        steps = lambda: [torch.zeros(n, device=dev) for n in blocks.values()]  # noqa: E731
        # vectors (norms, gates) are not decayed
        self.tensors = L.make_adam_tensors(
            list(self.master.values()), list(self.grad.values()), codes(torch.int8), codes(torch.uint8), m_steps=steps(),
            v_steps=steps(), params_bf16=list(self.param.values()),
            decay_scales=[float(v.dim() == 2) for v in self.master.values()], dither=dither)
        self.t = 0

    def logits(self, x: torch.Tensor):
        """Logits [T, V] bf16 of x [T, H] bf16, and what the backward pass needs."""
        T, dev, p = x.shape[0], x.device, self.param
        new = lambda *shape, dtype=BF16: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        nb = -(-self.F // L.LOCO_CKPT_BLOCK)
        h, u = x, new(T, self.H)
        kept = {"x": x, "mean": new(T, dtype=F32), "rstd": new(T, dtype=F32), "blocks": []}
        L.loco_norm_forward(self.norm, x, p["gamma0"], p.get("beta0"), u, mean=kept["mean"], rstd=kept["rstd"])
        for i in range(self.layers):
            b = {"u": u, "codes": new(T, nb * L.LOCO_CKPT_BLOCK, dtype=torch.int8), "scales": new(T, nb, dtype=torch.uint8),
                 "y": new(T, self.H), "h": new(T, self.H), "stats": new(4, T, dtype=F32)}
            a, u = new(T, self.F), new(T, self.H)
            L.loco_linear_forward(b["u"], p[f"w1.{i}"], a, act=self.act, codes=b["codes"], scales=b["scales"])
            L.loco_linear_forward(a, p[f"w2.{i}"], b["y"])
            L.loco_join_forward(self.join, h, b["y"], b["h"], u, gamma=p[f"gamma.{i}"], beta=p.get(f"beta.{i}"),
                                post_gamma=p[f"post_gamma.{i}"], post_beta=p.get(f"post_beta.{i}"), gate=p[f"gate.{i}"],
                                stats=b["stats"])
            h = b["h"]
            kept["blocks"].append(b)
        out = new(T, self.V)
        L.loco_linear_forward(u, p["head"], out)
        kept["u"] = u
        return out, kept

    def forward(self, x: torch.Tensor, targets: torch.Tensor):
        """Log probabilities and entropies [T] of the targets [T] (negative: no target), and what the backward pass needs."""
        logits, kept = self.logits(x)
        logp, lse, entropy = (torch.empty(x.shape[0], device=x.device) for _ in range(3))
        L.loco_logprob_forward(logits, targets, logp, lse=lse, entropy=entropy)
        kept |= {"logits": logits, "targets": targets, "lse": lse, "entropy": entropy}
        return logp, entropy, kept

    def backward(self, kept, dlogp: torch.Tensor, dentropy: torch.Tensor | None = None) -> torch.Tensor:
        """dx [T, H] for the gradients of the log probabilities and the entropies [T]; every parameter's gradient goes to
        its tensor in self.grad.  The logits in `kept` are overwritten."""
        T, dev, p, g = dlogp.shape[0], dlogp.device, self.param, self.grad
        new = lambda *shape: torch.empty(shape, dtype=BF16, device=dev)  # noqa: E731
        # of this pass, like its other buffers: a captured one writes to it as long as its graph lives
        workspace = torch.empty(max(L.loco_join_workspace_bytes(T, self.H), L.loco_norm_workspace_bytes(T, self.H)),
                                dtype=torch.uint8, device=dev)
        dz = kept["logits"]
        L.loco_logprob_backward(dz, kept["targets"], kept["lse"], dz, dlogp=dlogp, entropy=kept["entropy"], dentropy=dentropy)
        du, dh = new(T, self.H), None
        L.loco_linear_backward_weight(dz, g["head"], x=kept["u"])
        L.loco_linear_backward_input(dz, p["head"], du)
        for i in reversed(range(self.layers)):
            b = kept["blocks"][i]
            dx, dy, a, da = new(T, self.H), new(T, self.H), new(T, self.F), new(T, self.F)
            L.loco_join_backward(self.join, dh, du, b["h"], b["y"], b["stats"], dx, dy, gamma=p[f"gamma.{i}"],
                                 post_gamma=p[f"post_gamma.{i}"], post_beta=p.get(f"post_beta.{i}"), gate=p[f"gate.{i}"],
                                 dgamma=g[f"gamma.{i}"], dbeta=g.get(f"beta.{i}"), dpost_gamma=g[f"post_gamma.{i}"],
                                 dpost_beta=g.get(f"post_beta.{i}"), dgate=g[f"gate.{i}"], workspace=workspace)
            L.loco_ckpt_decode(b["codes"], b["scales"], a, act=self.act)
            L.loco_linear_backward_weight(dy, g[f"w2.{i}"], x=a)
            L.loco_linear_backward_input(dy, p[f"w2.{i}"], da, act=self.act, codes=b["codes"], scales=b["scales"])
            L.loco_linear_backward_weight(da, g[f"w1.{i}"], x=b["u"])
            L.loco_linear_backward_input(da, p[f"w1.{i}"], du)
            dh = dx
        dx = new(T, self.H)
        L.loco_norm_backward(self.norm, du, p["gamma0"], kept["rstd"], dx, x=kept["x"], mean=kept["mean"], residual=dh,
                             dgamma=g["gamma0"], dbeta=g.get("beta0"), workspace=workspace)
        return dx

    def step(self, hp, grad_scale: torch.Tensor | None = None):
        """One Adam(W) step on every parameter; grad_scale: one fp32 value on the device, the factor of every gradient."""
        self.t += 1
        L.loco_adam_tensors(self.tensors, hp, self.t, grad_scale=grad_scale)

    def likely(self, x: torch.Tensor, top: int, temperature: float = 1.0):
        """The `top` most likely next tokens of every row of x [T, H] and their log probabilities, the likeliest first."""
        logits, _ = self.logits(x)
        ids = torch.empty(x.shape[0], top, dtype=torch.int64, device=x.device)
        logp = torch.empty(x.shape[0], top, device=x.device)
        L.loco_logprob_forward(logits, None, None, top_ids=ids, top_logp=logp, scale=1.0 / temperature)
        return ids, logp


def train(steps: int = 200, tokens: int = 512, vocab: int = 1000, hidden: int = 128, ffn: int = 344, layers: int = 2,
          lr: float = 2e-3, seed: int = 1):
    """Mean negative log probabilities of a model that learns a fixed random cycle of tokens."""
    model = TokenModel(vocab, hidden, ffn, layers, seed=seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    table = torch.randn(vocab, hidden, generator=g, device="cuda").to(BF16)
    cycle = torch.randperm(vocab, generator=g, device="cuda")
    after = torch.empty_like(cycle)
    after[cycle] = cycle.roll(-1)
    hp, losses = L.make_adam(lr=lr, beta1=0.9, beta2=0.95), []
    dlogp = torch.full((tokens,), -1.0 / tokens, device="cuda")
    for _ in range(steps):
        now = torch.randint(vocab, (tokens,), generator=g, device="cuda")
        logp, _, kept = model.forward(table[now], after[now])
        losses.append(-logp.mean())
        model.backward(kept, dlogp)
        model.step(hp)
    return [float(v) for v in losses]


if __name__ == "__main__":
    got = train()
    for i in range(0, len(got), 20):
        print(f"step {i:4d}  loss {got[i]:.5f}")
    print(f"step {len(got) - 1:4d}  loss {got[-1]:.5f}")
