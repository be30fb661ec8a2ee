"""A transformer's MLP block trained from its activations' 8-bit checkpoints to the compressed step.

One pre-norm block, ``out = x + w2 act(w1 norm(x) + b1) + b2``, over the library's layer entry points,
with its parameters and their gradients in one flat bucket each, as a data-parallel step keeps them:

* forward: ``loco_norm_forward`` (the normalised rows kept in 8 bits), ``loco_linear_forward`` (bias and
  activation in the product's epilogue, the pre-activation kept in 8 bits), ``loco_linear_forward`` (bias
  and residual).  Of [T, H] and [T, F] activations, one byte and 1/32 per value is kept for the backward
  pass; neither the input, nor the norm's output, nor the activation's.
* backward: ``loco_ckpt_decode`` (the activation again), ``loco_linear_backward_weight`` and
  ``loco_linear_backward_input`` (through the activation's slope), the first layer's weight gradient
  straight from the codes of the normalised rows, ``loco_norm_backward`` (the residual stream's
  gradient added); every parameter's gradient lands in its slice of the gradient bucket.
* step: ``loco_compress`` of the bucket and ``loco_adam_step_bf16`` on the ranks' packed buckets, which
  also writes the bf16 parameters that the next forward pass reads.

    python -m bit_gradient_compression_gb300.mlp_block

trains the block to imitate a fixed random one on random inputs and prints the loss.
"""
from __future__ import annotations

import torch

from bit_gradient_compression_gb300 import loco as L


class MlpBlock:
    """The block's parameters, their flat buckets and one rank's compression state, on one device."""

    def __init__(self, hidden: int, ffn: int, *, act: int = L.LOCO_ACT_GELU_TANH, kind: int = L.LOCO_NORM_LAYER,
                 eps: float = 1e-5, bits: int = 4, block: int = 256, device="cuda", seed: int = 0):
        self.H, self.F, self.act, self.norm = hidden, ffn, act, L.make_norm(kind, eps)
        shapes = [("gamma", (hidden,)), ("beta", (hidden,)), ("b1", (ffn,)), ("b2", (hidden,)), ("w1", (ffn, hidden)),
                  ("w2", (hidden, ffn))]
        # every slice starts on a 16-byte boundary of the bf16 bucket, so that products fetch it whole
        self.slices, at = {}, 0
        for name, shape in shapes:
            size = int(torch.Size(shape).numel())
            self.slices[name] = (at, size, shape)
            at += -(-size // 8) * 8
        self.n = at
        dev = torch.device(device)
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        self.master = torch.zeros(self.n, device=dev)
        self.view(self.master, "gamma").fill_(1.0)
        self.view(self.master, "w1").normal_(0.0, hidden ** -0.5, generator=g)
        self.view(self.master, "w2").normal_(0.0, ffn ** -0.5, generator=g)
        self.param = self.master.to(torch.bfloat16)                        # what the passes read
        self.grad = torch.zeros(self.n, dtype=torch.bfloat16, device=dev)  # what the passes write
        self.m, self.v, self.err = (torch.zeros(self.n, device=dev) for _ in range(3))
        self.cfg = L.make_config(bits=bits, block=block, beta=0.9, err_scale_mult=4.0, reset_period=512)
        self.codes = torch.empty(L.loco_code_bytes(self.n, bits, block), dtype=torch.uint8, device=dev)
        self.scales = torch.empty(L.loco_num_blocks(self.n, block), device=dev)
        self.ws_linear = torch.empty(L.loco_linear_workspace_bytes(ffn), dtype=torch.uint8, device=dev)
        self.ws_norm = torch.empty(0, dtype=torch.uint8, device=dev)
        self.t = 0

    def view(self, bucket: torch.Tensor, name: str) -> torch.Tensor:
        """A parameter's slice of a flat bucket, in its shape."""
        at, size, shape = self.slices[name]
        return bucket[at:at + size].view(shape)

    def forward(self, x: torch.Tensor):
        """out [T, H] bf16 of x [T, H] bf16, and what the backward pass needs."""
        T, H, F, dev = x.shape[0], self.H, self.F, x.device
        p = lambda name: self.view(self.param, name)  # noqa: E731
        new = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        kept = {"rstd": new(T, dtype=torch.float32)}
        for name, cols in (("norm", H), ("pre", F)):
            nb = -(-cols // L.LOCO_CKPT_BLOCK)
            kept[name] = (new(T, nb * L.LOCO_CKPT_BLOCK, dtype=torch.int8), new(T, nb, dtype=torch.uint8))
        y, h, out = new(T, H), new(T, F), new(T, H)
        codes, scales = kept["norm"]
        L.loco_norm_forward(self.norm, x, p("gamma"), p("beta"), y, rstd=kept["rstd"], codes=codes, scales=scales)
        codes, scales = kept["pre"]
        L.loco_linear_forward(y, p("w1"), h, act=self.act, bias=p("b1"), codes=codes, scales=scales)
        L.loco_linear_forward(h, p("w2"), out, bias=p("b2"), residual=x)
        return out, kept

    def backward(self, dout: torch.Tensor, kept) -> torch.Tensor:
        """dx [T, H] for dout [T, H] bf16; every parameter's gradient goes to its slice of self.grad."""
        T, H, F, dev = dout.shape[0], self.H, self.F, dout.device
        p = lambda name: self.view(self.param, name)  # noqa: E731
        g = lambda name: self.view(self.grad, name)  # noqa: E731
        h, dz = (torch.empty(T, F, dtype=torch.bfloat16, device=dev) for _ in range(2))
        dy, dx = (torch.empty(T, H, dtype=torch.bfloat16, device=dev) for _ in range(2))
        need = L.loco_norm_workspace_bytes(T, H)
        if self.ws_norm.numel() < need:
            self.ws_norm = torch.empty(need, dtype=torch.uint8, device=dev)
        codes, scales = kept["pre"]
        L.loco_ckpt_decode(codes, scales, h, act=self.act)
        L.loco_linear_backward_weight(dout, g("w2"), x=h, db=g("b2"))
        L.loco_linear_backward_input(dout, p("w2"), dz, act=self.act, codes=codes, scales=scales)
        codes, scales = kept["norm"]
        L.loco_linear_backward_weight(dz, g("w1"), codes=codes, scales=scales, gamma=p("gamma"), beta=p("beta"),
                                      db=g("b1"), workspace=self.ws_linear)
        L.loco_linear_backward_input(dz, p("w1"), dy)
        L.loco_norm_backward(self.norm, dy, p("gamma"), kept["rstd"], dx, codes=codes, scales=scales, residual=dout,
                             dgamma=g("gamma"), dbeta=g("beta"), workspace=self.ws_norm)
        return dx

    def compress(self):
        """This rank's packed bucket of the gradients (codes, scales): what the ranks exchange."""
        self.t += 1
        L.loco_compress(self.cfg, self.grad, self.err, self.t, self.codes, self.scales)
        return self.codes, self.scales

    def step(self, codes, scales, hp):
        """One Adam(W) step on the average of the ranks' packed buckets (lists, one entry per rank)."""
        L.loco_adam_step_bf16(self.cfg, codes, scales, self.n, self.master, self.m, self.v,
                              self.param.view(torch.int16), hp, self.t)


def train(steps: int = 200, tokens: int = 512, hidden: int = 256, ffn: int = 688, lr: float = 2e-3, seed: int = 1):
    """Losses of a block that learns a fixed random block's outputs, one rank."""
    teacher, block = MlpBlock(hidden, ffn, seed=seed), MlpBlock(hidden, ffn, seed=seed + 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    hp, losses = L.make_adam(lr=lr, beta1=0.9, beta2=0.95), []
    for _ in range(steps):
        x = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
        want, _ = teacher.forward(x)
        out, kept = block.forward(x)
        off = out.float() - want.float()
        losses.append(off.square().mean())
        block.backward((off * (2.0 / off.numel())).to(torch.bfloat16), kept)
        codes, scales = block.compress()
        block.step([codes], [scales], hp)
    return [float(v) for v in losses]


if __name__ == "__main__":
    got = train()
    for i in range(0, len(got), 20):
        print(f"step {i:4d}  loss {got[i]:.5f}")
    print(f"step {len(got) - 1:4d}  loss {got[-1]:.5f}")
