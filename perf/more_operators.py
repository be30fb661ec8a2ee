"""Cases of a training step's other operators: joins of blocks, the loss on given tokens, AdamW on many tensors.

    join_forward      a block's output normalised (or as it is), gated, scaled and added to the scaled residual
                      stream, and the norm in front of the next block, in one call
    join_backward     the gradients of the stream, of the block's output, of both norms' parameters and of the gates
    logprob_forward   log probabilities of given tokens under logits, entropies, and the most likely alternatives
    logprob_backward  the gradient of the logits
    adam              one AdamW step on many tensors, states in 32 bits or in 8 (then their values read back)

8-bit states hold every 256 values of a tensor with one fp32 step: the first moment m = c * step, step = max |m| / 127,
and the root of the second sqrt(v) = c * step, step = max sqrt(v) / 255.  A code is rint(x + d), x = value * (127 / max)
or value * (255 / max), d = 0 or a dither from a hash of the seed, the step, the tensor and the element; the code of a
sqrt(v) that is not zero is at least 1.

`own = False` computes the plain form in 32 bits with elementary torch operations; `own = True` makes the library's
calls.  `exact` restates the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

F32, BF16 = "f32", "bf16"
DTYPES = {F32: torch.float32, BF16: torch.bfloat16}
BLOCK = 256
EPS = 1e-5
INF = float("inf")


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one token's hidden state at the 7B model's width between two blocks, while answering: a call's latency
        dict(name="join-token", op="join_forward", kind="rms", post=True, rows=1, cols=4096, x=BF16, y=BF16, gate=False,
             rowgate=False, a=1.0, s=1.0, pad=0),
        # a ragged batch on a strided fp32 stream at an odd width: layer norms, every gate and scale
        dict(name="join-ragged", op="join_forward", kind="layer", post=True, rows=777, cols=2049, x=F32, y=BF16, gate=True,
             rowgate=True, a=0.75, s=0.5, pad=3),
        # a training batch's tokens at the 7B model's width, a gate for each channel
        dict(name="join-train", op="join_forward", kind="rms", post=True, rows=16384, cols=4096, x=BF16, y=BF16, gate=True,
             rowgate=False, a=1.0, s=0.25, pad=0),
        # backward of a short batch at the 1.1B model's width, fp32 stream, no norm behind the block, weighted rows
        dict(name="joingrad-short", op="join_backward", kind="layer", post=False, rows=500, cols=2048, x=F32, y=BF16,
             gate=True, rowgate=True, a=1.0, s=0.5, grad=F32, pad=0),
        # backward of the training batch
        dict(name="joingrad-train", op="join_backward", kind="rms", post=True, rows=16384, cols=4096, x=BF16, y=BF16,
             gate=True, rowgate=False, a=1.0, s=0.25, grad=BF16, pad=0),
        # the token just chosen, with the alternatives a user is shown: one row of the 7B model's vocabulary
        dict(name="logprob-token", op="logprob_forward", rows=1, vocab=32000, x=BF16, scale=1.0, top=20, mask=False, pad=0),
        # scoring a training batch under a large vocabulary, few alternatives
        dict(name="logprob-train", op="logprob_forward", rows=4096, vocab=131072, x=BF16, scale=1.0, top=8, mask=False, pad=0),
        # gradient of a small batch with masked tokens, an odd vocabulary, a temperature, fp32 logits in wider rows
        dict(name="logprobgrad-ragged", op="logprob_backward", rows=333, vocab=32003, x=F32, scale=0.7, mask=True, pad=5),
        # gradient of a training batch at the 7B model's vocabulary
        dict(name="logprobgrad-train", op="logprob_backward", rows=8192, vocab=32000, x=BF16, scale=1.0, mask=False, pad=0),
        # the parameters of one small block, states in 8 bits with dithered rounding: a call's latency
        dict(name="adam-block", op="adam", tensors="mlp", hidden=256, ffn=688, bits=8, p=F32, g=BF16, copy=True, dither=7,
             t=3, gscale=True, shift=0),
        # the 1.1B model's 201 tensors, states in 32 bits, and the bf16 parameters that the next pass reads
        dict(name="adam-1.1b", op="adam", tensors="llama", hidden=2048, ffn=5632, layers=22, kv=256, vocab=32000, bits=32,
             p=F32, g=BF16, copy=True, dither=0, t=100, gscale=True, shift=0),
        # one layer's eight experts, states in 8 bits, dithered
        dict(name="adam-experts", op="adam", tensors="moe", hidden=4096, ffn=14336, experts=8, bits=8, p=F32, g=BF16, copy=True,
             dither=11, t=100, gscale=False, shift=0),
    ]


#: bounds of the drawn cases: the largest listed pass of each kind
MOST_ROWS, MOST_COLS, MOST_JOIN = 16384, 16384, 16384 * 4096
MOST_TOKENS, MOST_VOCAB, MOST_FORWARD, MOST_BACKWARD = 8192, 200000, 4096 * 131072, 8192 * 32000
MOST_PARAMS, MOST_TENSORS = 1_000_000_000, 300


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm; half of them rounded to a multiple of 8."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 8:
        v -= v % 8
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["join_forward", "join_backward", "logprob_forward", "logprob_backward", "adam"])
    pad = rng.choice([0, 0, 0, 1, 8, 40])
    if op.startswith("join"):
        rows, cols = _spread(rng, 1, MOST_ROWS), _spread(rng, 4, MOST_COLS)
        x, y = rng.choice([(BF16, BF16), (BF16, BF16), (F32, BF16), (F32, BF16), (F32, F32)])
        c = dict(op=op, kind=rng.choice(["layer", "rms"]), post=rng.random() < 0.6, rows=max(1, min(rows, MOST_JOIN // cols)),
                 cols=cols, x=x, y=y, gate=rng.random() < 0.5, rowgate=rng.random() < 0.3, a=rng.choice([1.0, 0.875]),
                 s=rng.choice([1.0, 0.22]), pad=pad)
        return c if op == "join_forward" else dict(c, grad=rng.choice([F32, BF16]))
    if op.startswith("logprob"):
        rows, vocab = _spread(rng, 1, MOST_TOKENS), _spread(rng, 8, MOST_VOCAB)
        rows = max(1, min(rows, (MOST_FORWARD if op == "logprob_forward" else MOST_BACKWARD) // vocab))
        c = dict(op=op, rows=rows, vocab=vocab, x=rng.choice([F32, BF16]), scale=rng.choice([1.0, 0.5, 1.3]),
                 mask=rng.random() < 0.4, pad=pad)
        return dict(c, top=rng.choice([0, 1, 5, 20, 32])) if op == "logprob_forward" else c
    bits, p = rng.choice([8, 32]), rng.choice([F32, F32, BF16])
    return dict(op=op, tensors="mixed", count=_spread(rng, 1, MOST_TENSORS), total=_spread(rng, 1000, MOST_PARAMS),
                mix=rng.randrange(1 << 30), bits=bits, p=p, g=rng.choice([BF16, F32]), copy=p == F32 and rng.random() < 0.5,
                dither=rng.choice([0, rng.randrange(1, 1 << 32)]), t=_spread(rng, 1, 10000), gscale=rng.random() < 0.5,
                shift=rng.choice([0, 0, 0, 1, 4]))


def _sizes(c):
    """Elements of each tensor of an optimizer case."""
    H, F = c.get("hidden"), c.get("ffn")
    if c["tensors"] == "mlp":
        return [H, H, F, H, F * H, H * F]
    if c["tensors"] == "llama":
        return [c["vocab"] * H, *([H * H, c["kv"] * H, c["kv"] * H, H * H, F * H, F * H, H * F, H, H] * c["layers"]), H,
                c["vocab"] * H]
    if c["tensors"] == "moe":
        return [F * H, H * F, F * H] * c["experts"]
    r = random.Random(c["mix"])
    w = [math.exp(r.uniform(0, 7)) for _ in range(c["count"])]
    return [max(1, int(c["total"] * v / sum(w))) for v in w]


def _size(d):
    return 2 if d == BF16 else 4


def work(case):
    """Bytes read and written once, and a few operations an element."""
    c, op = case, case["op"]
    if op.startswith("join"):
        R, C, sx, sy = c["rows"], c["cols"], _size(c["x"]), _size(c["y"])
        params = (2 if c["kind"] == "layer" else 1) * (2 if c["post"] else 1) + (1 if c["gate"] else 0)
        b = 16 * R + 2 * C * params + (4 * R if c["rowgate"] else 0)
        if op == "join_forward":
            return {"bytes": b + 2 * R * C * (sx + sy), "flops": 16 * R * C}
        y_read = c["post"] or c["gate"] or c["rowgate"]
        b += R * C * (3 * sx + (3 if y_read else 2) * sy) + _size(c["grad"]) * C * params + (4 * R if c["rowgate"] else 0)
        return {"bytes": b, "flops": 40 * R * C}
    if op.startswith("logprob"):
        R, V, s = c["rows"], c["vocab"], _size(c["x"])
        if op == "logprob_forward":
            return {"bytes": R * V * s + R * (20 + 12 * c["top"]), "flops": 5 * R * V}
        return {"bytes": 2 * R * V * s + 24 * R, "flops": 6 * R * V}
    n, p = sum(_sizes(c)), _size(c["p"])
    b = n * (2 * p + _size(c["g"]) + (2 if c["copy"] else 0))
    # 8-bit states are read back in bf16
    b += n * 16 if c["bits"] == 32 else n * (4 + 2 + 4) + (n // BLOCK) * (16 + 8)
    return {"bytes": b, "flops": 25 * n}


# ----------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, rows, cols, dtype, sigma=1.0, channels=0.0, pad=0, zero_row=False):
    """[rows, cols] of noise in a buffer of cols + pad columns; channels: spread of the columns' own sizes."""
    z = torch.randn(rows, cols + pad, generator=g, device="cuda") * sigma
    if channels:
        z *= torch.exp(channels * torch.randn(cols + pad, generator=g, device="cuda"))
    if zero_row and rows > 4:
        z[rows // 2] = 0.0  # a padding token
    return z.to(dtype)[:, :cols]


def _new(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _prepare_join(c, g):
    R, C, pad, dx, dy = c["rows"], c["cols"], c["pad"], DTYPES[c["x"]], DTYPES[c["y"]]
    layer = c["kind"] == "layer"
    vec = lambda mid, off: (mid + _normal(g, 1, C, torch.float32, off)[0]).to(torch.bfloat16)  # noqa: E731
    st = {"case": c, "ws": None}
    st["gamma"], st["beta"] = vec(1.0, 0.1), vec(0.0, 0.1) if layer else None
    st["pgamma"], st["pbeta"] = (vec(1.0, 0.1), vec(0.0, 0.1) if layer else None) if c["post"] else (None, None)
    st["gate"] = vec(0.5, 0.2) if c["gate"] else None
    st["rowgate"] = torch.rand(R, generator=g, device="cuda") if c["rowgate"] else None
    x = _normal(g, R, C, dx, 1.0, 0.5, pad, True)
    st["y"] = _normal(g, R, C, dy, 2.0, 0.3, pad, True)
    if c["op"] == "join_forward":
        st["x"] = x
        st["h"], st["u"], st["stats"] = _new(dx, R, C), _new(dy, R, C), _new(torch.float32, 4, R)
        return st
    # what the forward pass kept: the joined stream and the rows' statistics
    st["x"] = x
    st["h"], _, st["stats"] = _join_plain(st)
    del st["x"]
    st["dh"] = _normal(g, R, C, dx, 1e-3, 0.5, pad, True)
    st["du"] = _normal(g, R, C, dy, 1e-3, 0.5, pad, True)
    gd = DTYPES[c["grad"]]
    st["dx"], st["dy"] = _new(dx, R, C), _new(dy, R, C)
    for name in ("gamma", "beta", "pgamma", "pbeta", "gate"):
        st["d" + name] = _new(gd, C) if st[name] is not None else None
    st["drowgate"] = _new(torch.float32, R) if c["rowgate"] else None
    return st


def _prepare_logprob(c, g):
    R, V, dt = c["rows"], c["vocab"], DTYPES[c["x"]]
    st = {"case": c}
    z = torch.randn(R, V + c["pad"], generator=g, device="cuda") * 2.5
    y = torch.randint(0, V, (R,), generator=g, device="cuda")
    rows = torch.arange(R, device="cuda")
    z[rows, y] += 6.0 * torch.rand(R, generator=g, device="cuda")  # the given token is a likely one
    if R > 4:
        y[R // 2] = -1  # a padding token: none is given
    if c["mask"]:
        z.masked_fill_(torch.rand(V + c["pad"], generator=g, device="cuda") < 0.3, -INF)
        if R > 4:
            z[R // 3] = -INF  # nothing is left of this row
    st["logits"], st["targets"] = z.to(dt)[:, :V], y
    st["lse"], st["entropy"] = _new(torch.float32, R), _new(torch.float32, R)
    if c["op"] == "logprob_forward":
        st["logp"] = _new(torch.float32, R)
        st["ids"] = _new(torch.int64, R, c["top"]) if c["top"] else None
        st["alts"] = _new(torch.float32, R, c["top"]) if c["top"] else None
        return st
    # what the forward pass kept, and the gradients of its outputs
    st["lse"], st["entropy"] = _lse_plain(st["logits"].float() * c["scale"])[:2]
    st["dlogp"] = torch.rand(R, generator=g, device="cuda") * (-1.0 / R)
    st["dentropy"] = torch.randn(R, generator=g, device="cuda") * (0.01 / R)
    st["dlogits"] = _new(dt, R, V)
    return st


def _prepare_adam(c, g):
    """Flat buffers in which every tensor begins at a multiple of 256 elements, as slices of a gradient bucket do."""
    sizes = _sizes(c)
    blocks = [-(-n // BLOCK) for n in sizes]
    nb, shift = sum(blocks), c["shift"]
    st = {"case": c, "t": c["t"], "tensors": None}
    st["sizes"], st["first"] = sizes, [0]
    for b in blocks:
        st["first"].append(st["first"][-1] + b)
    ids = torch.repeat_interleave(torch.arange(len(sizes)), torch.tensor(blocks)).to("cuda")
    st["id"] = ids
    st["inside"] = torch.arange(nb, device="cuda") - torch.tensor(st["first"][:-1], device="cuda")[ids]   # block of its tensor
    left = torch.tensor(sizes, device="cuda")[ids] - st["inside"] * BLOCK                                 # elements from there on
    lane = torch.arange(BLOCK, device="cuda")
    ragged = (left < BLOCK).nonzero()[:, 0]
    keep = lane < left[ragged, None]

    def filled(values, dtype):
        """values [nb, 256], zeros past each tensor's end, in a buffer that begins `shift` elements in."""
        values[ragged] = values[ragged] * keep
        buf = _new(dtype, nb * BLOCK + shift)
        buf[shift:].copy_(values.view(-1))
        return buf[shift:]

    sigma = torch.pow(10.0, -5.0 + 3.0 * torch.rand(len(sizes), generator=g, device="cuda"))[ids][:, None]
    noise = lambda: torch.randn(nb, BLOCK, generator=g, device="cuda")  # noqa: E731
    st["grad"] = filled(noise().mul_(sigma), DTYPES[c["g"]])
    st["param"] = filled(noise().mul_(0.02), DTYPES[c["p"]])
    st["copy"] = filled(torch.zeros(nb, BLOCK, device="cuda"), torch.bfloat16) if c["copy"] else None
    if c["bits"] == 32:
        st["m"] = filled(noise().mul_(0.3 * sigma), torch.float32)
        st["v"] = filled(noise().square_().add_(0.1).mul_(sigma * sigma), torch.float32)
    else:
        m = torch.randint(-127, 128, (nb, BLOCK), generator=g, device="cuda", dtype=torch.int8)
        v = torch.randint(1, 256, (nb, BLOCK), generator=g, device="cuda", dtype=torch.uint8)
        m[ragged] = m[ragged] * keep
        v[ragged] = v[ragged] * keep
        st["m"], st["v"] = m.view(-1), v.view(-1)
        st["msteps"] = (sigma[:, 0] * (0.5 / 127)).contiguous()
        st["vsteps"] = (sigma[:, 0] * (1.5 / 255)).contiguous()
        st["mvalues"], st["vvalues"] = _new(torch.bfloat16, nb * BLOCK), _new(torch.bfloat16, nb * BLOCK)
    # vectors (every fifth tensor) learn faster and do not decay
    st["lr_scale"] = [2.0 if i % 5 == 4 else 1.0 for i in range(len(sizes))]
    st["decay_scale"] = [0.0 if i % 5 == 4 else 1.0 for i in range(len(sizes))]
    st["gscale"] = torch.full((1,), 0.37, device="cuda") if c["gscale"] else None  # of gradient clipping
    return st


def prepare(case, seed):
    g = _gen(seed)
    if case["op"].startswith("join"):
        return _prepare_join(case, g)
    if case["op"].startswith("logprob"):
        return _prepare_logprob(case, g)
    return _prepare_adam(case, g)


# ----------------------------------------------------------------------------- one pass

LR, BETA1, BETA2, ADAM_EPS, DECAY = 1e-4, 0.9, 0.95, 1e-8, 0.1


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from bit_gradient_compression_gb300 import loco as L
    c = st["case"]
    op = c["op"]
    if op.startswith("join"):
        cfg = L.make_join(L.LOCO_NORM_LAYER if c["kind"] == "layer" else L.LOCO_NORM_RMS, eps=EPS, post=c["post"],
                          residual_scale=c["a"], block_scale=c["s"])
        if op == "join_forward":
            L.loco_join_forward(cfg, st["x"], st["y"], st["h"], st["u"], gamma=st["gamma"], beta=st["beta"],
                                post_gamma=st["pgamma"], post_beta=st["pbeta"], gate=st["gate"], row_gate=st["rowgate"],
                                stats=st["stats"])
            return {"h": st["h"], "u": st["u"], "stats": st["stats"]}
        if st["ws"] is None:
            st["ws"] = torch.empty(L.loco_join_workspace_bytes(c["rows"], c["cols"]), dtype=torch.uint8, device="cuda")
        L.loco_join_backward(cfg, st["dh"], st["du"], st["h"], st["y"], st["stats"], st["dx"], st["dy"], gamma=st["gamma"],
                             post_gamma=st["pgamma"], post_beta=st["pbeta"], gate=st["gate"], row_gate=st["rowgate"],
                             dgamma=st["dgamma"], dbeta=st["dbeta"], dpost_gamma=st["dpgamma"], dpost_beta=st["dpbeta"],
                             dgate=st["dgate"], drow_gate=st["drowgate"], workspace=st["ws"])
        return _join_grads(st)
    if op == "logprob_forward":
        L.loco_logprob_forward(st["logits"], st["targets"], st["logp"], lse=st["lse"], entropy=st["entropy"],
                               top_ids=st["ids"], top_logp=st["alts"], scale=c["scale"])
        return _logprob_outputs(st)
    if op == "logprob_backward":
        L.loco_logprob_backward(st["logits"], st["targets"], st["lse"], st["dlogits"], dlogp=st["dlogp"],
                                entropy=st["entropy"], dentropy=st["dentropy"], scale=c["scale"])
        return {"dlogits": st["dlogits"]}
    if st["tensors"] is None:  # the list of tensors and its addresses, as a program keeps it from step to step
        at = [(BLOCK * f, BLOCK * f + n) for f, n in zip(st["first"], st["sizes"])]
        cut = lambda buf: None if buf is None else [buf[lo:hi] for lo, hi in at]  # noqa: E731
        whole = lambda buf: [buf[BLOCK * f:BLOCK * e] for f, e in zip(st["first"], st["first"][1:])]  # noqa: E731
        steps = lambda buf: [buf[f:e] for f, e in zip(st["first"], st["first"][1:])]  # noqa: E731
        eight = c["bits"] == 8
        st["tensors"] = L.make_adam_tensors(
            cut(st["param"]), cut(st["grad"]), whole(st["m"]) if eight else cut(st["m"]),
            whole(st["v"]) if eight else cut(st["v"]), m_steps=steps(st["msteps"]) if eight else None,
            v_steps=steps(st["vsteps"]) if eight else None, params_bf16=cut(st["copy"]), lr_scales=st["lr_scale"],
            decay_scales=st["decay_scale"], dither=c["dither"])
        st["hp"] = L.make_adam(lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, weight_decay=DECAY)
    L.loco_adam_tensors(st["tensors"], st["hp"], st["t"], grad_scale=st["gscale"])
    st["t"] += 1
    got = {"param": st["param"]}
    if c["copy"]:
        got["copy"] = st["copy"]
    if c["bits"] == 32:
        return {**got, "m": st["m"], "v": st["v"]}
    L.loco_adam_state_decode(st["m"], st["msteps"], st["mvalues"])
    L.loco_adam_state_decode(st["v"], st["vsteps"], st["vvalues"])
    return {**got, "m": st["mvalues"], "v": st["vvalues"]}


def _join_grads(st):
    names = ("dx", "dy", "dgamma", "dbeta", "dpgamma", "dpbeta", "dgate", "drowgate")
    return {n: st[n] for n in names if st[n] is not None}


def _logprob_outputs(st):
    got = {"logp": st["logp"], "lse": st["lse"], "entropy": st["entropy"]}
    return {**got, "ids": st["ids"], "alts": st["alts"]} if st["case"]["top"] else got


def _normed_plain(v, kind):
    """(normalised rows, mean, reciprocal root of the variance)."""
    m = v.mean(1) if kind == "layer" else torch.zeros(v.shape[0], device=v.device)
    d = v - m[:, None]
    r = 1.0 / torch.sqrt(d.square().mean(1) + EPS)
    return d * r[:, None], m, r


def _affine(v, gamma, beta):
    v = v if gamma is None else v * gamma.float()
    return v if beta is None else v + beta.float()


def _join_plain(st):
    c = st["case"]
    y = st["y"].float()
    if c["post"]:
        n, m1, r1 = _normed_plain(y, c["kind"])
        n = _affine(n, st["pgamma"], st["pbeta"])
    else:
        n, m1, r1 = y, torch.zeros(c["rows"], device="cuda"), torch.ones(c["rows"], device="cuda")
    if st["gate"] is not None:
        n = n * st["gate"].float()
    if st["rowgate"] is not None:
        n = n * st["rowgate"][:, None]
    h = (c["a"] * st["x"].float() + c["s"] * n).to(DTYPES[c["x"]])
    u, m2, r2 = _normed_plain(h.float(), c["kind"])
    u = _affine(u, st["gamma"], st["beta"]).to(DTYPES[c["y"]])
    return h, u, torch.stack([m1, r1, m2, r2])


def _lse_plain(z):
    """(log of the sum of exponentials, entropy, log probabilities) of each row; -inf, 0 and -inf where nothing is left."""
    top = z.amax(1)
    some = top > -INF
    d = z - torch.where(some, top, torch.zeros_like(top))[:, None]
    e = torch.exp(d)
    s = e.sum(1)
    lse = torch.where(some, top + torch.log(s), top)
    entropy = torch.log(s) - torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1) / s
    return lse, torch.where(some, entropy, torch.zeros_like(s)), torch.where(some[:, None], d - torch.log(s)[:, None], z)


def _ordered(z):
    """Whole numbers in the order of the values z (fp32), and among equal ones of their columns, the first highest."""
    b = torch.where(z == 0, torch.zeros_like(z), z).view(torch.int32).to(torch.int64)
    b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
    return (b << 32) | (0x7FFFFFFF - torch.arange(z.shape[1], device=z.device))


def _run_plain(st):
    c = st["case"]
    op = c["op"]
    if op == "join_forward":
        h, u, stats = _join_plain(st)
        return {"h": h, "u": u, "stats": stats}
    if op == "join_backward":
        return _join_backward_plain(st)
    if op.startswith("logprob"):
        return _logprob_plain(st)
    return _adam_plain(st)


def _join_backward_plain(st):
    c, gd = st["case"], DTYPES[st["case"]["grad"]]
    layer = c["kind"] == "layer"
    m1, r1, m2, r2 = (v[:, None] for v in st["stats"])
    du, hh = st["du"].float(), (st["h"].float() - m2) * r2
    got = {"dgamma": (du * hh).sum(0).to(gd)}
    if layer:
        got["dbeta"] = du.sum(0).to(gd)
    q = du * st["gamma"].float()
    t = q - hh * (q * hh).mean(1, keepdim=True)
    if layer:
        t = t - q.mean(1, keepdim=True)
    t = st["dh"].float() + t * r2
    got["dx"] = (c["a"] * t).to(DTYPES[c["x"]])
    e = c["s"] * t
    yh = (st["y"].float() - m1) * r1 if c["post"] else st["y"].float()
    n = _affine(yh, st["pgamma"], st["pbeta"])
    if c["rowgate"]:
        gn = n if st["gate"] is None else n * st["gate"].float()
        got["drowgate"] = (e * gn).sum(1)
        e = e * st["rowgate"][:, None]
    if c["gate"]:
        got["dgate"] = (e * n).sum(0).to(gd)
        e = e * st["gate"].float()
    if c["post"]:
        got["dpgamma"] = (e * yh).sum(0).to(gd)
        if layer:
            got["dpbeta"] = e.sum(0).to(gd)
        q = e * st["pgamma"].float()
        e = q - yh * (q * yh).mean(1, keepdim=True)
        if layer:
            e = e - q.mean(1, keepdim=True)
        e = e * r1
    got["dy"] = e.to(DTYPES[c["y"]])
    return got


def _logprob_plain(st):
    c, y = st["case"], st["targets"]
    z = st["logits"].float() * c["scale"]
    given = y >= 0
    if c["op"] == "logprob_forward":
        lse, entropy, logp = _lse_plain(z)
        at = logp.gather(1, y.clamp(min=0)[:, None])[:, 0]
        got = {"logp": torch.where(given, at, torch.zeros_like(at)), "lse": lse, "entropy": entropy}
        if c["top"]:
            k = min(c["top"], c["vocab"])
            key = _ordered(st["logits"].float()).topk(k, 1).values
            ids = 0x7FFFFFFF - (key & 0x7FFFFFFF)
            alts = logp.gather(1, ids)
            ids = torch.where(alts > -INF, ids, torch.full_like(ids, -1))
            more = (0, c["top"] - k)
            got["ids"] = torch.nn.functional.pad(ids, more, value=-1)
            got["alts"] = torch.nn.functional.pad(alts, more, value=-INF)
        return got
    some = st["lse"] > -INF
    logp = z - torch.where(some, st["lse"], torch.zeros_like(st["lse"]))[:, None]
    p = torch.where(some[:, None], torch.exp(logp), torch.zeros_like(z))
    d = torch.where(given & some, st["dlogp"], torch.zeros_like(st["dlogp"]))
    inner = torch.where(p > 0, logp + st["entropy"][:, None], torch.zeros_like(z))
    dz = -p * (d[:, None] + st["dentropy"][:, None] * inner)
    dz.scatter_add_(1, y.clamp(min=0)[:, None], d[:, None])
    return {"dlogits": (dz * c["scale"]).to(DTYPES[c["x"]])}


def _f32(v):
    return float(np.float32(v))


def _mix(x):
    """A hash of 32 bits (in 64-bit integers)."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random_bits(st):
    """32 random bits for each element of [nb, 256]."""
    key = _mix(_mix(torch.full_like(st["id"], st["case"]["dither"])) ^ (st["t"] & 0xFFFFFFFF))
    e = st["inside"] * BLOCK
    key = _mix(_mix(key ^ st["id"]) ^ (e >> 32))
    return _mix(((e & 0xFFFFFFFF)[:, None] + torch.arange(BLOCK, device="cuda")) ^ key[:, None])


def _adam_plain(st):
    c, t = st["case"], st["t"]
    rows = lambda v: v.view(-1, BLOCK)  # noqa: E731
    f32 = lambda v: torch.tensor([_f32(x) for x in v], device="cuda")[st["id"]][:, None]  # noqa: E731
    lr = [_f32(_f32(LR) * s) for s in st["lr_scale"]]
    decay = f32([_f32(a) * _f32(_f32(DECAY) * s) for a, s in zip(lr, st["decay_scale"])])
    b1, b2 = _f32(BETA1), _f32(BETA2)
    c1 = f32([a / (1.0 - b1 ** t) for a in lr])
    c2 = _f32(1.0 / math.sqrt(1.0 - b2 ** t))
    n1, n2 = _f32(np.float32(1) - np.float32(b1)), _f32(np.float32(1) - np.float32(b2))
    g = rows(st["grad"]).float()
    if st["gscale"] is not None:
        g = g * st["gscale"]
    p = rows(st["param"]).float()
    p = p - decay * p
    if c["bits"] == 32:
        m, v = rows(st["m"]), rows(st["v"])
    else:
        m = rows(st["m"]).float() * st["msteps"][:, None]
        v = (rows(st["v"]).float() * st["vsteps"][:, None]).square()
    m = b1 * m + n1 * g
    v = b2 * v + n2 * (g * g)
    root = torch.sqrt(v)
    p = p - c1 * (m / (root * c2 + _f32(ADAM_EPS)))
    bits = _random_bits(st) if c["dither"] else None
    st["t"] += 1
    if c["p"] == F32:
        st["param"].view(-1, BLOCK).copy_(p)
    elif bits is None:
        rows(st["param"]).copy_(p)  # rounded to nearest
    else:
        rows(st["param"]).copy_(((p.contiguous().view(torch.int32).to(torch.int64) + (bits >> 16)) & -65536).to(torch.int32)
                                .view(torch.float32))
    got = {"param": st["param"]}
    if c["copy"]:
        rows(st["copy"]).copy_(p)
        got["copy"] = st["copy"]
    if c["bits"] == 32:
        rows(st["m"]).copy_(m)
        rows(st["v"]).copy_(v)
        return {**got, "m": st["m"], "v": st["v"]}
    for value, codes, steps, most, low, out in ((m, "m", "msteps", 127.0, 0, "mvalues"), (root, "v", "vsteps", 255.0, 8, "vvalues")):
        top = value.abs().amax(1, keepdim=True)
        inv = torch.where(top > 0, most / top, torch.zeros_like(top))
        x = value * inv
        if bits is not None:
            x = x + (((bits >> low) & 255).float() - 127.5) * (1.0 / 256.0)
        q = torch.round(x)
        if codes == "v":
            q = torch.where(value > 0, q.clamp(min=1.0), q)
        step = top / most
        rows(st[codes]).copy_(q)
        st[steps].copy_(step[:, 0])
        q = q * step
        rows(st[out]).copy_(q if codes == "m" else q * q)
    return {**got, "m": st["mvalues"], "v": st["vvalues"]}


# ----------------------------------------------------------------------------- 64 bits

def _norm64(v, kind):
    if kind == "layer":
        var, mean = torch.var_mean(v, 1, correction=0)
    else:
        var, mean = (v * v).mean(1), torch.zeros_like(v[:, 0])
    rstd = (var + EPS) ** -0.5
    return (v - mean[:, None]) * rstd[:, None], mean, rstd


def _or64(t, other):
    return other if t is None else t.double()


def _join64(st):
    c = st["case"]
    y = st["y"].double()
    one = torch.ones(c["rows"], dtype=torch.float64, device="cuda")
    yh, m1, r1 = _norm64(y, c["kind"]) if c["post"] else (y, 0 * one, one)
    branch = torch.addcmul(torch.as_tensor(_or64(st["pbeta"], 0.0), device="cuda", dtype=torch.float64), yh,
                           torch.as_tensor(_or64(st["pgamma"], 1.0), device="cuda", dtype=torch.float64))
    weight = c["s"] * _or64(st["gate"], 1.0) * (_or64(st["rowgate"], one)[:, None])
    h = torch.addcmul(c["a"] * st["x"].double(), branch, weight.expand_as(branch))
    # the next norm is that of the stream as it is stored
    kept = h.to(DTYPES[c["x"]]).double()
    hh, m2, r2 = _norm64(kept, c["kind"])
    return {"h": h, "u": hh * _or64(st["gamma"], 1.0) + _or64(st["beta"], 0.0), "stats": torch.stack([m1, r1, m2, r2])}


def _joingrad64(st):
    c, C = st["case"], st["case"]["cols"]
    level = 1.0 if c["kind"] == "layer" else 0.0
    m1, r1, m2, r2 = st["stats"].double().unbind()

    def through(q, vh, r):
        """The gradient that a norm passes on: r (q - <q> - vh <q vh>)."""
        inner = torch.einsum("ij,ij->i", q, vh) / C
        return r[:, None] * (q - level * q.mean(1)[:, None] - vh * inner[:, None])

    du, hh = st["du"].double(), (st["h"].double() - m2[:, None]) * r2[:, None]
    total = st["dh"].double() + through(du * st["gamma"].double(), hh, r2)
    branch = c["s"] * total
    yh = (st["y"].double() - m1[:, None]) * r1[:, None] if c["post"] else st["y"].double()
    n = yh * _or64(st["pgamma"], 1.0) + _or64(st["pbeta"], 0.0)
    gate, w = _or64(st["gate"], 1.0), _or64(st["rowgate"], torch.ones_like(r1))[:, None]
    dn = branch * gate * w
    got = {"dx": c["a"] * total, "dy": through(dn * st["pgamma"].double(), yh, r1) if c["post"] else dn,
           "dgamma": torch.einsum("ij,ij->j", du, hh)}
    if c["kind"] == "layer":
        got["dbeta"] = du.sum(0)
    if c["post"]:
        got["dpgamma"] = torch.einsum("ij,ij->j", dn, yh)
        if c["kind"] == "layer":
            got["dpbeta"] = dn.sum(0)
    if c["gate"]:
        got["dgate"] = torch.einsum("ij,ij->j", branch * w, n)
    if c["rowgate"]:
        got["drowgate"] = (branch * gate * n).sum(1)
    return got


def _logprob64(st):
    c, y = st["case"], st["targets"]
    z = st["logits"].double() * c["scale"]
    given = y >= 0
    if c["op"] == "logprob_forward":
        lse = torch.logsumexp(z, 1)
        empty = lse == -INF
        logp = torch.where(empty[:, None], z, z - lse[:, None])
        entropy = torch.special.entr(torch.exp(logp)).sum(1)
        at = torch.take_along_dim(logp, y.clamp(min=0)[:, None], 1)[:, 0]
        got = {"logp": at.masked_fill(~given, 0.0), "lse": lse, "entropy": entropy}
        if c["top"]:
            k = min(c["top"], c["vocab"])
            got["ids"] = None
            got["alts"] = torch.full((c["rows"], c["top"]), -INF, dtype=torch.float64, device="cuda")
            got["alts"][:, :k] = torch.topk(logp, k, 1).values
        return got
    lse, entropy = torch.logsumexp(z, 1), st["entropy"].double()
    empty = st["lse"] == -INF
    p = torch.exp(z - st["lse"].double()[:, None]).masked_fill(empty[:, None], 0.0)
    d = st["dlogp"].double().masked_fill(~given | empty, 0.0)
    # p log p is 0 where p is
    plogp = -torch.special.entr(p)
    dz = -d[:, None] * p - st["dentropy"].double()[:, None] * (plogp + p * entropy[:, None])
    rows = torch.arange(c["rows"], device="cuda")
    dz[rows, y.clamp(min=0)] += d
    return {"dlogits": c["scale"] * dz}


def _adam64(st):
    c, t, i = st["case"], st["t"], st["id"]
    per = lambda v: torch.tensor(v, dtype=torch.float64, device="cuda")[i].unsqueeze(1)  # noqa: E731
    cut = lambda v: v.unflatten(0, (-1, BLOCK)).double()  # noqa: E731
    lr, wd = per([_f32(LR) * s for s in st["lr_scale"]]), per([_f32(DECAY) * s for s in st["decay_scale"]])
    b1, b2 = _f32(BETA1), _f32(BETA2)
    g = cut(st["grad"]) * (1.0 if st["gscale"] is None else st["gscale"].double())
    m, v = cut(st["m"]), cut(st["v"])
    if c["bits"] == 8:
        m, v = m * st["msteps"].double()[:, None], (v * st["vsteps"].double()[:, None]) ** 2
    m.mul_(b1).add_(g, alpha=1.0 - b1)
    v.mul_(b2).addcmul_(g, g, value=1.0 - b2)
    del g
    mhat, vhat = m / (1.0 - b1 ** t), v / (1.0 - b2 ** t)
    p = cut(st["param"]) * (1.0 - lr * wd) - lr * mhat / (vhat.sqrt() + ADAM_EPS)
    del mhat, vhat
    got = {"param": p.flatten()}
    if c["copy"]:
        got["copy"] = got["param"]
    if c["bits"] == 32:
        return {**got, "m": m.flatten(), "v": v.flatten()}
    bits = _random_bits(st) if c["dither"] else None

    def kept(x, most, low):
        step = x.abs().amax(1, keepdim=True) / most
        q = x / step.clamp(min=1e-300)
        if bits is not None:
            q += ((bits >> low).bitwise_and(255).double() - 127.5) / 256
        q = q.round_()
        if most == 255:
            q.clamp_(min=1.0).masked_fill_(x == 0, 0.0)
        return q * step

    return {**got, "m": kept(m, 127, 0).flatten(), "v": kept(v.sqrt_(), 255, 8).square_().flatten()}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "join_forward":
        return _join64(st)
    if case["op"] == "join_backward":
        return _joingrad64(st)
    return _adam64(st) if case["op"] == "adam" else _logprob64(st)
