"""Joins, log probabilities and many-tensor optimizer steps without a GPU: struct layouts, sizes, and every refusal that
the host makes before it looks at device memory."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

import steps_ref as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD = 1  # LOCO_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def L():
    from bit_gradient_compression_gb300 import build
    build.build()
    from bit_gradient_compression_gb300 import loco
    return loco


def test_struct_layouts(L, tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    structs = {"loco_join_config": L.loco_join_config, "loco_adam_tensor": L.loco_adam_tensor,
               "loco_adam_tensors_config": L.loco_adam_tensors_config}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "loco.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'  printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'  printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    enums = ("LOCO_STATE_BLOCK", "LOCO_MAX_TOP", "LOCO_STATE_M", "LOCO_STATE_V")
    lines += [f'  printf("enum {e} %lld\\n", (long long){e});' for e in enums] + ["  return 0;", "}"]
    (tmp_path / "l.c").write_text("\n".join(lines) + "\n")
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o",
                           str(tmp_path / "l")])
    got = {tuple(line.split()[:2]): int(line.split()[2])
           for line in subprocess.check_output([str(tmp_path / "l")], text=True).splitlines()}
    for name, cls in structs.items():
        assert got[(name, "size")] == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert got[(name, f)] == getattr(cls, f).offset
    for e in enums:
        assert got[("enum", e)] == getattr(L, e)


def test_workspace(L):
    m = L.LOCO_MAX_DIM
    assert L.loco_join_workspace_bytes(0, 64) > 0 and L.loco_join_workspace_bytes(5, 0) == 0
    assert L.loco_join_workspace_bytes(-1, 5) == 0 and L.loco_join_workspace_bytes(m + 1, 5) == 0
    assert L.loco_join_workspace_bytes(10 ** 6, 64) == L.loco_join_workspace_bytes(10 ** 5, 64)
    assert L.loco_join_workspace_bytes(m, m) > 0


JOIN = ("kind", "post", "eps", "residual_scale", "block_scale", "x_dtype", "y_dtype", "param_dtype", "grad_dtype")
BASE = {
    "loco_join_forward": dict(x=0x100000, ldx=64, y=0x200000, ldy=64, rows=4, cols=64, post_gamma=0x300000,
                              post_beta=0x310000, gate=0x320000, row_gate=0x330000, gamma=0x340000, beta=0x350000,
                              h=0x400000, ldh=64, u=0x500000, ldu=64, stats=0x600000, stream=0),
    "loco_join_backward": dict(dh=0x100000, lddh=64, du=0x110000, lddu=64, h=0x120000, ldh=64, y=0x130000, ldy=64,
                               stats=0x140000, rows=4, cols=64, post_gamma=0x150000, post_beta=0x160000, gate=0x170000,
                               row_gate=0x180000, gamma=0x190000, dx=0x200000, lddx=64, dy=0x210000, lddy=64,
                               dpost_gamma=0x220000, dpost_beta=0x230000, dgate=0x240000, drow_gate=0x250000,
                               dgamma=0x260000, dbeta=0x270000, workspace=0x280000, ws_bytes=1 << 20, stream=0),
    "loco_logprob_forward": dict(logits=0x100000, dtype=1, ld=64, rows=4, vocab=64, scale=1.0, targets=0x200000,
                                 logp=0x210000, lse=0x220000, entropy=0x230000, top=5, top_ids=0x240000,
                                 top_logp=0x250000, stream=0),
    "loco_logprob_backward": dict(logits=0x100000, dtype=1, ld=64, rows=4, vocab=64, scale=1.0, targets=0x200000,
                                  lse=0x210000, entropy=0x220000, dlogp=0x230000, dentropy=0x240000, dlogits=0x300000,
                                  ldd=64, stream=0),
    "loco_adam_state_decode": dict(kind=0, codes=0x100000, steps=0x200000, n=1000, out=0x300000, out_dtype=0, stream=0),
}


def call(L, name, cfg=None, **change):
    a = {**BASE[name], **change}
    first = ()
    if "join" in name:
        values = dict(zip(JOIN, (0, 1, 1e-5, 1.0, 1.0, 0, 1, 1, 0)), **(cfg or {}))
        first = (ctypes.byref(L.loco_join_config(*values.values())),)
    return getattr(L.lib, name)(*first, *a.values()), L.lib.loco_last_error().decode()


REFUSED = [
    ("loco_join_forward", dict(), dict(kind=2), 2, "kind"),
    ("loco_join_forward", dict(), dict(post=2), 2, "post"),
    ("loco_join_forward", dict(), dict(eps=-1.0), 1, "eps"),
    ("loco_join_forward", dict(), dict(eps=math.nan), 1, "eps"),
    ("loco_join_forward", dict(), dict(residual_scale=math.inf), 1, "residual_scale"),
    ("loco_join_forward", dict(), dict(block_scale=math.nan), 1, "block_scale"),
    ("loco_join_forward", dict(), dict(x_dtype=2), 2, "x_dtype"),
    ("loco_join_forward", dict(), dict(param_dtype=-1), 2, "param_dtype"),
    ("loco_join_forward", dict(rows=-1), None, 1, "rows"),
    ("loco_join_forward", dict(cols=0), None, 1, "cols"),
    ("loco_join_forward", dict(cols=1 << 31), None, 1, "cols"),
    ("loco_join_forward", dict(ldx=63), None, 1, "x"),
    ("loco_join_forward", dict(ldu=63), None, 1, "u"),
    ("loco_join_forward", dict(x=0), None, 1, "x is NULL"),
    ("loco_join_forward", dict(y=0), None, 1, "y is NULL"),
    ("loco_join_forward", dict(h=0), None, 1, "h is NULL"),
    ("loco_join_forward", dict(x=0x100002), None, 3, "x"),
    ("loco_join_forward", dict(stats=0x600002), None, 3, "stats"),
    ("loco_join_backward", dict(), dict(grad_dtype=3), 2, "grad_dtype"),
    ("loco_join_backward", dict(workspace=0), None, 1, "workspace"),
    ("loco_join_backward", dict(ws_bytes=4095), None, 1, "workspace"),
    ("loco_join_backward", dict(workspace=0x280004), None, 3, "workspace"),
    ("loco_join_backward", dict(h=0), None, 1, "h is NULL"),
    ("loco_join_backward", dict(y=0), None, 1, "y is NULL"),
    ("loco_join_backward", dict(y=0), dict(post=0), 1, "y is NULL"),
    ("loco_join_backward", dict(stats=0), None, 1, "stats is NULL"),
    ("loco_join_backward", dict(dx=0), None, 1, "dx is NULL"),
    ("loco_join_backward", dict(dy=0), None, 1, "dy is NULL"),
    ("loco_join_backward", dict(lddy=60), None, 1, "dy"),
    ("loco_logprob_forward", dict(dtype=2), None, 2, "dtype"),
    ("loco_logprob_forward", dict(vocab=0), None, 1, "vocab"),
    ("loco_logprob_forward", dict(rows=-3), None, 1, "rows"),
    ("loco_logprob_forward", dict(scale=0.0), None, 1, "scale"),
    ("loco_logprob_forward", dict(scale=-1.0), None, 1, "scale"),
    ("loco_logprob_forward", dict(scale=math.inf), None, 1, "scale"),
    ("loco_logprob_forward", dict(scale=math.nan), None, 1, "scale"),
    ("loco_logprob_forward", dict(top=33), None, 1, "top"),
    ("loco_logprob_forward", dict(top=-1), None, 1, "top"),
    ("loco_logprob_forward", dict(ld=63), None, 1, "logits"),
    ("loco_logprob_forward", dict(logits=0), None, 1, "logits is NULL"),
    ("loco_logprob_forward", dict(targets=0), None, 1, "targets is NULL"),
    ("loco_logprob_forward", dict(targets=0x200004), None, 3, "targets"),
    ("loco_logprob_forward", dict(top_ids=0x240004), None, 3, "top_ids"),
    ("loco_logprob_backward", dict(lse=0), None, 1, "lse is NULL"),
    ("loco_logprob_backward", dict(entropy=0), None, 1, "entropy is NULL"),
    ("loco_logprob_backward", dict(targets=0), None, 1, "targets is NULL"),
    ("loco_logprob_backward", dict(dlogits=0), None, 1, "dlogits is NULL"),
    ("loco_logprob_backward", dict(ldd=10), None, 1, "dlogits"),
    ("loco_logprob_backward", dict(logits=0x100001), None, 3, "logits"),
    ("loco_adam_state_decode", dict(kind=2), None, 2, "kind"),
    ("loco_adam_state_decode", dict(out_dtype=2), None, 2, "out_dtype"),
    ("loco_adam_state_decode", dict(n=-1), None, 1, "n"),
    ("loco_adam_state_decode", dict(codes=0), None, 1, "codes is NULL"),
    ("loco_adam_state_decode", dict(codes=0x100008), None, 3, "codes"),
    ("loco_adam_state_decode", dict(out=0x300002), None, 3, "out"),
]


@pytest.mark.parametrize("name,change,cfg,status,text", REFUSED)
def test_refusals(L, name, change, cfg, status, text):
    got, said = call(L, name, cfg, **change)
    assert got == status and text in said, (got, said)


def test_no_config(L):
    a = list(BASE["loco_join_forward"].values())
    assert L.lib.loco_join_forward(None, *a) == BAD
    assert L.lib.loco_join_backward(None, *BASE["loco_join_backward"].values()) == BAD


@pytest.mark.parametrize("name", sorted(BASE))
def test_host_memory_is_refused(L, name):
    """Addresses that are no device memory are an argument error on a machine without a GPU too."""
    got, said = call(L, name)
    assert got == BAD and said


@pytest.mark.parametrize("name,empty", [("loco_join_forward", dict(rows=0)), ("loco_logprob_forward", dict(rows=0)),
                                        ("loco_logprob_backward", dict(rows=0)), ("loco_adam_state_decode", dict(n=0))])
def test_empty_calls(L, name, empty):
    assert call(L, name, **empty)[0] == 0


# ------------------------------------------------------------------ many tensors

def tensor(L, k=0, **change):
    base = 0x1000000 * (k + 1)
    v = dict(param=base, grad=base + 0x100000, m=base + 0x200000, v=base + 0x300000, m_steps=base + 0x400000,
             v_steps=base + 0x500000, param_bf16=base + 0x600000, n=1000, lr_scale=1.0, decay_scale=1.0)
    return L.loco_adam_tensor(*{**v, **change}.values())


def adam(L, tensors, hp=None, t=1, cfg=(8, 0, 1, 5), count=None, scale=0):
    array = (L.loco_adam_tensor * max(1, len(tensors)))(*tensors)
    got = L.lib.loco_adam_tensors(ctypes.byref(L.loco_adam_tensors_config(*cfg)), array, len(tensors) if count is None else count,
                                  ctypes.byref(hp or L.make_adam()), t, scale, 0)
    return got, L.lib.loco_last_error().decode()


@pytest.mark.parametrize("change,status,text", [
    (dict(param=0), 1, "tensors[1].param is NULL"), (dict(grad=0), 1, "tensors[1].grad is NULL"),
    (dict(m=0), 1, "tensors[1].m is NULL"), (dict(v_steps=0), 1, "tensors[1].v_steps is NULL"),
    (dict(param=0x2000002), 3, "tensors[1].param"), (dict(grad=0x2100001), 3, "tensors[1].grad"),
    (dict(m=0x2200008), 3, "tensors[1].m"), (dict(v_steps=0x2500002), 3, "tensors[1].v_steps"),
    (dict(param_bf16=0x2600001), 3, "tensors[1].param_bf16"), (dict(n=-1), 1, "tensors[1].n"),
    (dict(n=(1 << 48) + 1), 1, "tensors[1].n"), (dict(lr_scale=math.nan), 1, "tensors[1]"),
    (dict(decay_scale=math.inf), 1, "tensors[1]")])
def test_tensor_refusals(L, change, status, text):
    got, said = adam(L, [tensor(L), tensor(L, 1, **change)])
    assert got == status and text in said, (got, said)


@pytest.mark.parametrize("cfg,status", [((16, 0, 1, 0), 2), ((8, 2, 1, 0), 2), ((8, 0, 7, 0), 2)])
def test_config_refusals(L, cfg, status):
    assert adam(L, [tensor(L)], cfg=cfg)[0] == status


def test_step_refusals(L):
    assert adam(L, [tensor(L)], t=0)[0] == BAD
    assert adam(L, [tensor(L)], count=-1)[0] == BAD
    assert adam(L, [tensor(L)], cfg=(32, 1, 1, 0))[0] == BAD           # a bf16 copy of bf16 parameters
    for change in (dict(lr=math.inf), dict(eps=-1.0), dict(beta1=1.0), dict(beta2=-0.1), dict(weight_decay=math.nan)):
        assert adam(L, [tensor(L)], hp=L.make_adam(**change))[0] == BAD
    got, said = adam(L, [tensor(L)], scale=0x7000002)
    assert got == 3 and "grad_scale" in said
    got, said = adam(L, [tensor(L)])
    assert got == BAD and "tensors[0].param" in said                    # no device memory
    assert adam(L, [], count=0)[0] == 0
    assert adam(L, [tensor(L, n=0, param=0, m=0)])[0] == 0              # nothing to do, nothing looked at


def test_binding_refuses_what_does_not_fit(L):
    f, b = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.bfloat16)
    cfg = L.make_join()
    for call in (lambda: L.loco_join_forward(cfg, f, b, f[:, :32]), lambda: L.loco_join_forward(cfg, f, b, b),
                 lambda: L.loco_join_forward(cfg, f, b, f, f), lambda: L.loco_join_forward(cfg, f, b, f, b, gamma=torch.zeros(63)),
                 lambda: L.loco_join_forward(cfg, f, b, f, b, row_gate=torch.zeros(64)),
                 lambda: L.loco_join_forward(cfg, f, b, f, b, stats=torch.zeros(3, 4)),
                 lambda: L.loco_join_forward(cfg, f, b, f, b, gamma=torch.zeros(64), gate=torch.zeros(64).bfloat16()),
                 lambda: L.loco_join_forward(cfg, f.T, b.T, f.T),
                 lambda: L.loco_join_backward(cfg, f, b, b, b, None, f, b),
                 lambda: L.loco_join_backward(cfg, f, b, f, b, torch.zeros(4, 4), f, b, dgamma=torch.zeros(64), dgate=torch.zeros(64).bfloat16()),
                 lambda: L.loco_logprob_forward(f, torch.zeros(4), torch.zeros(4)),
                 lambda: L.loco_logprob_forward(f, torch.zeros(4, dtype=torch.int32), torch.zeros(4)),
                 lambda: L.loco_logprob_forward(f, None, None, top_ids=torch.zeros(4, 5, dtype=torch.int64), top_logp=torch.zeros(4, 4)),
                 lambda: L.loco_logprob_forward(f, None, None, top_ids=torch.zeros(4, 5)),
                 lambda: L.loco_logprob_forward(f.half(), None, None, lse=torch.zeros(4)),
                 lambda: L.loco_logprob_backward(f, None, torch.zeros(4), b),
                 lambda: L.loco_logprob_backward(f, None, torch.zeros(5), f),
                 lambda: L.loco_adam_state_decode(torch.zeros(256), torch.zeros(1), torch.zeros(7)),
                 lambda: L.loco_adam_state_decode(torch.zeros(255, dtype=torch.int8), torch.zeros(1), torch.zeros(7)),
                 lambda: L.loco_adam_state_decode(torch.zeros(256, dtype=torch.int8), torch.zeros(2), torch.zeros(7))):
        with pytest.raises(ValueError):
            call()
    p, n = [torch.zeros(10)], 10
    i8, u8, s = torch.zeros(256, dtype=torch.int8), torch.zeros(256, dtype=torch.uint8), torch.zeros(1)
    good = dict(params=p, grads=p, ms=[i8], vs=[u8], m_steps=[s], v_steps=[s])
    assert L.make_adam_tensors(**good).count == 1
    for change in (dict(grads=[]), dict(grads=[torch.zeros(n + 1)]), dict(ms=[u8]), dict(vs=[u8[:n]]), dict(m_steps=None),
                   dict(m_steps=[torch.zeros(2)]), dict(params_bf16=p), dict(lr_scales=[1.0, 2.0]), dict(dither=-1),
                   dict(dither=1 << 32), dict(params=[torch.zeros(10).half()]), dict(params=[torch.zeros(20)[::2]]),
                   dict(params=p + [torch.zeros(3).bfloat16()])):
        with pytest.raises(ValueError):
            L.make_adam_tensors(**{**good, **change})
    with pytest.raises(ValueError):
        L.loco_adam_tensors(L.make_adam_tensors(**good), L.make_adam(), 1, grad_scale=torch.zeros(2))


def test_pieces_stay_inside_the_matrix():
    """The join kernels copy rows that lie anywhere as the aligned 16-byte pieces they lie in.  Every piece that is copied
    whole lies inside the matrix, by the rule that the source states, for narrow matrices at every alignment."""
    import os
    import re
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_gradient_compression_gb300", "csrc",
                        "join_common.cuh")
    with open(path) as f:
        text = re.sub(r"\s+", " ", f.read())
    back, reach = map(int, re.search(r"kReachBack = (\d+), kReach = (\d+);", text).groups())
    assert "head = !ANY || ld >= kReachBack ? 1 : kReachBack, tail = !ANY || ld >= kReach ? 1 : kReach;" in text
    assert ("!((off != 0 && row < head && edges.first && c0 == 0) || "
            "(edges.last_row - row < tail && c0 + 8 + (off != 0 ? 16 / kElem : 0) > edges.rest));") in text
    for elem in (2, 4):
        whole = 8 * elem // 16
        for cols in [*range(1, 30), 250, 257]:
            for ld in (cols, cols + 1, cols + 7):
                for rows in (1, 2, 3, 9, 40):
                    for base in range(0, 16, elem):
                        end = base + ((rows - 1) * ld + cols) * elem
                        for row in range(rows):
                            start = base + row * ld * elem
                            off = start % 16
                            for c0 in range(0, cols + 8, 8):
                                head, tail = 1 if ld >= back else back, 1 if ld >= reach else reach
                                if (off and row < head and c0 == 0) or (
                                        rows - 1 - row < tail and c0 + 8 + (16 // elem if off else 0) > cols):
                                    continue  # element by element
                                pieces = [k for k in range(whole) if k == 0 or c0 < cols]
                                if off and c0 < cols:
                                    pieces.append(whole)  # a warp's last lane's
                                for k in pieces:
                                    at = start + c0 * elem - off + 16 * k
                                    assert base <= at and at + 16 <= end, (elem, cols, ld, rows, base, row, c0, k)


def test_every_wait_is_bounded():
    """Read in the source, as no test may make a wait run out on a device: the CTAs that share a row wait for one another
    only in `arrived`, which ends by the clock; what is read after a wait that ran out is NaN, and nothing is waited for."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_gradient_compression_gb300", "csrc")
    text = {}
    for name in ("join_common.cuh", "join_forward.cu", "join_backward.cu"):
        with open(os.path.join(csrc, name)) as f:
            text[name] = re.sub(r"//[^\n]*", "", f.read())
    common = text["join_common.cuh"]
    assert sum(t.count("try_wait") for t in text.values()) == 1
    assert "mbar_wait" not in "".join(text.values()) and "for (;;)" not in "".join(text.values())
    wait = common[common.index("bool arrived("):]
    wait = wait[:wait.index("float read(")]
    assert re.search(r"while \(global_ns\(\) - start < kWaitNs\)\s+if \(test\(\)\) return true;\s+return false;", wait)
    assert re.search(r"kWaitNs = (\d+);", common).group(1) == "2000000000"
    assert "if (!lost && !arrived(" in common and common.count("arrived(") == 2
    assert "if (lost) v = __uint_as_float(0x7FC00000u);" in common and "team.lost ? __uint_as_float(0x7FC00000u)" in common
    # no CTA leaves its cluster before the others are done with its memory
    for name in ("join_forward.cu", "join_backward.cu"):
        assert text[name].count("team.part();") == 1


def test_dither_bits_are_even_and_independent():
    """Each byte of the hash over neighbouring elements, tensors and steps.  A value between two codes is rounded up with
    the probability that its byte exceeds a threshold, so what counts is the distribution function: it may be off by half
    of what a byte resolves (1/512) and five standard errors (0.5 / sqrt(n) each at most).  (The bins themselves are not
    held to uniformity: multiplications by these two constants leave them 2 % uneven, 0.1 % in the distribution.)  The
    bytes of the two states, and those of neighbours, are uncorrelated within five standard errors."""
    n = 1 << 18
    for dither, t, i in ((1, 1, 0), (1, 2, 0), (2, 1, 0), (7, 1, 3)):
        r = S.random_bits(dither, t, i, n, "cpu")
        for byte in range(4):
            below = torch.bincount((r >> (8 * byte)) & 255, minlength=256).double().cumsum(0) / n
            off = (below - torch.arange(1, 257) / 256).abs().max()
            assert float(off) <= 1 / 512 + 5 * 0.5 / math.sqrt(n), (dither, t, i, byte)
        a, b = (r & 255).double(), ((r >> 8) & 255).double()
        for u, v in ((a, b), (a[1:], a[:-1]), (a[256:], a[:-256])):
            c = torch.corrcoef(torch.stack([u, v]))[0, 1]
            assert abs(float(c)) < 5 / math.sqrt(len(u))
