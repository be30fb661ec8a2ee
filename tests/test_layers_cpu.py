"""The layers' entry points without a GPU: sizes, struct layouts, and every refusal on the host."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    from bit_gradient_compression_gb300 import build
    build.build()
    from bit_gradient_compression_gb300 import loco
    return loco


def test_sizes(L):
    assert L.loco_ckpt_code_bytes(1, 1) == 32 and L.loco_ckpt_scale_bytes(1, 1) == 1
    assert L.loco_ckpt_code_bytes(3, 33) == 3 * 64 and L.loco_ckpt_scale_bytes(3, 33) == 6
    assert L.loco_ckpt_code_bytes(16384, 11008) == 16384 * 11008
    m = L.LOCO_MAX_DIM
    assert L.loco_ckpt_code_bytes(m, m) == m * ((m + 31) // 32) * 32        # no overflow at the limits
    for rows, cols in ((0, 5), (5, 0), (-1, 5), (m + 1, 5), (5, m + 1)):
        assert L.loco_ckpt_code_bytes(rows, cols) == 0 and L.loco_ckpt_scale_bytes(rows, cols) == 0
    assert L.loco_norm_workspace_bytes(0, 64) > 0 and L.loco_norm_workspace_bytes(5, 0) == 0
    assert L.loco_norm_workspace_bytes(10 ** 6, 64) == L.loco_norm_workspace_bytes(10 ** 5, 64)
    assert L.loco_linear_workspace_bytes(100) >= 400 and L.loco_linear_workspace_bytes(0) == 0


def test_struct_layouts(L, tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    structs = {"loco_norm_config": L.loco_norm_config, "loco_linear_config": L.loco_linear_config}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "loco.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'  printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'  printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    enums = ("LOCO_ACT_NONE", "LOCO_ACT_RELU", "LOCO_ACT_GELU", "LOCO_ACT_GELU_TANH", "LOCO_ACT_SILU",
             "LOCO_NORM_LAYER", "LOCO_NORM_RMS", "LOCO_CKPT_BLOCK", "LOCO_MAX_DIM")
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


BASE = {
    "loco_ckpt_encode": dict(x=0x10000, x_dtype=0, ldx=64, rows=4, cols=64, codes=0x20000, scales=0x30000),
    "loco_ckpt_decode": dict(codes=0x20000, scales=0x30000, rows=4, cols=64, act=0, gamma=0x40000, beta=0x50000,
                             param_dtype=0, out=0x60000, out_dtype=1, ldo=64),
    "loco_norm_forward": dict(cfg=(0, 1e-5, 0, 1, 0, 0), x=0x10000, ldx=64, rows=4, cols=64, gamma=0x20000,
                              beta=0x30000, y=0x40000, ldy=64, mean=0x50000, rstd=0x60000, codes=0x70000,
                              scales=0x80000),
    "loco_norm_backward": dict(cfg=(0, 1e-5, 0, 1, 0, 0), dy=0x10000, lddy=64, x=0x20000, ldx=64, codes=0, scales=0,
                               mean=0x30000, rstd=0x40000, rows=4, cols=64, gamma=0x50000, residual=0x60000, ldr=64,
                               dx=0x70000, lddx=64, dgamma=0x80000, dbeta=0x90000, workspace=0xA0000, ws_bytes=1 << 16),
    "loco_linear_forward": dict(cfg=(4, 1, 1), x=0x10000, ldx=64, w=0x20000, ldw=64, bias=0x30000, residual=0x40000,
                                ldr=32, T=4, N=32, K=64, y=0x50000, ldy=32, codes=0x60000, scales=0x70000),
    "loco_linear_backward_input": dict(cfg=(4, 1, 1), dy=0x10000, lddy=32, w=0x20000, ldw=64, codes=0x30000,
                                       scales=0x40000, residual=0x50000, ldr=64, T=4, N=32, K=64, dx=0x60000, lddx=64),
    "loco_linear_backward_weight": dict(cfg=(0, 1, 1), dy=0x10000, lddy=32, x=0, ldx=64, codes=0x30000, scales=0x40000,
                                        gamma=0x50000, beta=0x60000, T=4, N=32, K=64, dw=0x70000, lddw=64, db=0x80000,
                                        workspace=0x90000, ws_bytes=1 << 16),
}


def call(L, fn, **change):
    kw = {**BASE[fn], **change}
    args = list(kw.values())
    if "cfg" in kw:
        cls = L.loco_norm_config if "norm" in fn else L.loco_linear_config
        args[0] = ctypes.byref(cls(*kw["cfg"])) if kw["cfg"] is not None else None
    return getattr(L.lib, fn)(*args, 0)


NULLS = {
    "loco_ckpt_encode": ["x", "codes", "scales"],
    "loco_ckpt_decode": ["codes", "scales", "out"],
    "loco_norm_forward": ["cfg", "x", "y", "codes", "scales"],
    "loco_norm_backward": ["cfg", "dy", "mean", "rstd", "dx", "workspace"],
    "loco_linear_forward": ["cfg", "x", "w", "y", "codes", "scales"],
    "loco_linear_backward_input": ["cfg", "dy", "w", "codes", "scales", "dx"],
    "loco_linear_backward_weight": ["cfg", "dy", "codes", "scales", "dw", "workspace"],
}


@pytest.mark.parametrize("fn", BASE)
def test_null_arguments(L, fn):
    for name in NULLS[fn]:
        assert call(L, fn, **{name: None if name == "cfg" else 0}) == L.LOCO_ERR_INVALID_ARG, name
        assert L.lib.loco_last_error() != b""


@pytest.mark.parametrize("fn", BASE)
def test_sizes_and_pitches_out_of_range(L, fn):
    big = L.LOCO_MAX_DIM + 1
    for name in ("rows", "cols", "T", "N", "K"):
        if name in BASE[fn]:
            for v in (-1, big, -2 ** 63):
                assert call(L, fn, **{name: v}) == L.LOCO_ERR_INVALID_ARG, (name, v)
    for name in BASE[fn]:
        if name.startswith("ld") and not (fn.endswith("weight") and name == "ldx"):
            for v in (BASE[fn][name] - 1, 0, -8, big):
                assert call(L, fn, **{name: v}) == L.LOCO_ERR_INVALID_ARG, (name, v)
    if "cols" in BASE[fn] and "norm" in fn:
        assert call(L, fn, cols=0) == L.LOCO_ERR_INVALID_ARG


@pytest.mark.parametrize("fn", BASE)
def test_unknown_types_and_kinds(L, fn):
    kw = BASE[fn]
    for name in ("x_dtype", "param_dtype", "out_dtype"):
        if name in kw:
            assert call(L, fn, **{name: 2}) == L.LOCO_ERR_UNSUPPORTED
    if "act" in kw:
        for v in (-1, 5):
            assert call(L, fn, act=v) == L.LOCO_ERR_UNSUPPORTED
    if "cfg" in kw:
        for i, v in enumerate(kw["cfg"]):
            if isinstance(v, int) and not (fn.endswith("weight") and i == 0):
                bad = list(kw["cfg"])
                bad[i] = 7
                assert call(L, fn, cfg=tuple(bad)) == L.LOCO_ERR_UNSUPPORTED, i
    if "norm" in fn:
        for eps in (-1.0, float("nan"), float("inf")):
            assert call(L, fn, cfg=(0, eps, 0, 1, 0, 0)) == L.LOCO_ERR_INVALID_ARG


@pytest.mark.parametrize("fn", BASE)
def test_misaligned_pointers(L, fn):
    for name, v in BASE[fn].items():
        if not isinstance(v, int) or v < 0x10000 or name in ("scales", "ws_bytes"):
            continue
        assert call(L, fn, **{name: v + 1}) == L.LOCO_ERR_MISALIGNED, name
    for name in ("codes", "workspace"):
        if BASE[fn].get(name):
            assert call(L, fn, **{name: BASE[fn][name] + 8}) == L.LOCO_ERR_MISALIGNED, name


@pytest.mark.parametrize("fn", BASE)
def test_host_memory_is_refused(L, fn):
    if torch.cuda.is_available():
        pytest.skip("addresses that are nobody's device memory are only known so without a device")
    assert call(L, fn) == L.LOCO_ERR_INVALID_ARG


def test_short_workspace(L):
    need = L.loco_norm_workspace_bytes(4, 64)
    assert call(L, "loco_norm_backward", ws_bytes=need - 1) == L.LOCO_ERR_INVALID_ARG
    need = L.loco_linear_workspace_bytes(32)
    assert call(L, "loco_linear_backward_weight", ws_bytes=need - 1) == L.LOCO_ERR_INVALID_ARG


def test_half_a_checkpoint(L):
    for fn in ("loco_norm_forward", "loco_linear_forward"):
        for name in ("codes", "scales"):
            assert call(L, fn, **{name: 0}) == L.LOCO_ERR_INVALID_ARG


def test_empty_calls_succeed(L):
    assert call(L, "loco_ckpt_encode", rows=0, x=0, codes=0, scales=0) == L.LOCO_OK
    assert call(L, "loco_ckpt_decode", cols=0, out=0, codes=0, scales=0) == L.LOCO_OK
    assert call(L, "loco_norm_forward", rows=0, x=0, y=0) == L.LOCO_OK
    assert call(L, "loco_norm_backward", rows=0, dgamma=0, dbeta=0, workspace=0, ws_bytes=0) == L.LOCO_OK
    assert call(L, "loco_linear_forward", T=0, x=0, y=0) == L.LOCO_OK
    assert call(L, "loco_linear_backward_input", K=0, w=0, dx=0) == L.LOCO_OK
    assert call(L, "loco_linear_backward_weight", N=0, dy=0, dw=0, db=0) == L.LOCO_OK
    assert L.lib.loco_last_error() == b""


def test_binding_refusals(L):
    t = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d)
    b = torch.bfloat16
    codes, scales = t(4, 64, d=torch.int8), t(4, 2, d=torch.uint8)
    cfg = L.make_norm()
    with pytest.raises(ValueError, match="two-dimensional"):
        L.loco_ckpt_encode(t(64), codes, scales, stream=0)
    with pytest.raises(ValueError, match="row must be contiguous"):
        L.loco_ckpt_encode(t(64, 4).t(), codes, scales, stream=0)
    with pytest.raises(ValueError, match="codes must be"):
        L.loco_ckpt_encode(t(4, 65), codes, scales, stream=0)
    with pytest.raises(ValueError, match="not supported"):
        L.loco_ckpt_encode(t(4, 64, d=torch.float16), codes, scales, stream=0)
    with pytest.raises(ValueError, match="one dtype"):
        L.loco_ckpt_decode(codes, scales, t(4, 64), gamma=t(64), beta=t(64, d=b), stream=0)
    with pytest.raises(ValueError, match="vector of 64"):
        L.loco_norm_forward(cfg, t(4, 64), t(63), None, t(4, 64), stream=0)
    with pytest.raises(ValueError, match="y must be"):
        L.loco_norm_forward(cfg, t(4, 64), None, None, t(4, 65), stream=0)
    with pytest.raises(ValueError, match="one dtype"):
        L.loco_norm_backward(cfg, t(4, 64), None, t(4), t(4, 64), x=t(4, 64, d=b), stream=0)
    with pytest.raises(ValueError, match="rstd must be"):
        L.loco_norm_backward(cfg, t(4, 64), None, t(4, d=b), t(4, 64), x=t(4, 64), stream=0)
    with pytest.raises(ValueError, match="bfloat16"):
        L.loco_linear_forward(t(4, 64), t(32, 64, d=b), t(4, 32), stream=0)
    with pytest.raises(ValueError, match="w must be"):
        L.loco_linear_forward(t(4, 64, d=b), t(32, 63, d=b), t(4, 32), stream=0)
    with pytest.raises(ValueError, match="residual must be"):
        L.loco_linear_backward_input(t(4, 32, d=b), t(32, 64, d=b), t(4, 64), residual=t(4, 63), stream=0)
    with pytest.raises(ValueError, match="one dtype"):
        L.loco_linear_backward_weight(t(4, 32, d=b), t(32, 64), x=t(4, 64, d=b), db=t(32, d=b), stream=0)
    with pytest.raises(L.LocoError) as e:                      # a broadcast row: its pitch is 0
        L.loco_ckpt_encode(t(1, 64).expand(4, 64), codes, scales, stream=0)
    assert e.value.status == L.LOCO_ERR_INVALID_ARG
