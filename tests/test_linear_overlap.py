"""Outputs that share memory with an operand are refused, also where the call would read an aligned copy of it."""
import random
import types

import pytest
import torch

from bit_gradient_compression_gb300 import loco as L

B = torch.bfloat16
T, N, K = 333, 1407, 1031


def bytes_of(p, ld, rows, cols, elem):
    return {p + (i * ld + j) * elem + b for i in range(rows) for j in range(cols) for b in range(elem)}


def test_overlap_of_matrices():
    """Never missed; exact for rows of one pitch, for single rows, and for matrices that lie apart."""
    rng, seen = random.Random(5), [0, 0]
    for _ in range(4000):
        mats = []
        pitch = rng.randint(1, 12)
        for _ in range(2):
            elem, rows, cols = rng.choice([1, 2, 4]), rng.randint(1, 4), rng.randint(1, 6)
            ld = rng.choice([pitch * 4 // elem, cols + rng.randint(0, 5)])
            mats.append((0x1000 + rng.randint(0, 40), max(ld, cols), rows, cols, elem))
        a, b = mats
        true = bool(bytes_of(*a) & bytes_of(*b))
        got = L.loco_matrices_overlap(*a, *b)
        assert got == L.loco_matrices_overlap(*b, *a)
        assert got or not true, mats
        if not true:
            ranges = min(a[0] + ((a[2] - 1) * a[1] + a[3]) * a[4], b[0] + ((b[2] - 1) * b[1] + b[3]) * b[4]) > max(a[0], b[0])
            if not ranges or a[2] == 1 or b[2] == 1 or a[1] * a[4] == b[1] * b[4]:
                assert not got, mats
        seen[got] += 1
    assert min(seen) > 500
    assert not L.loco_matrices_overlap(0, 4, 4, 4, 2, 0x1000, 4, 4, 4, 2)         # a matrix that is not there
    assert not L.loco_matrices_overlap(0x1000, 4, 0, 4, 2, 0x1000, 4, 4, 4, 2)    # no rows


def rand(rows, cols, d=B):
    return torch.randn(rows, cols, device="cuda").to(d)


def at(t, start, rows, cols, dtype, ld=None):
    """A matrix of dtype that begins `start` elements into t's memory."""
    return t.view(-1).view(dtype).as_strided((rows, cols), (ld or cols, 1), start)


def cases():
    x, w, dy = rand(T, K), rand(N, K), rand(T, N)
    y, dw = rand(T, N), rand(N, K)
    nb = -(-N // 32)
    codes, scales = torch.zeros(T, nb * 32, dtype=torch.int8, device="cuda"), torch.zeros(T, nb, dtype=torch.uint8, device="cuda")
    big = torch.zeros(2 * N * K + 8, dtype=B, device="cuda")          # an operand with room behind it
    ws = at(big, 64, 1, 4 * N, torch.uint8)[0]
    nk = -(-K // 32)
    kcodes, kscales = torch.zeros(T, nk * 32, dtype=torch.int8, device="cuda"), torch.zeros(T, nk, dtype=torch.uint8, device="cuda")
    return {
        "y in x": (big, lambda s: L.loco_linear_forward(at(big, 1, T, K, B), w, at(big, K, T, N, B), stream=s)),
        "y in w": (big, lambda s: L.loco_linear_forward(x, at(big, 0, N, K, B), at(big, N * K - 1, T, N, B), stream=s)),
        "codes in x": (big, lambda s: L.loco_linear_forward(
            at(big, 0, T, K, B), w, y, codes=at(big, 0, T, nb * 32, torch.int8), scales=scales, stream=s)),
        "scales in w": (big, lambda s: L.loco_linear_forward(
            x, at(big, 0, N, K, B), y, codes=codes, scales=at(big, 2 * N * K - 1, T, nb, torch.uint8), stream=s)),
        "dx in dy": (big, lambda s: L.loco_linear_backward_input(at(big, 0, T, N, B), w, at(big, T * N - 1, T, K, B), stream=s)),
        "dx in w": (big, lambda s: L.loco_linear_backward_input(dy, at(big, 3, N, K, B), at(big, 0, T, K, B), stream=s)),
        "dw in dy": (big, lambda s: L.loco_linear_backward_weight(at(big, 0, T, N, B), at(big, 5, N, K, B), x=x, stream=s)),
        "db in x": (big, lambda s: L.loco_linear_backward_weight(dy, dw, x=at(big, 0, T, K, B), db=at(big, K, 1, N, B)[0], stream=s)),
        "workspace in dy": (big, lambda s: L.loco_linear_backward_weight(
            at(big, 0, T, N, B), dw, codes=kcodes, scales=kscales, beta=torch.ones(K, device="cuda"), workspace=ws, stream=s)),
    }


NAMES = ["y in x", "y in w", "codes in x", "scales in w", "dx in dy", "dx in w", "dw in dy", "db in x", "workspace in dy"]


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("path", ["c", "python", "stream"])
def test_refused(monkeypatch, name, path):
    assert T * N * K >= L.ALIGN_WORK and T >= L.ALIGN_ROWS
    made = cases()
    assert list(made) == NAMES
    memory, call = made[name]
    memory.normal_()
    before = memory.clone()
    torch.cuda.synchronize()
    if path == "python":
        L._dtypes()
        monkeypatch.setattr(L, "_marshal", types.SimpleNamespace(**{n: lambda *a: None for n in dir(L._marshal)
                                                                    if n.startswith("linear")}))
    with pytest.raises(L.LocoError) as e:
        call(torch.cuda.Stream() if path == "stream" else None)
    assert e.value.status == L.LOCO_ERR_INVALID_ARG and "overlaps" in str(e.value)
    torch.cuda.synchronize()
    assert torch.equal(memory.view(torch.int16), before.view(torch.int16))


@pytest.mark.gpu
def test_columns_of_one_buffer():
    """An operand and the output side by side in a wider matrix do not overlap, and the operand is copied as always."""
    wide = torch.zeros(T, K + N + 3, dtype=B, device="cuda")
    x, y, w = wide[:, 1:1 + K], wide[:, 2 + K:2 + K + N], rand(N, K)
    x.copy_(rand(T, K))
    kept, copies = x.clone(), []
    real = L._scratch
    L._scratch = lambda n: copies.append(n) or real(n)
    try:
        L.loco_linear_forward(x, w, y)
    finally:
        L._scratch = real
    want = torch.empty(T, N, dtype=B, device="cuda")
    L.loco_linear_forward(kept, w, want)
    assert copies and torch.equal(y, want) and torch.equal(x, kept)


def test_no_output():
    """An output that is not there is refused by the entry point, whichever way the call is marshalled."""
    x, w, dy = (torch.zeros(s, dtype=B) for s in ((T, K), (N, K), (T, N)))
    for call in (lambda: L.loco_linear_forward(x, w, None, stream=0), lambda: L.loco_linear_backward_input(dy, w, None, stream=0)):
        with pytest.raises(L.LocoError) as e:
            call()
        assert e.value.status == L.LOCO_ERR_INVALID_ARG
