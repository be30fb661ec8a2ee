"""Marshalling in C of the calls of joins, log probabilities and optimizer states: it gives up on what does not fit."""
import pytest

torch = pytest.importorskip("torch")

from bit_gradient_compression_gb300 import loco as L  # noqa: E402

marshal = pytest.importorskip("bit_gradient_compression_gb300._marshal", reason="built without Python's headers")
B, I = torch.bfloat16, torch.int64


def t(*shape, d=torch.float32):
    return torch.zeros(*shape, dtype=d)


def jf(**change):
    a = dict(kind=0, post=1, eps=1e-5, a=1.0, s=1.0, x=t(4, 64), y=t(4, 64, d=B), h=t(4, 64), u=t(4, 64, d=B), gamma=None,
             beta=None, post_gamma=None, post_beta=None, gate=None, row_gate=None, stats=None, stream=0)
    return marshal.join_forward(*{**a, **change}.values())


def jb(**change):
    a = dict(kind=0, post=1, eps=1e-5, a=1.0, s=1.0, dh=t(4, 64), du=t(4, 64, d=B), h=t(4, 64), y=t(4, 64, d=B), stats=t(4, 4),
             dx=t(4, 64), dy=t(4, 64, d=B), gamma=None, post_gamma=None, post_beta=None, gate=None, row_gate=None, dgamma=None,
             dbeta=None, dpost_gamma=None, dpost_beta=None, dgate=None, drow_gate=None, workspace=None, stream=0)
    return marshal.join_backward(*{**a, **change}.values())


def lf(**change):
    a = dict(logits=t(4, 64), targets=t(4, d=I), logp=t(4), lse=None, entropy=None, top_ids=None, top_logp=None, scale=1.0, stream=0)
    return marshal.logprob_forward(*{**a, **change}.values())


def lb(**change):
    a = dict(logits=t(4, 64), targets=t(4, d=I), lse=t(4), dlogits=t(4, 64), dlogp=t(4), entropy=None, dentropy=None, scale=1.0,
             stream=0)
    return marshal.logprob_backward(*{**a, **change}.values())


def sd(codes=t(256, d=torch.int8), steps=t(1), out=t(200), stream=0):
    return marshal.adam_state_decode(codes, steps, out, stream)


GIVES_UP = [
    (jf, dict(x=None)), (jf, dict(y=t(4, 63))), (jf, dict(h=t(4, 64, d=B))), (jf, dict(u=t(4, 64))), (jf, dict(u=t(5, 64, d=B))),
    (jf, dict(gamma=t(64), gate=t(64, d=B))), (jf, dict(beta=t(63))), (jf, dict(row_gate=t(4, d=B))), (jf, dict(row_gate=t(64))),
    (jf, dict(stats=t(3, 4))), (jf, dict(stats=t(4, 4, d=B))), (jf, dict(stats=t(4, 8)[:, ::2])), (jf, dict(eps="eps")),
    (jf, dict(x=t(64, 4).t())), (jf, dict(stream="s")),
    (jb, dict(dx=None)), (jb, dict(dy=None)), (jb, dict(dh=t(4, 64, d=B))), (jb, dict(h=t(4, 64, d=B))), (jb, dict(y=t(4, 64))),
    (jb, dict(dgamma=t(64), dgate=t(64, d=B))), (jb, dict(drow_gate=t(64))), (jb, dict(workspace=t(64))), (jb, dict(stats=t(4, 5))),
    (lf, dict(logits=None)), (lf, dict(targets=t(4))), (lf, dict(targets=t(5, d=I))), (lf, dict(logp=t(4, d=B))),
    (lf, dict(top_ids=t(4, 5, d=I), top_logp=t(4, 4))), (lf, dict(top_ids=t(4, 5))), (lf, dict(top_logp=t(4, 10)[:, ::2])),
    (lf, dict(top_logp=t(4, 33))), (lf, dict(logits=t(4, 64, d=torch.float64))), (lf, dict(scale="s")),
    (lb, dict(dlogits=t(4, 64, d=B))), (lb, dict(dlogits=None)), (lb, dict(lse=t(5))), (lb, dict(dentropy=t(4, d=B))),
    (sd, dict(codes=t(256))), (sd, dict(codes=t(255, d=torch.uint8))), (sd, dict(steps=t(2))), (sd, dict(out=t(2, 100))),
    (sd, dict(out=t(400)[::2])), (sd, dict(codes=None)),
]


@pytest.mark.parametrize("call,change", GIVES_UP)
def test_gives_up(call, change):
    L._dtypes()
    assert call(**change) is None


@pytest.mark.parametrize("call", [jf, jb, lf, lb, sd])
def test_calls(call):
    """What fits reaches the entry point, which refuses host memory."""
    L._dtypes()
    assert call() == L.LOCO_ERR_INVALID_ARG


@pytest.mark.parametrize("name,count", [("join_forward", 17), ("join_backward", 25), ("logprob_forward", 9),
                                        ("logprob_backward", 9), ("adam_state_decode", 4)])
def test_wrong_number_of_arguments(name, count):
    for n in (count - 1, count + 1):
        with pytest.raises(TypeError):
            getattr(marshal, name)(*[None] * n)
