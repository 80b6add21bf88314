"""A host thread whose first CUDA work is a call of the library: encoding a
tensor map needs a current context, which no earlier call has bound there."""

import threading

import pytest
import torch

from gpu_util import W  # noqa: F401

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def codes(*shape):
    return (torch.randn(shape, device="cuda") * 50).clamp(-448, 448).to(F8).view(torch.uint8)


def pertoken(W, M):
    x, w, st, sc = codes(M, 256), codes(512, 256), torch.rand((M,), device="cuda"), torch.rand((512,), device="cuda")
    return lambda out: W.fp8_linear_w8a8_pertoken(x, st, w, sc, out=out), (M, 512)


def w8a8(W):
    x, w, s = codes(300, 256), codes(512, 256), torch.full((1,), 0.01, device="cuda")
    return lambda out: W.fp8_linear_w8a8(x, w, s, s, out=out), (300, 512)


def w8a16(W):
    x = torch.randn((300, 256), device="cuda").bfloat16()
    w, s = codes(512, 256), torch.full((1,), 0.01, device="cuda")
    return lambda out: W.fp8_linear_w8a16(x, w, s, out=out), (300, 512)


def attention(W, Lq):
    q, k, v = (torch.randn((1, n, 4, 64), device="cuda").bfloat16() for n in (Lq, 300, 300))
    return lambda out: W.cross_attention(q, k, v, out=out), (1, Lq, 4, 64)


@pytest.mark.parametrize("make", [lambda W: pertoken(W, 3), lambda W: pertoken(W, 3000), w8a8, w8a16,
                                  lambda W: attention(W, 1), lambda W: attention(W, 400)],
                         ids=["pertoken-few", "pertoken-many", "w8a8", "w8a16", "attention-1", "attention-400"])
def test_first_call_of_a_thread(W, make):
    call, shape = make(W)
    want, got = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    call(want)
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            call(got)
        except Exception as e:   # shown by the assertion below
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    W.poll_device_error()
    assert not errors, errors
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
