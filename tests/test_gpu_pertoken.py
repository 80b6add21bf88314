"""GPU parity of the W8A8 linear with a scale for each token and channel.

The products of E4M3 values are exact in binary32; K of them summed on the
tensor cores are within 2 K 2^-24 sum|terms| of the exact sum, and the two
scales and the bf16 output round once each: |y^ - y| <= (2^-8 + 2^-22) |y| +
2 K 2^-24 s_tok s_ch sum|terms|.  Where all partial sums are integers below
2^24 and the scales powers of two, y^ is the rounded exact value, bit for bit.
"""

import pytest
import torch

from gpu_util import W  # noqa: F401

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def make(M, K, Ns, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qx = (torch.randn((M, K), generator=g, device="cuda") * 100).clamp(-448, 448).to(F8).view(torch.uint8)
    s_tok = torch.rand((M,), generator=g, device="cuda") * 0.02 + 1e-4
    ws, cs = [], []
    for N in Ns:
        ws.append((torch.randn((N, K), generator=g, device="cuda") * 100).clamp(-448, 448).to(F8).view(torch.uint8))
        cs.append(torch.rand((N,), generator=g, device="cuda") * 1e-3 + 1e-6)
    return qx, s_tok, ws, cs


def check(y, qx, s_tok, w, c):
    a, b = qx.view(F8).double(), w.view(F8).double()
    s = s_tok.double()[:, None] * c.double()[None, :]
    y64 = (a @ b.T) * s
    bound = (2.0 ** -8 + 2.0 ** -22) * y64.abs() + 2 * qx.shape[1] * 2.0 ** -24 * (a.abs() @ b.abs().T) * s
    assert ((y.double() - y64).abs() <= bound).all()


@pytest.mark.parametrize("M,K,Ns", [(1, 16, (16,)), (1, 4096, (4096,)), (1, 4096, (1024, 16, 528)), (2, 272, (144,)),
                                    (7, 1008, (256, 256)), (16, 16384, (512,)), (17, 2064, (1040,)), (33, 512, (400,)),
                                    (64, 4096, (1024, 1024)), (100, 1024, (4096, 1024, 1024)), (127, 528, (272,)),
                                    (128, 4096, (512,)), (129, 4096, (512, 80)), (300, 1040, (656,)), (1000, 768, (2064,)),
                                    (60, 528, (12288, 8208)), (300, 528, (6992,)), (1100, 784, (2064, 1040)),
                                    (32, 512, (16384, 8208))])
def test_against_64_bits(W, M, K, Ns):
    qx, s_tok, ws, cs = make(M, K, Ns, seed=M + K)
    ys = W.fp8_linear_w8a8_pertoken_group(qx, s_tok, ws, cs)
    torch.cuda.synchronize()
    W.poll_device_error()
    for y, w, c in zip(ys, ws, cs):
        check(y, qx, s_tok, w, c)
    one = W.fp8_linear_w8a8_pertoken(qx, s_tok, ws[0], cs[0])
    torch.cuda.synchronize()
    check(one, qx, s_tok, ws[0], cs[0])


@pytest.mark.parametrize("M,K,N", [(1, 1024, 272), (5, 4096, 512), (40, 2048, 528), (150, 1024, 512), (600, 640, 304),
                                   (100, 272, 20496), (1100, 640, 2320)])
def test_exact_sums(W, M, K, N):
    g = torch.Generator(device="cuda").manual_seed(K + M)
    a = torch.randint(-4, 5, (M, K), generator=g, device="cuda").float()
    b = torch.randint(-4, 5, (N, K), generator=g, device="cuda").float()
    s_tok = 2.0 ** torch.randint(-6, 3, (M,), generator=g, device="cuda").float()
    s_ch = 2.0 ** torch.randint(-6, 3, (N,), generator=g, device="cuda").float()
    y = W.fp8_linear_w8a8_pertoken(a.to(F8).view(torch.uint8), s_tok, b.to(F8).view(torch.uint8), s_ch)
    torch.cuda.synchronize()
    want = ((a.double() @ b.double().T) * s_tok.double()[:, None] * s_ch.double()).to(torch.bfloat16)
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))


def test_a_scale_belongs_to_its_token_and_channel(W):
    """NaN or infinite scales reach their own row and column only; the bytes
    behind the output stay as they were."""
    for M, N in ((3, 272), (200, 272), (1100, 2320), (70, 20496)):
        qx, s_tok, ws, cs = make(M, 512, (N,), seed=8)
        whole = torch.full((M + 1, N), -7.0, dtype=torch.bfloat16, device="cuda")
        s_tok[1] = float("nan")
        cs[0][5] = float("nan")
        y = W.fp8_linear_w8a8_pertoken(qx, s_tok, ws[0], cs[0], out=whole[:M])
        torch.cuda.synchronize()
        bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
        bad[1] = True
        bad[:, 5] = True
        assert torch.equal(torch.isnan(y), bad)
        assert (whole[M] == -7).all()


def test_group_equals_single_and_repeats(W):
    for M in (1, 20, 200):
        qx, s_tok, ws, cs = make(M, 1024, (256, 512), seed=M)
        a = W.fp8_linear_w8a8_pertoken_group(qx, s_tok, ws, cs)
        b = W.fp8_linear_w8a8_pertoken_group(qx, s_tok, ws, cs)
        torch.cuda.synchronize()
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_on_another_stream(W):
    qx, s_tok, ws, cs = make(9, 2048, (1024,), seed=9)
    want = W.fp8_linear_w8a8_pertoken(qx, s_tok, ws[0], cs[0])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = W.fp8_linear_w8a8_pertoken(qx, s_tok, ws[0], cs[0], out=torch.empty_like(want), stream=st)
    st.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(want.view(torch.int16), got.view(torch.int16))
