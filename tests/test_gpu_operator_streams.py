"""The operators of a cross-attention site on a stream given to the call, while
the current stream allocates and writes: the serial calls' bits."""

import pytest
import torch

from gpu_util import W  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [False, True])
def test_cross_attention_without_a_workspace_on_its_own_stream(W, lens):
    """The keys are cut over the CTAs: partial results, their sums and the tile
    table stand in a workspace that the call allocates, which has the size of
    the tensors that the current stream goes on to make and fill."""
    g = torch.Generator(device="cuda").manual_seed(21)
    q, k, v = (torch.randn(s, generator=g, device="cuda").bfloat16()
               for s in ((4, 1, 16, 128), (4, 9000, 4, 128), (4, 9000, 4, 128)))
    kv_len = torch.tensor([9000, 4500, 1, 7777], dtype=torch.int32, device="cuda") if lens else None
    want = W.cross_attention(q, k, v, kv_len=kv_len)
    n = W.cross_attention_workspace(q, k, v).numel()
    assert n > 0
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(30):
        got = W.cross_attention(q, k, v, kv_len=kv_len, stream=st)
        others = [torch.full((n,), float(i), device="cuda") for i in range(4)]
        torch.cuda.synchronize()
        W.poll_device_error()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        assert all(bool((t == float(i)).all()) for i, t in enumerate(others))


def test_a_chain_on_a_stream_given_to_each_call(W):
    g = torch.Generator(device="cuda").manual_seed(22)
    x, r = (torch.randn((700, 1024), generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.ones((1024,), dtype=torch.bfloat16, device="cuda")
    m = (torch.randn((512, 1024), generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    c = torch.rand((512,), generator=g, device="cuda") * 1e-3

    def chain(stream):
        codes, s_tok, res = W.add_rms_norm_quant(x, r, w, stream=stream)
        return [codes, s_tok, res, W.fp8_linear_w8a8_pertoken(codes, s_tok, m.view(torch.uint8), c, stream=stream)]

    want = chain(None)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for _ in range(10):
        got = chain(st)
        others = [torch.full((700, 1024), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert all(bool((t == 9).all()) for t in others)


def test_w8a8_from_bf16_without_a_workspace_on_its_own_stream(W):
    """The codes of the activation stand in a workspace of the call's own."""
    g = torch.Generator(device="cuda").manual_seed(23)
    x = torch.randn((4000, 2048), generator=g, device="cuda").bfloat16()
    m = (torch.randn((1024, 2048), generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s = torch.full((1,), 0.01, device="cuda")
    out = torch.empty((4000, 1024), dtype=torch.bfloat16, device="cuda")
    want = W.fp8_linear_w8a8(x, m, s, s)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for i in range(20):
        W.fp8_linear_w8a8(x, m, s, s, out=out, stream=st)
        others = [torch.full((4000, 2048), i, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        assert all(bool((t == i).all()) for t in others)
