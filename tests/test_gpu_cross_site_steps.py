"""Each step of a cross-attention site against the formula in 64 bits of the
codes, scales and 16-bit values that the step before has left: every weight,
scale and buffer has to be the right one, to the steps' own tolerances (each
derived in the test of its operator)."""

import pytest
import torch

import test_gpu_attention as attention
import test_gpu_pertoken as linear
import test_gpu_rms_norm as norm
from gpu_util import W  # noqa: F401
from test_gpu_cross_site import weights
from w8a16_linear_gb300.stack import CrossSite

pytestmark = pytest.mark.gpu


def check_norm(codes, s_tok, x, r, w):
    h = norm.exact_h(x, r, w, 1e-6)
    s = (h.abs().amax(1) / 448).clamp_min(2.0 ** -126)
    assert ((s_tok.double() - s).abs() <= norm.REL * s).all()
    assert norm.codes_ok(codes, h / s[:, None])


@pytest.mark.parametrize("B,L,hidden,enc,heads,kv_heads,D,T", [(2, 1, 512, 384, 8, 2, 64, 77), (2, 1, 512, 384, 8, 2, 128, 9000),
                                                               (2, 150, 512, 384, 4, 4, 128, 300), (1, 600, 1024, 512, 6, 2, 96, 200)])
def test_each_step(W, B, L, hidden, enc, heads, kv_heads, D, T):
    w, _ = weights(hidden, enc, heads, kv_heads, D, seed=L)
    g = torch.Generator(device="cuda").manual_seed(L + 2)
    x, r = (torch.randn((B * L, hidden), generator=g, device="cuda").bfloat16() for _ in range(2))
    states = torch.randn((B, T, enc), generator=g, device="cuda").bfloat16()
    lens = torch.randint(T // 2, T + 1, (B,), generator=g, device="cuda").to(torch.int32)
    site = CrossSite(B, L, hidden, heads, kv_heads, D, x.device)
    site.encode(W, w, states)
    y, res = site.run(W, w, x, r, kv_len=lens)
    codes, s_tok, _ = W.add_rms_norm_quant(states.view(B * T, enc), None, w.enc_norm)
    torch.cuda.synchronize()
    W.poll_device_error()
    check_norm(codes, s_tok, states.view(B * T, enc), None, w.enc_norm)
    for got, m in ((site.k, w.k), (site.v, w.v)):
        linear.check(got.reshape(B * T, -1), codes, s_tok, *m)
    check_norm(site.codes, site.s_tok, x, r, w.norm)
    assert torch.equal(res, (x.float() + r.float()).bfloat16())
    linear.check(site.q, site.codes, site.s_tok, *w.q)
    ref, err = attention.exact(site.q.view(B, L, heads, D), site.k, site.v, attention.keep_of(B, T, lens))
    attention.check(site.attn, ref, err, w.s_attn)
    # the out-projection has one scale for all tokens and one for all channels
    linear.check(y, site.attn.view(B * L, -1), w.s_attn.expand(B * L), w.out[0], w.out[1].expand(hidden))
