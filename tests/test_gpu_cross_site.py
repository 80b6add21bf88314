"""A cross-attention site end to end: norm with the residual's addition,
query projection, attention over an encoder's states, out-projection.

Each step's own kernel is checked elsewhere; here the site's output is compared
with the same site in 32 bits throughout, without any quantization.  Three E4M3
roundings lie between the two (tokens, attention output, weights): each has a
relative error of at most 2^-4 a value, 2^-4 / sqrt(3) in the mean square, and
values of independent signs add in squares, so the output's relative error (2-norm) stays
below sqrt(6) 2^-4 / sqrt(3) < 0.1; the queries' and keys' errors also pass
through the softmax, whose scores here are of the order of one.
"""

import pytest
import torch

from gpu_util import W, dev_f32  # noqa: F401
from w8a16_linear_gb300.stack import CrossSite, CrossWeights

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def weights(hidden, enc, heads, kv_heads, D, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def mat(n, k):
        w = torch.randn((n, k), generator=g, device="cuda") * k ** -0.5
        s = w.abs().amax(1) / 448
        return w, ((w / s[:, None]).to(F8).view(torch.uint8), s)

    def norm(n):
        return (1 + 0.1 * torch.randn((n,), generator=g, device="cuda")).bfloat16()

    q, k, v = mat(heads * D, hidden), mat(kv_heads * D, enc), mat(kv_heads * D, enc)
    o = torch.randn((hidden, heads * D), generator=g, device="cuda") * (heads * D) ** -0.5
    s_o = o.abs().max() / 448
    w = CrossWeights(norm(hidden), norm(enc), q[1], k[1], v[1],
                     ((o / s_o).to(F8).view(torch.uint8), s_o.reshape(1)), dev_f32(2.0 / 448))
    return w, (q[0], k[0], v[0], o)


def plain(w, mats, x, residual, states, heads, kv_heads, D, keep):
    def rms(t, n):
        return t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * n.float()

    B, T, _ = states.shape
    q = (rms(x.float() + residual.float(), w.norm) @ mats[0].T).view(B, -1, heads, D)
    e = rms(states.float(), w.enc_norm)
    G = heads // kv_heads
    k, v = ((e @ m.T).view(B, T, kv_heads, D).repeat_interleave(G, 2) for m in mats[1:3])
    s = torch.einsum("blhd,bthd->bhlt", q, k) * D ** -0.5
    p = torch.softmax(s.masked_fill(~keep[:, None, None, :], float("-inf")), -1)
    return torch.einsum("bhlt,bthd->blhd", p, v).reshape(x.shape[0], -1) @ mats[3].T


@pytest.mark.parametrize("B,L,hidden,enc,heads,kv_heads,D,T", [(2, 1, 512, 384, 8, 2, 64, 77), (2, 150, 512, 384, 4, 4, 128, 300),
                                                               (1, 600, 1024, 512, 8, 8, 128, 96)])
def test_site_matches_its_unquantized_form(W, B, L, hidden, enc, heads, kv_heads, D, T):
    w, mats = weights(hidden, enc, heads, kv_heads, D, seed=L)
    g = torch.Generator(device="cuda").manual_seed(L + 1)
    x, r = (torch.randn((B * L, hidden), generator=g, device="cuda").bfloat16() for _ in range(2))
    states = torch.randn((B, T, enc), generator=g, device="cuda").bfloat16()
    lens = torch.randint(T // 2, T + 1, (B,), generator=g, device="cuda").to(torch.int32)
    site = CrossSite(B, L, hidden, heads, kv_heads, D, x.device)
    site.encode(W, w, states)
    y, res = site.run(W, w, x, r, kv_len=lens)
    torch.cuda.synchronize()
    W.poll_device_error()
    keep = torch.arange(T, device="cuda")[None] < lens[:, None]
    ref = plain(w, mats, x, r, states, heads, kv_heads, D, keep)
    assert float((y.float() - ref).norm() / ref.norm()) < 0.1
    assert torch.equal(res, (x.float() + r.float()).bfloat16())


def test_site_in_a_graph_repeats_its_bits(W):
    B, L, hidden, heads, kv_heads, D, T = 2, 3, 512, 8, 2, 64, 2000
    w, _ = weights(hidden, 384, heads, kv_heads, D)
    g = torch.Generator(device="cuda").manual_seed(9)
    x, r = (torch.randn((B * L, hidden), generator=g, device="cuda").bfloat16() for _ in range(2))
    site = CrossSite(B, L, hidden, heads, kv_heads, D, x.device)
    site.encode(W, w, torch.randn((B, T, 384), generator=g, device="cuda").bfloat16())
    want = [t.clone() for t in site.run(W, w, x, r)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        site.run(W, w, x, r)
    for _ in range(3):
        site.y.zero_()
        site.res.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(site.y.view(torch.int16), want[0].view(torch.int16))
        assert torch.equal(site.res.view(torch.int16), want[1].view(torch.int16))
    W.poll_device_error()
