"""GPU parity of qk_norm_rope against the formula in 64 bits.

With u = 2^-24: the kernel adds 8 squares in a lane and at most five butterfly
levels, so the mean of squares is within 16 u relatively; its reciprocal root has
half of that and 2 ulps, the products with the weight and with it one rounding
each: |h^ - h| <= 16 u |h| < 2^-18 |h|.  The phase is exact to 2^-32 of a turn and
rounded to binary32 in half turns (at most 2^-24 of one half turn): pi 2^-24 +
2 pi 2^-32 < 2^-22 radians; sincospi adds an ulp, the amplitude one rounding: cosine
and sine are within amplitude * 2^-21.  A rotated value is then within
(|a| + |b|) amplitude (2^-18 + 2^-21 + 3 u) < (|a| + |b|) amplitude 2^-17 before its
one rounding.
"""

import pytest
import torch

from gpu_util import W  # noqa: F401
from paged_util import DT, exact_heads, near, spread

pytestmark = pytest.mark.gpu


def make(M, Hq, Hk, D, dtype="bf16", seed=0, std=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qk = (torch.randn((M, Hq + Hk, D), generator=g, device="cuda") * std).to(DT[dtype])
    wq, wk = ((1 + 0.2 * torch.randn((D,), generator=g, device="cuda")).to(DT[dtype]) for _ in range(2))
    pos = torch.randint(-3, 1 << 20, (M,), generator=g, device="cuda").to(torch.int32)
    return qk[:, :Hq], qk[:, Hq:], wq, wk, pos


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("M,Hq,Hk,D,rot", [(1, 32, 8, 128, 128), (1, 1, 1, 16, 16), (3, 5, 1, 64, 64), (333, 20, 4, 80, 32),
                                           (7, 3, 3, 72, 48), (130, 4, 2, 256, 256), (65, 9, 3, 136, 16), (5, 40, 8, 96, 96),
                                           (2500, 3, 1, 128, 128), (2, 1, 0, 40, 32)])
def test_shapes(W, M, Hq, Hk, D, rot, interleaved, dtype):
    q, k, wq, wk, pos = make(M, Hq, Hk, D, dtype, seed=M + D)
    f = W.rope_frequencies(rot)
    for norm in (True, False):
        qo, ko = W.qk_norm_rope(q, k if Hk else None, pos, W.rope_turns(f), q_weight=wq if norm else None,
                                k_weight=wk if norm and Hk else None, interleaved=interleaved, amplitude=1.125)
        torch.cuda.synchronize()
        for x, w, got in ((q, wq, qo), (k, wk, ko)):
            if got is None:
                continue
            y, e = exact_heads(x, w if norm else None, spread(pos, rot // 2), f.cuda(), interleaved=interleaved, amplitude=1.125)
            assert near(got, y, e)


@pytest.mark.parametrize("dim", [64, 128])
def test_norm_alone_and_one_sided(W, dim):
    q, k, wq, wk, pos = make(37, 4, 2, dim)
    qo, ko = W.qk_norm_rope(q, k, q_weight=wq, eps=1e-3)
    torch.cuda.synchronize()
    assert near(qo, *exact_heads(q, wq, None, None, eps=1e-3))
    assert torch.equal(ko, k)                                # neither norm nor rotation: a copy
    f = W.rope_frequencies(dim // 2)
    qo, ko = W.qk_norm_rope(q, k, pos, W.rope_turns(f), k_weight=wk)
    torch.cuda.synchronize()
    assert near(qo, *exact_heads(q, None, spread(pos, dim // 4), f.cuda()))
    assert near(ko, *exact_heads(k, wk, spread(pos, dim // 4), f.cuda()))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [(16, 24, 24), (5, 0, 59), (30, 34), (64,)])
def test_axes(W, axes, interleaved):
    M = 211
    q, k, wq, wk, _ = make(M, 6, 2, 128)
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.randint(0, 5000, (len(axes), M + 9), generator=g, device="cuda").to(torch.int32)[:, 4:4 + M]
    f = W.rope_frequencies(128, base=500.0)
    qo, ko = W.qk_norm_rope(q, k, pos, W.rope_turns(f), q_weight=wq, k_weight=wk, axes=axes, interleaved=interleaved)
    torch.cuda.synchronize()
    per = torch.cat([spread(p, n) for p, n in zip(pos, axes)], 1)
    assert near(qo, *exact_heads(q, wq, per, f.cuda(), interleaved=interleaved))
    assert near(ko, *exact_heads(k, wk, per, f.cuda(), interleaved=interleaved))


def test_far_positions_and_stretched_frequencies(W):
    M = 64
    q, k, *_ = make(M, 2, 2, 128)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6, 10 ** 9 + 7, 131071] * 8, dtype=torch.int32, device="cuda")
    for f in (W.rope_frequencies(128), W.rope_frequencies(128, 1e6, factor=8.0, trained=8192), torch.linspace(-9, 9, 64).double()):
        qo, _ = W.qk_norm_rope(q, k, pos, W.rope_turns(f))
        torch.cuda.synchronize()
        # 64 bits keep the angle to 2^31 * 9 * 2^-53 < 2^-18: as much again as the bound
        y, e = exact_heads(q, None, spread(pos, 64), f.cuda())
        assert near(qo, y, 2 * e)


def test_in_place_and_strided(W):
    M, D = 77, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.randn((M, 12 * D), generator=g, device="cuda").bfloat16()
    whole = qkv.clone()
    q, k = qkv[:, :8 * D].view(M, 8, D), qkv[:, 8 * D:10 * D].view(M, 2, D)
    pos = torch.arange(M, device="cuda", dtype=torch.int32)
    t = W.rope_turns(W.rope_frequencies(D))
    want = W.qk_norm_rope(q.clone(), k.clone(), pos, t)
    got = W.qk_norm_rope(q, k, pos, t, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[:, 10 * D:], whole[:, 10 * D:])   # the values beside them are left alone
    # heads further apart than their sizes, tokens fastest
    odd = torch.randn((5, M, 136), generator=g, device="cuda").half()[:, :, :128].transpose(0, 1)
    out = torch.zeros((5, M, 136), device="cuda").half()[:, :, :128].transpose(0, 1)
    W.qk_norm_rope(odd, None, pos, t, q_out=out)
    torch.cuda.synchronize()
    assert near(out, *exact_heads(odd, None, spread(pos, 64), W.rope_frequencies(D).cuda()))


def test_values_that_are_not_finite_stay_in_their_head(W):
    q, k, wq, wk, pos = make(9, 4, 2, 128)
    q = q.contiguous()
    t = W.rope_turns(W.rope_frequencies(64))
    want, _ = W.qk_norm_rope(q, k, pos, t, q_weight=wq)
    q[3, 2, 5], q[4, 1, 100] = float("nan"), float("inf")
    got, _ = W.qk_norm_rope(q, k, pos, t, q_weight=wq)
    plain, _ = W.qk_norm_rope(q, k, pos, t)
    torch.cuda.synchronize()
    same = torch.ones((9, 4), dtype=torch.bool, device="cuda")
    same[3, 2] = same[4, 1] = False
    assert torch.equal(got[same], want[same])
    assert torch.isnan(got[3, 2]).all()
    # without a norm an infinity beyond the rotated part stays one value
    assert torch.isinf(plain[4, 1, 100]) and torch.isfinite(plain[4, 1, :100]).all()
    # and a NaN in it spoils its pair
    assert torch.isnan(plain[3, 2]).nonzero().flatten().tolist() == [5, 37]


def test_rows_of_zeros_and_no_rows(W):
    t = W.rope_turns(W.rope_frequencies(64))
    q = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((64,), dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    qo, ko = W.qk_norm_rope(q, q, pos, t, q_weight=w, k_weight=w)
    torch.cuda.synchronize()
    assert not qo.any() and not ko.any()
    qo, _ = W.qk_norm_rope(q[:0], q[:0], pos[:0], t)
    assert qo.shape == (0, 2, 64)


def test_same_bits_in_a_graph_and_on_a_stream(W):
    q, k, wq, wk, pos = make(50, 8, 2, 128)
    t = W.rope_turns(W.rope_frequencies(128))
    want = [x.clone() for x in W.qk_norm_rope(q, k, pos, t, q_weight=wq, k_weight=wk)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = W.qk_norm_rope(q, k, pos, t, q_weight=wq, k_weight=wk, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W.qk_norm_rope(q, k, pos, t, q_weight=wq, k_weight=wk, q_out=got[0], k_out=got[1])
    got[0].zero_(), got[1].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
