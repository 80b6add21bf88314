"""GPU parity of add_rms_norm_quant against the formula in 64 bits.

With u = 2^-24 and r^ = fl32(x + res): |r^ - r| <= u |r|.  The kernel adds at
most 32 squares in a thread, five butterfly levels and 16 warp sums, so the
mean of squares is within 60 u of the exact one relatively; the reciprocal
root halves that and adds 2 ulps (4 u), the products with w and with it one
rounding each: |h^ - h| <= 40 u |h|.  A token's scale has the root's error and
two roundings, the codes' argument three more.  All stay below 2^-18, which is
what the tests take: a code (or a 16-bit h) has to lie between the roundings of
the exact value times 1 - 2^-18 and 1 + 2^-18.  r's own 16-bit rounding is
taken from the one binary32 sum, so it is compared bit for bit.
"""

import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import W, dev_f32  # noqa: F401

pytestmark = pytest.mark.gpu

REL = 2.0 ** -18
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def make(M, K, dtype, residual=True, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((M, K), generator=g) * std).to(DT[dtype]).cuda()
    r = (torch.randn((M, K), generator=g) * 2 * std).to(DT[dtype]).cuda() if residual else None
    w = (1 + 0.2 * torch.randn((K,), generator=g)).to(DT[dtype]).cuda()
    return x, r, w


def exact_h(x, r, w, eps):
    t = x.double() + (r.double() if r is not None else 0)
    return t / ((t * t).mean(-1, keepdim=True) + eps).sqrt() * w.double()


def between(got, lo, hi):
    return ((lo <= got) & (got <= hi)) | (torch.isnan(lo) & torch.isnan(got))


def window16(v, dt):
    a, b = (v * (1 - REL)).to(dt).double(), (v * (1 + REL)).to(dt).double()
    return torch.minimum(a, b), torch.maximum(a, b)


def codes_ok(q, y):
    """q: codes; y: exact arguments (64 bits)."""
    val = torch.from_numpy(O.e4m3_decode(q.cpu().numpy()).astype(np.float64))
    ends = [torch.from_numpy(O.e4m3_decode(O.e4m3_encode((y * (1 + s * REL)).cpu().numpy().astype(np.float32))).astype(np.float64))
            for s in (-1, 1)]
    return between(val, torch.minimum(*ends), torch.maximum(*ends)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K", [(1, 8), (1, 4096), (3, 264), (5, 1000), (7, 2312), (130, 64), (700, 2048), (701, 4104),
                                 (2, 16384), (620, 8200), (1300, 136)])
@pytest.mark.parametrize("static", [False, True])
def test_codes_scales_and_sum(W, M, K, dtype, static):
    x, r, w = make(M, K, dtype, seed=M + K)
    s_in = dev_f32(5.0 / 448) if static else None
    h = torch.empty_like(x)
    q, s_tok, res = W.add_rms_norm_quant(x, r, w, eps=1e-5, s_in=s_in, h_out=h)
    torch.cuda.synchronize()
    h64 = exact_h(x, r, w, 1e-5)
    assert torch.equal(res.view(torch.int16), (x.float() + r.float()).to(x.dtype).view(torch.int16))
    assert between(h.double(), *window16(h64, x.dtype)).all()
    if static:
        assert s_tok is None
        assert codes_ok(q, h64 / s_in.double())
    else:
        s64 = (h64.abs().amax(1) / 448).clamp_min(2.0 ** -126)
        assert ((s_tok.double() - s64).abs() <= REL * s64).all()
        assert codes_ok(q, h64 / s64[:, None])
        # the largest value of a row has the largest code
        assert (q.view(torch.float8_e4m3fn).float().abs().amax(1) == 448).all()


def test_without_residual_and_norm_alone(W):
    from w8a16_linear_gb300 import binding as b
    x, _, w = make(9, 1032, "bf16", residual=False)
    q, s_tok, res = W.add_rms_norm_quant(x, None, w)
    h = torch.empty_like(x)
    # the C entry with h alone
    assert b.lib().add_rms_norm_quant(x.data_ptr(), None, 0, 9, 1032, w.data_ptr(), 1e-6, None, None, None, h.data_ptr(),
                                      None, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    h64 = exact_h(x, None, w, 1e-6)
    assert res is None
    assert codes_ok(q, h64 / (h64.abs().amax(1) / 448)[:, None])
    assert between(h.double(), *window16(h64, x.dtype)).all()


def test_sum_in_place_of_the_residual(W):
    x, r, w = make(1500, 4096, "bf16", seed=3)
    want = W.add_rms_norm_quant(x, r.clone(), w)
    got = W.add_rms_norm_quant(x, r, w, res_out=r)
    torch.cuda.synchronize()
    assert got[2] is r
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_special_rows(W):
    x, r, w = make(8, 512, "bf16", seed=4)
    x[0] = 0
    r[0] = 0                        # a zero row: zero codes, the least scale
    x[1, 5] = float("nan")          # a NaN spoils its own row only
    x[2] = -r[2]                    # x + res cancels exactly
    x[3, :] = 0
    r[3, :] = 0
    r[3, 7] = 3.0                   # one value
    q, s, res = W.add_rms_norm_quant(x, r, w)
    torch.cuda.synchronize()
    v = q.view(torch.float8_e4m3fn).float()
    for i in (0, 2):
        assert (v[i] == 0).all() and float(s[i]) == 2.0 ** -126 and (res[i] == 0).all()
    assert torch.isnan(s[1]) and torch.isnan(v[1]).all()
    assert float(v[3, 7]) == 448 * torch.sign(w[7]) and int((v[3] != 0).sum()) == 1
    good = [4, 5, 6, 7]
    h64 = exact_h(x, r, w, 1e-6)[good]
    assert codes_ok(q[good], h64 / (h64.abs().amax(1) / 448)[:, None])


def test_static_scale_saturates(W):
    x, r, w = make(4, 256, "f16", seed=5)
    q, _, _ = W.add_rms_norm_quant(x, r, w, s_in=dev_f32(1e-4))
    torch.cuda.synchronize()
    h64 = exact_h(x, r, w, 1e-6)
    assert codes_ok(q, h64 / 1e-4)
    assert int((q & 0x7F == 0x7E).sum()) > 900      # 448, of 1024


def test_other_stream_and_repeat(W):
    x, r, w = make(333, 4096, "bf16", seed=6)
    want = W.add_rms_norm_quant(x, r, w)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = W.add_rms_norm_quant(x, r, w)
    st.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
