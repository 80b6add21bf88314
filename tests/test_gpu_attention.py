"""GPU parity of cross_attention against the formula in 64 bits.

Let P_j be the weights (sum 1) and A = sum_j P_j |v_j| per output value.  The
kernel's score is within 2 D 2^-24 scale sum|q k| of the exact one, plus two
roundings of its own size in the exponent; the exponential adds 2^-22; P is
rounded to the 16-bit type (half an ulp: h = 2^-8 for bf16, 2^-11 for f16); the
accumulator adds 2 Lk 2^-24.  Twice the score's error enters, once by the
numerator and once by the sum:
    |o^ - o| <= A E + h (|o| + A E),
    E = h + 2 (2 D 2^-24 scale max sum|q k| + 2^-22 max|s log2 e| + 2^-22) + 4 (Lk + 64) 2^-24
and for f16, whose P is subnormal below 2^-14, another Lk 2^-25 max|v|.
Codes have to lie between those of the ends of that interval.
"""

import math

import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import W, dev_f32  # noqa: F401

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def make(B, Lq, Lk, H, Hk, D, dtype="bf16", seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(DT[dtype])

    return n(B, Lq, H, D), n(B, Lk, Hk, D), n(B, Lk, Hk, D)


def exact(q, k, v, keep=None, scale=None):
    """(o, bound on the kernel's error) in 64 bits; keep [B, Lk]."""
    B, Lq, H, D = q.shape
    Lk, G = k.shape[1], H // k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    h = 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -11
    q, k, v = q.double(), k.double(), v.double()
    if keep is not None:
        k = torch.where(keep[:, :, None, None], k, 0.0)
        v = torch.where(keep[:, :, None, None], v, 0.0)
    k, v = k.repeat_interleave(G, 2), v.repeat_interleave(G, 2)
    s = torch.einsum("blhd,bthd->bhlt", q, k) * scale
    size = torch.einsum("blhd,bthd->bhlt", q.abs(), k.abs()) * scale
    if keep is not None:
        s = s.masked_fill(~keep[:, None, None, :], float("-inf"))
    if Lk == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    some = (s > float("-inf")).any(-1, keepdim=True)
    p = torch.where(some, torch.softmax(torch.where(some, s, 0.0), -1), 0.0)
    o = torch.einsum("bhlt,bthd->blhd", p, v)
    A = torch.einsum("bhlt,bthd->blhd", p, v.abs())
    top = torch.where(s > float("-inf"), s.abs(), 0.0).max()
    E = h + 2 * (2 * D * 2.0 ** -24 * size.max() + 2.0 ** -22 * top * 1.45 + 2.0 ** -22) + 4 * (Lk + 64) * 2.0 ** -24
    err = A * E + h * (o.abs() + A * E)
    if h < 2.0 ** -10:
        err = err + Lk * 2.0 ** -25 * v.abs().max()
    return o, err


def check(got, o, err, s_out=None):
    torch.cuda.synchronize()
    if s_out is None:
        bad = ~((got.double() - o).abs() <= err)
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((got.double() - o).abs().max()))
        return
    val = O.e4m3_decode(got.cpu().numpy()).astype(np.float64)
    lo, hi = (O.e4m3_decode(O.e4m3_encode((((o + s * err) / float(s_out)) * (1 + 0.0)).cpu().numpy().astype(np.float32)))
              for s in (-1.0001, 1.0001))
    assert ((lo <= val) & (val <= hi)).all()


def keep_of(B, Lk, lens=None, mask=None):
    keep = torch.ones((B, Lk), dtype=torch.bool, device="cuda")
    if lens is not None:
        keep &= torch.arange(Lk, device="cuda")[None] < lens[:, None]
    if mask is not None:
        keep &= mask.bool()
    return keep


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,Lq,Lk,H,Hk,D", [
    (1, 1, 1, 1, 1, 64), (1, 1, 512, 4, 4, 128), (2, 1, 700, 8, 2, 128), (1, 1, 5003, 8, 1, 64), (1, 3, 129, 5, 1, 80),
    (1, 128, 128, 2, 2, 128), (1, 129, 127, 2, 2, 64), (2, 256, 640, 3, 3, 128), (1, 257, 1000, 2, 1, 96),
    (2, 100, 300, 14, 2, 128), (1, 385, 64, 3, 3, 72), (3, 77, 999, 20, 4, 64), (1, 1000, 2, 6, 2, 8),
    (1, 1, 300, 128, 1, 128), (1, 2, 300, 100, 1, 128), (5, 640, 333, 2, 2, 40), (1, 20, 12000, 16, 2, 128)])
def test_shapes(W, B, Lq, Lk, H, Hk, D, dtype):
    q, k, v = make(B, Lq, Lk, H, Hk, D, dtype, seed=Lq + Lk)
    o = W.cross_attention(q, k, v)
    W.poll_device_error()
    check(o, *exact(q, k, v))


@pytest.mark.parametrize("B,Lq,Lk,H,Hk,D", [(4, 1, 600, 4, 2, 128), (4, 300, 600, 2, 2, 64), (4, 130, 300, 3, 1, 128),
                                            (4, 2, 3000, 4, 1, 80)])
@pytest.mark.parametrize("kind", ["lens", "mask", "both"])
@pytest.mark.parametrize("codes", [False, True])
def test_masks_with_anything_behind_them(W, B, Lq, Lk, H, Hk, D, kind, codes):
    """Lengths and masks, a sample without any key, and NaN, infinities and the
    type's largest values in keys and values that do not count."""
    q, k, v = make(B, Lq, Lk, H, Hk, D, seed=Lk)
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = mask = None
    if kind != "mask":
        lens = torch.tensor([0, Lk, 129, Lk - 1], dtype=torch.int32, device="cuda")
    if kind != "lens":
        mask = torch.rand((B, Lk), generator=g, device="cuda") < 0.5
        mask[1] = False
        mask[1, 200] = True                  # whole tiles without a key, then one
        mask[3, :140] = False
        if kind == "mask":
            mask[2] = False
    keep = keep_of(B, Lk, lens, mask)
    fill = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38], device="cuda").to(q.dtype)
    off = ~keep
    n = int(off.sum())
    k[off] = fill[torch.arange(n, device="cuda") % 4][:, None, None]
    v[off] = fill[(torch.arange(n, device="cuda") + 1) % 4][:, None, None]
    s_out = dev_f32(0.01) if codes else None
    o = W.cross_attention(q, k, v, kv_len=lens, kv_mask=mask, s_out=s_out)
    W.poll_device_error()
    ref, err = exact(q, k, v, keep)
    assert (ref[(~keep).all(1)] == 0).all()
    check(o, ref, err, s_out)


def test_lengths_out_of_range_are_clamped(W):
    q, k, v = make(3, 5, 200, 2, 2, 64)
    lens = torch.tensor([-5, 1000, 7], dtype=torch.int32, device="cuda")
    o = W.cross_attention(q, k, v, kv_len=lens)
    check(o, *exact(q, k, v, keep_of(3, 200, lens)))


def test_no_keys_and_no_queries(W):
    q, k, v = make(2, 3, 0, 4, 2, 64)
    o = W.cross_attention(q, k, v, out=torch.full_like(q, 9.0))
    torch.cuda.synchronize()
    assert (o == 0).all()
    q0 = q[:, :0]
    assert W.cross_attention(q0, k, v).shape == q0.shape
    assert W.cross_attention(q[:0], k[:0], v[:0]).numel() == 0


@pytest.mark.parametrize("Lq", [1, 300])
def test_strided_views(W, Lq):
    """Heads first in memory, slices of wider arrays, one array for all samples."""
    g = torch.Generator(device="cuda").manual_seed(2)
    wide = torch.randn((2, Lq, 3, 4, 128), generator=g, device="cuda").to(torch.bfloat16)
    q = wide[:, :, 1, :, 16:112]                                          # D = 96 inside 128
    kv = torch.randn((2, 2, 700, 2 * 96), generator=g, device="cuda").to(torch.bfloat16)
    k, v = kv[..., :96].transpose(1, 2), kv[..., 96:].transpose(1, 2)     # [B, Lk, Hk, D], heads outermost
    out = torch.zeros((2, 4, Lq, 104), dtype=torch.bfloat16, device="cuda")
    o = W.cross_attention(q, k, v, out=out[..., :96].transpose(1, 2))
    check(o, *exact(q, k, v))
    assert (out[..., 96:] == 0).all()
    k1, v1 = k[1:].expand(2, -1, -1, -1), v[1:].expand(2, -1, -1, -1)
    mask = torch.rand((1, 700), generator=g, device="cuda").lt(0.6).expand(2, -1)
    check(W.cross_attention(q, k1, v1, kv_mask=mask), *exact(q, k1, v1, mask))


@pytest.mark.parametrize("Lq,Lk", [(1, 2000), (300, 700)])
def test_scores_far_apart(W, Lq, Lk):
    """A running maximum that keeps growing, by little and by much, and a scale
    of its own."""
    q, k, v = make(1, Lq, Lk, 2, 2, 128, seed=7)
    k *= torch.linspace(0.01, 6.0, Lk, device="cuda").to(k.dtype)[None, :, None, None]
    check(W.cross_attention(q, k, v), *exact(q, k, v))
    q2 = q.abs()
    k2 = k.abs()                               # every later key is larger
    check(W.cross_attention(q2, k2, v, scale=0.2), *exact(q2, k2, v, scale=0.2))
    k3 = -k2                                   # the maximum stands in the first tile
    check(W.cross_attention(q2, k3, v, scale=0.05), *exact(q2, k3, v, scale=0.05))


def test_a_nan_query_spoils_its_own_row_only(W):
    q, k, v = make(1, 200, 300, 2, 1, 64)
    q[0, 17, 1] = float("nan")
    o = W.cross_attention(q, k, v)
    torch.cuda.synchronize()
    bad = torch.zeros((1, 200, 2, 64), dtype=torch.bool, device="cuda")
    bad[0, 17, 1] = True
    assert torch.equal(torch.isnan(o), bad)


@pytest.mark.parametrize("Lq", [1, 400])
def test_codes_are_the_rounded_output(W, Lq):
    for dtype, D in (("bf16", 128), ("f16", 72)):
        q, k, v = make(2, Lq, 260, 4, 2, D, dtype, seed=5)
        s_out = dev_f32(0.004)
        o = W.cross_attention(q, k, v, s_out=s_out)
        check(o, *exact(q, k, v), s_out)


def test_equal_calls_give_equal_bits_on_any_stream(W):
    for Lq, Lk in ((1, 6000), (500, 900)):
        q, k, v = make(1, Lq, Lk, 8, 2, 128, seed=11)
        want = W.cross_attention(q, k, v)
        ws = W.cross_attention_workspace(q, k, v)
        ws.fill_(float("nan"))                 # its contents mean nothing
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got = W.cross_attention(q, k, v, ws=ws)
        st.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(want.view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "f16")])
def test_long_keys_of_few_queries_back_to_back(W, D, dtype):
    """Key sides that come from memory tile by tile, cut over all CTAs, in calls
    that follow one another without a pause: the same bits each time."""
    q, k, v = make(6, 1, 9001, 12, 4, D, dtype, seed=13)
    outs = [W.cross_attention(q, k, v) for _ in range(12)]
    torch.cuda.synchronize()
    W.poll_device_error()
    for o in outs[1:]:
        assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))
    check(outs[0], *exact(q, k, v))


@pytest.mark.parametrize("Lq,H,Hk", [(1, 8, 2), (700, 4, 4)])
def test_lengths_of_many_samples(W, Lq, H, Hk):
    """Lengths from none to all of the keys, one tile and part of one, in turn:
    units of one and two tiles next to long ones in the same CTA; and more
    samples than the tile table has room for."""
    for B in (9, 70):
        if B == 70 and Lq > 1:
            continue
        q, k, v = make(B, Lq, 1500, H, Hk, 64, seed=B)
        lens = torch.tensor([[0, 1500, 128, 129, 1, 640, 0, 257, 1499][b % 9] for b in range(B)], dtype=torch.int32,
                            device="cuda")
        o = W.cross_attention(q, k, v, kv_len=lens)
        W.poll_device_error()
        check(o, *exact(q, k, v, keep_of(B, 1500, lens)))


@pytest.mark.parametrize("B,Lq,Lk,H,Hk,D", [(8, 1, 9000, 8, 2, 128), (100, 1, 6000, 2, 1, 64), (40, 1, 1500, 4, 4, 128),
                                            (2, 1, 2100, 64, 64, 64), (2, 2000, 2000, 12, 12, 64)])
def test_nothing_is_written_behind_the_workspace(W, B, Lq, Lk, H, Hk, D):
    """Exactly the workspace that was asked for, with and without lengths: what
    lies behind it keeps its contents."""
    q, k, v = make(B, Lq, Lk, H, Hk, D, seed=17)
    lens = torch.tensor([(b * 977) % (Lk + 1) for b in range(B)], dtype=torch.int32, device="cuda")
    n = W.cross_attention_workspace(q, k, v).numel()
    for kv_len in (lens, None):
        mem = torch.full((n + 4096,), 3.0, device="cuda")
        o = W.cross_attention(q, k, v, kv_len=kv_len, ws=mem[:n])
        W.poll_device_error()
        torch.cuda.synchronize()
        assert (mem[n:] == 3.0).all()
        rows = slice(0, 8) if Lq > 100 else slice(None)
        ref, err = exact(q[:, rows], k, v, None if kv_len is None else keep_of(B, Lk, kv_len))
        check(o[:, rows], ref, err)


def test_a_workspace_too_small_is_refused(W):
    q, k, v = make(1, 1, 6000, 8, 2, 128)
    ws = W.cross_attention_workspace(q, k, v)
    assert ws.numel() > 0
    with pytest.raises(W.W8Error) as e:
        W.cross_attention(q, k, v, ws=ws[:-8])
    assert e.value.status == 2


def test_long_offsets(W):
    """Keys whose offsets pass 32 bits: a view that starts 2^32 bytes into its
    array, with a sample's stride of more than 2^31 elements."""
    big = torch.zeros((2, 270000, 64, 128), dtype=torch.bfloat16, device="cuda")   # 8.8 GB
    g = torch.Generator(device="cuda").manual_seed(3)
    big[:, -300:] = torch.randn((2, 300, 64, 128), generator=g, device="cuda").to(torch.bfloat16)
    k, v = big[:, -300:, :32], big[:, -300:, 32:]
    q = torch.randn((2, 150, 32, 128), generator=g, device="cuda").to(torch.bfloat16)
    assert math.prod(big.shape[1:]) > 2 ** 31
    check(W.cross_attention(q, k, v), *exact(q, k, v))
