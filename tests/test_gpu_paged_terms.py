"""Queries of widely spread magnitudes over E4M3 cells with few rows, where a query is held as three
E4M3 terms x = (t0 + t1 / 16 + t2 / 256) 2^e.

With 2^e the row's largest value is in [2^7, 2^8) of the terms.  Each term has 4 significant bits, so
three of them hold a bf16 value (8 bits) and an f16 value (11) exactly until t2 is below 2^-6 and has
fewer: for bf16 from 2^-17 of the row's largest on nothing is left, for f16 from 2^-14, and
otherwise at most half of t2's smallest step, 2^-10 / 256 = 2^-18 in units of the terms, 2^-25 of the
row's largest.  A score is then off by at most scale 2^-25 max|q| sum|k|, which
changes each weight by twice that (both ends of the quotient) and the result by that times max|v|.
"""

import pytest
import torch

from gpu_util import W  # noqa: F401
from paged_util import F8, batch, exact_attention, half_step, values
from test_gpu_paged_attention import call, check


def terms(x):
    """x (64 bits, in units of the terms) as the kernel holds it."""
    y, s = torch.zeros_like(x), 1.0
    rest = x.clone()
    for _ in range(3):
        t = rest.clamp(-448, 448).float().to(F8).double()
        y, rest, s = y + t * s, (rest - t) * 16, s / 16
    return y


@pytest.mark.parametrize("bits,exact", [(7, -17), (10, -14)])
@pytest.mark.parametrize("top", [128.0, 192.0, 255.0])
def test_what_the_terms_leave(bits, exact, top):
    m = 1 + torch.arange(2 ** bits).double() / 2 ** bits
    for e in range(-50, 8):
        x = m * 2.0 ** e
        x = x[x <= top]
        left = (terms(x) - x).abs()
        assert (left <= 2.0 ** -25 * top).all()
        assert (left[x >= 2.0 ** exact * top] == 0).all()


def spread_queries(b, H, D, largest, low, seed):
    """Magnitudes of [low, 2 low) but for dimension 0 of each row, which is `largest`."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (low + low * torch.rand((b.T, H, D), generator=g, device="cuda")) * (torch.randint(0, 2, (b.T, H, D), generator=g, device="cuda") * 2 - 1)
    q[..., 0] = largest
    return q.to(b.dt)


SHAPES = [([1], [700], 8, 2, 64), ([3, 1], [3000, 200], 4, 1, 128), ([1] * 4, [900, 5000, 33, 1], 8, 2, 80)]


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens,H,Hk,D", SHAPES)
@pytest.mark.parametrize("dtype,largest", [("bf16", 2.0 ** 16), ("f16", 2.0 ** 13)])
def test_values_that_the_terms_hold(W, new, lens, H, Hk, D, dtype, largest):
    """The small ones make the scores: the keys' dimension 0 is 0."""
    b = batch(new, lens, 16, Hk, D, dtype, codes=True)
    b.k[..., 0] = 0
    q = spread_queries(b, H, D, largest, 1.0, seed=D)
    check(call(W, b, q), *exact_attention(b, q))


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens,H,Hk,D", SHAPES)
@pytest.mark.parametrize("dtype,largest,low", [("bf16", 2.0 ** 19, 1.0), ("bf16", 2.0 ** 60, 2.0 ** 36), ("f16", 2.0 ** 15, 2.0 ** -3)])
def test_values_that_they_round(W, new, lens, H, Hk, D, dtype, largest, low):
    b = batch(new, lens, 16, Hk, D, dtype, codes=True)
    b.k[..., 0] = 0
    q = spread_queries(b, H, D, largest, low, seed=D)
    scale = D ** -0.5 / low
    o, err, written = exact_attention(b, q, scale=scale)
    for i, x in enumerate(lens):
        t0 = sum(new[:i])
        k, v = values(b, "k", i, x), values(b, "v", i, x)
        delta = scale * 2.0 ** -25 * largest * float(k.abs().sum(-1).max())
        err[t0:t0 + new[i]] += (torch.tensor(2 * delta).exp().double() - 1).item() * float(v.abs().max()) * (1 + half_step(b.dt))
    check(call(W, b, q, scale=scale), o, err, written)
