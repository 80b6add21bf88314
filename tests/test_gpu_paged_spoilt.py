"""paged_attention over values that are not finite: what one unit of a CTA meets must
not change how another unit's rows are written, and what a row gets does not depend
on how the tokens are taken together.
"""

import pytest
import torch

from gpu_util import W, dev_f32  # noqa: F401
from paged_util import batch
from test_gpu_paged_attention import call, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("out8", [False, True])
def test_other_sequences_keep_their_bits(W, codes, out8):
    """More units than CTAs; NaN among the values of every third sequence's new tokens, met
    while a CTA's unit before is written by whole rows."""
    B = 90
    new = [300 + 7 * i % 40 for i in range(B)]
    b = batch(new, new, 16, 2, 128, codes=codes)
    q = queries(b, 8, 128)
    kw = dict(max_q=max(new), s_out=dev_f32(2.0 / 448) if out8 else None)
    want = call(W, b, q, **kw).clone()
    for i in range(0, B, 3):
        for p in (new[i] // 3, new[i] - 2):
            b.v[b.table[i, p // 16].long(), p % 16, 0, 5] = 0x7F if codes else float("nan")
    for _ in range(5):
        got = call(W, b, q, **kw)
        t = 0
        for i, n in enumerate(new):
            rows, whole = got[t:t + n].clone(), want[t:t + n]
            if i % 3 == 0:
                bad = rows[n // 3:, :4, 5]
                assert (bad & 0x7F == 0x7F).all() if out8 else torch.isnan(bad).all()
                rows[n // 3:, :4, 5] = whole[n // 3:, :4, 5]
            assert torch.equal(rows.view(torch.uint8), whole.view(torch.uint8)), i
            t += n


def outcome(b, i, value, causal=True):
    """For each new token of sequence i and key head and dimension: +1, -1 where it sees infinities
    of one sign alone, 0 where it sees none, NaN where it sees both or NaN."""
    n, x = b.new[i], b.lens[i]
    at = torch.arange(x, device="cuda")
    v = b.v[b.table[i][at // b.page].long(), at % b.page]                       # [x, Hk, D]
    ok = (at[None] <= (x - n + torch.arange(n, device="cuda")[:, None] if causal else x)).expand(n, x)
    some = [(torch.einsum("lt,thd->lhd", ok.double(), m.double()) > 0) for m in value(v)]
    return torch.where(some[2] | (some[0] & some[1]), float("nan"), some[0].double() - some[1].double())


# 256 rows, 128 rows, few rows; whole units and cut ones
@pytest.mark.parametrize("new,lens,H,Hk,D", [([300], [300], 2, 2, 64), ([200, 280], [333, 700], 8, 2, 128), ([40], [300], 4, 2, 80),
                                             ([40, 31], [6000, 100], 2, 1, 128), ([400], [9000], 1, 1, 64), ([9], [200], 1, 1, 64),
                                             ([5, 3], [5000, 4000], 6, 2, 128), ([1], [900], 4, 1, 64)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("out8", [False, True])
def test_an_infinity_stays_one(W, new, lens, H, Hk, D, causal, out8):
    """The formula's infinity, whether all rows that are worked on together see it or some:
    scores are near 0, so that no weight vanishes.  E4M3 results saturate."""
    inf, nan = float("inf"), float("nan")
    b = batch(new, lens, 16, Hk, D)
    for i, (n, x) in enumerate(zip(new, lens)):
        for p, d, value in ((x - n, 0, inf), (x - n + n // 2, 1, -inf), (x - 1, 2, inf), (x - n + n // 3, 3, inf), (x - 1, 3, -inf),
                            (x - n + n // 3, 4, inf), (x - n + 2 * n // 3, 4, nan), (0, 5, -inf), (x // 2, 6, inf), (x - 1, 6, inf),
                            (x // 2, 7, inf), (x - n + n // 2, 7, -inf)):
            b.v[b.table[i, p // 16].long(), p % 16, Hk - 1, d] = value
    q = queries(b, H, D, std=0.1)
    s_out = dev_f32(2.0 / 448) if out8 else None
    got = call(W, b, q, causal=causal, s_out=s_out)
    t = 0
    for i, n in enumerate(new):
        want = outcome(b, i, lambda v: (v == inf, v == -inf, torch.isnan(v)), causal).repeat_interleave(H // Hk, 1)
        rows = got[t:t + n]
        if out8:
            rows = rows.view(torch.float8_e4m3fn)
        rows = rows.double()
        top = 448.0 if out8 else inf
        assert torch.equal(torch.isnan(rows), torch.isnan(want)), (torch.isnan(rows) != torch.isnan(want)).nonzero()[:5].tolist()
        assert (rows[want > 0] == top).all() and (rows[want < 0] == -top).all()
        assert out8 or torch.isfinite(rows[want == 0]).all()     # codes of 2 and more are 448 too: a row that sees few values
        t += n


@pytest.mark.parametrize("new,lens,H,Hk", [([300], [500], 2, 1), ([30], [3000], 4, 2), ([3], [2000], 4, 2)])
def test_nan_codes_reach_the_rows_that_see_them(W, new, lens, H, Hk):
    b = batch(new, lens, 16, Hk, 64, codes=True)
    n, x = new[0], lens[0]
    for p, d in ((x - n + n // 2, 0), (x - 1, 1), (3, 2)):
        b.v[b.table[0, p // 16].long(), p % 16, 0, d] = 0xFF
    got = call(W, b, queries(b, H, 64, std=0.1))
    want = outcome(b, 0, lambda v: (v < 0, v < 0, v & 0x7F == 0x7F)).repeat_interleave(H // Hk, 1)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and not torch.isinf(got).any()
