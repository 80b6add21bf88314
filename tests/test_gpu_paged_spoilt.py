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
