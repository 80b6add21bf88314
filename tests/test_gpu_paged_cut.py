"""paged_attention where units of 256 rows are cut: every CTA finds the unit in which
its share begins from the places where the sequences begin, which one warp's lanes write and
others read.  A CTA that read a stale place would begin elsewhere than its neighbour
ends, and rows of the units between would be missing or counted twice.
"""

import pytest
import torch

from gpu_util import W  # noqa: F401
from paged_util import batch, exact_attention
from test_gpu_paged_attention import call, check, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [2, 31, 33, 64, 130, 256])
@pytest.mark.parametrize("codes", [False, True])
def test_shares_begin_in_any_sequence(W, B, codes):
    """One long past beside many short ones makes the lengths uneven, so that tiles are
    shared out; sequences with no token or no past stand between."""
    new = [(29 * i) % 41 for i in range(B)]
    new[B // 2] = 200                                        # more than 128 rows: units of 256
    lens = [n + (53 * i) % 300 for i, n in enumerate(new)]
    lens[B - 1], new[B - 1] = 9000, 150
    b = batch(new, lens, 64, 1, 64, codes=codes, seed=B, cols=(9000 + 63) // 64)
    q = queries(b, 2, 64)
    o = exact_attention(b, q)
    got = call(W, b, q, max_q=200)
    check(got, *o)
    for _ in range(4):
        assert torch.equal(call(W, b, q, max_q=200), got)
