"""cross_attention at the ends of what its plan allows: the number of samples
whose lengths the tile table holds, and queries that all samples share."""

import pytest
import torch

from gpu_util import W  # noqa: F401
from test_gpu_attention import check, exact, keep_of, make

pytestmark = pytest.mark.gpu


def test_workspace_of_queries_that_all_samples_share(W):
    q, k, v = make(3, 1, 6000, 8, 2, 128, seed=41)
    q = q[:1].expand(3, -1, -1, -1)
    ws = W.cross_attention_workspace(q, k, v)
    assert ws.numel() == W.cross_attention_workspace(q.contiguous(), k, v).numel() > 0
    o = W.cross_attention(q, k, v, ws=ws)
    W.poll_device_error()
    check(o, *exact(q, k, v))
    assert torch.equal(o, W.cross_attention(q.contiguous(), k, v))


@pytest.mark.parametrize("B", [127, 128, 129])
def test_samples_around_what_the_tile_table_holds(W, B):
    """Up to 128 samples with lengths of their own are cut along the keys, by a
    table in shared memory; more are not.  One token over 30000 keys with one
    head: one item a sample, which the plan cuts where it may (a workspace is
    wanted)."""
    Lk = 30000
    q, k, v = make(B, 1, Lk, 1, 1, 64, seed=B)
    lens = torch.tensor([[Lk, 0, 1, 12345, 128, 29999, Lk, 777][b % 8] for b in range(B)], dtype=torch.int32, device="cuda")
    lens[-1] = Lk - 3                                  # the table's last entry
    ws = W.cross_attention_workspace(q, k, v)
    assert (ws.numel() > 0) == (B <= 128)
    o = W.cross_attention(q, k, v, kv_len=lens, ws=ws)
    W.poll_device_error()
    check(o, *exact(q, k, v, keep_of(B, Lk, lens)))
