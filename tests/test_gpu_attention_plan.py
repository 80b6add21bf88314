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
