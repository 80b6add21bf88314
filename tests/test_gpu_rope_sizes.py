"""qk_norm_rope over many tokens of heads whose sizes leave lanes without values; the bound is test_gpu_rope.py's."""

import pytest
import torch

from gpu_util import W  # noqa: F401
from paged_util import exact_heads, near, spread
from test_gpu_rope import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("M,Hq,Hk,D,rot", [(9001, 20, 4, 80, 80), (20670, 8, 8, 96, 48), (12345, 5, 1, 24, 16), (4099, 7, 2, 200, 192)])
def test_many_tokens(W, M, Hq, Hk, D, rot, interleaved, dtype):
    q, k, wq, wk, pos = make(M, Hq, Hk, D, dtype, seed=D)
    f = W.rope_frequencies(rot)
    qo, ko = W.qk_norm_rope(q, k, pos, W.rope_turns(f), q_weight=wq, k_weight=wk, interleaved=interleaved)
    torch.cuda.synchronize()
    for x, w, got in ((q, wq, qo), (k, wk, ko)):
        assert near(got, *exact_heads(x, w, spread(pos, rot // 2), f.cuda(), interleaved=interleaved))
    # the same in the inputs' own memory
    for t, out in zip(W.qk_norm_rope(q, k, pos, W.rope_turns(f), q_weight=wq, k_weight=wk, interleaved=interleaved, q_out=q, k_out=k),
                      (qo, ko)):
        assert torch.equal(t, out)
