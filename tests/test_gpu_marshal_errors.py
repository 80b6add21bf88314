"""Arguments that raise while they are read: the exception is the caller's, and nothing has run."""

import pytest
import torch

from gpu_util import W  # noqa: F401
from test_gpu_marshal import CALLS, b  # noqa: F401

pytestmark = pytest.mark.gpu


class Unclear:
    def __bool__(self):
        raise ValueError("neither")


@pytest.mark.parametrize("name,make", CALLS)
def test_a_flag_without_a_truth_value(b, name, make):  # noqa: F811
    args = make()
    flag = "causal" if name == "paged_attention" else "interleaved"
    outs = [args[k] for k in ("q_out", "k_out", "out") if k in args]
    before = [t.clone() for t in outs]
    with pytest.raises(ValueError, match="neither"):
        getattr(b, name)(**args, **{flag: Unclear()})
    torch.cuda.synchronize()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(outs, before))
    getattr(b, name)(**args)                                 # and no exception is left behind
    torch.cuda.synchronize()
