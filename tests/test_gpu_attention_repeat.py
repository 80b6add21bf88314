"""Equal calls of cross_attention give equal bits whatever ran before them.

Where the query heads of a key head do not divide 128, a slot has rows without
a query (two of 128 for groups of three or seven).  What they hold must not
reach the other rows, not even by way of when a warp raises its running maxima."""

import pytest
import torch

from gpu_util import W  # noqa: F401

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Lq,Hk,G", [(1, 5040, 3, 3), (1, 2160, 3, 7), (64, 18, 3, 7), (64, 42, 3, 3), (40, 25, 4, 5), (2, 200, 1, 100)])
def test_bits_do_not_depend_on_the_call_before(W, B, Lq, Hk, G, D, dtype):
    """Calls over full slots in between leave large and zero queries in the
    rows in question; the scores grow from tile to tile, by less than what
    makes a row raise its own maximum but by more for the large queries."""
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(G)
    Lk = 640
    q = (torch.randn((B, Lq, Hk * G, D), generator=g, device="cuda") * 0.3).to(dt)
    grow = torch.linspace(0.1, 2.0, Lk, device="cuda")[None, :, None, None]
    k = (grow * (1 + 0.3 * torch.randn((B, Lk, Hk, D), generator=g, device="cuda"))).to(dt)
    v = torch.randn((B, Lk, Hk, D), generator=g, device="cuda").to(dt)
    fills = [torch.full((1, 6400, 4, D), c, dtype=dt, device="cuda") for c in (0.0, 20.0, -20.0, 0.0)]
    fill_out, outs = torch.empty_like(fills[0]), [torch.empty_like(q) for _ in fills]
    fk = torch.ones((1, 128, 4, D), dtype=dt, device="cuda")
    ws = W.cross_attention_workspace(q, k, v)
    for f, o in zip(fills, outs):
        W.cross_attention(f, fk, fk, out=fill_out)
        W.cross_attention(q, k, v, out=o, ws=ws)
    torch.cuda.synchronize()
    W.poll_device_error()
    for o in outs[1:]:
        assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))
