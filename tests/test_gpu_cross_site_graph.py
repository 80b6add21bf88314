"""A captured pass of CrossSite after further encodes: the bits of an eager
pass over the states that the graph is to attend to."""

import pytest
import torch

from gpu_util import W  # noqa: F401
from test_gpu_cross_site import weights
from w8a16_linear_gb300.stack import CrossSite

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L,heads,kv_heads,D,T", [(3, 8, 2, 64, 2000), (300, 4, 4, 128, 200)])
def test_graph_attends_to_the_states_encoded_last(W, L, heads, kv_heads, D, T):
    B, hidden = 2, 512
    w, _ = weights(hidden, 384, heads, kv_heads, D)
    g = torch.Generator(device="cuda").manual_seed(31)
    x, r = (torch.randn((B * L, hidden), generator=g, device="cuda").bfloat16() for _ in range(2))
    prompts = [torch.randn((B, t, 384), generator=g, device="cuda").bfloat16() for t in (T, T, T // 2, T)]

    def eager(states):
        site = CrossSite(B, L, hidden, heads, kv_heads, D, x.device)
        site.encode(W, w, states)
        return site.run(W, w, x, r)[0].clone()

    want = [eager(p) for p in prompts]
    site = CrossSite(B, L, hidden, heads, kv_heads, D, x.device)
    site.encode(W, w, prompts[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        site.run(W, w, x, r)

    def replay():
        site.y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        return site.y.clone()

    def same(a, b):
        return torch.equal(a.view(torch.int16), b.view(torch.int16))

    assert same(replay(), want[0])
    site.encode(W, w, prompts[1])                  # as many positions: the graph sees them
    assert same(replay(), want[1])
    site.encode(W, w, prompts[2])                  # half as many: an eager pass, and the graph as before
    assert same(site.run(W, w, x, r)[0], want[2])
    others = [torch.full((B * T, kv_heads * D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(6)]
    assert same(replay(), want[1])
    assert all(bool((t == 5).all()) for t in others)
    site.encode(W, w, prompts[3])
    assert same(replay(), want[3])
    W.poll_device_error()
