"""A self-attention site makes its buffers once: passes of any number of tokens, captured
ones among them, allocate nothing, and the one workspace is enough for each."""

import pytest
import torch

from gpu_util import W  # noqa: F401
from test_gpu_self_site import weights
from w8a16_linear_gb300.stack import SelfSite

pytestmark = pytest.mark.gpu


def cells(pages, page, kv_heads, D, codes=False):
    return [torch.zeros((pages, page, kv_heads, D), dtype=torch.uint8 if codes else torch.bfloat16, device="cuda") for _ in range(2)]


# sequences, tokens, most of one, heads, key heads, D, page, columns of the table, cells of codes
@pytest.mark.parametrize("B,tokens,max_q,heads,kv_heads,D,page,cols,codes", [
    (1, 300, 300, 8, 2, 64, 16, 120, False),      # 15 tiles: cut with up to 16 rows and not with more
    (1, 300, 300, 8, 2, 64, 16, 120, True), (1, 300, 300, 1, 1, 128, 16, 90, False), (4, 700, 200, 32, 8, 128, 64, 300, False),
    (2, 40, 20, 20, 4, 64, 48, 200, False), (300, 600, 2, 4, 2, 64, 16, 500, False), (1, 9, 9, 100, 1, 64, 16, 300, False),
    (1, 700, 700, 128, 1, 64, 16, 300, True), (3, 3, 1, 8, 2, 128, 16, 8, False)])
def test_one_workspace_is_enough_for_any_pass(W, B, tokens, max_q, heads, kv_heads, D, page, cols, codes):
    site = SelfSite(B, tokens, max_q, 64, heads, kv_heads, D, *cells(4, page, kv_heads, D, codes), cols)
    table = torch.empty((B, cols), dtype=torch.int32, device="cuda")
    need = [W.paged_attention_workspace(site.q[:n], site.k_cache, table, max_q=max_q).numel() for n in range(1, tokens + 1)]
    assert site.ws.numel() == max(need)


def test_passes_of_many_lengths_hold_no_more_memory(W):
    B, hidden, heads, kv_heads, D, page, cols = 2, 512, 32, 8, 128, 64, 60
    w, _ = weights(W, hidden, heads, kv_heads, D, norms=True, codes=False)
    table = torch.arange(B * cols, dtype=torch.int32, device="cuda").view(B, cols)
    site = SelfSite(B, 640, 320, hidden, heads, kv_heads, D, *cells(B * cols, page, kv_heads, D), cols)
    x, r = (torch.randn((640, hidden), device="cuda").bfloat16() for _ in range(2))
    lens = torch.full((B,), 3000, dtype=torch.int32, device="cuda")
    site.run(W, w, x, r, table, None, lens)
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    for n in [1, 2, 3, 5, 8, 40, 61, 128, 129, 250, 319, 320]:
        site.run(W, w, x[:2 * n], r[:2 * n], table, None, lens)
        torch.cuda.synchronize()
        assert torch.cuda.memory_allocated() == held, n
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=st):                 # a number of tokens not met before
        held = torch.cuda.memory_allocated()                 # the graph has made its generators' state
        y, res = site.run(W, w, x[:34], r[:34], table, None, lens)
        assert torch.cuda.memory_allocated() == held
    graph.replay()
    got = [t.clone() for t in (y, res)]
    want = site.run(W, w, x[:34], r[:34], table, None, lens)
    torch.cuda.synchronize()
    W.poll_device_error()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_more_tokens_than_the_site_was_made_for_are_refused(W):
    w, _ = weights(W, 512, 8, 2, 64, norms=False, codes=False)
    site = SelfSite(1, 4, 4, 512, 8, 2, 64, *cells(4, 16, 2, 64), 4)
    x = torch.zeros((5, 512), dtype=torch.bfloat16, device="cuda")
    with pytest.raises((W.W8Error, RuntimeError)):
        site.run(W, w, x, x, torch.zeros((1, 4), dtype=torch.int32, device="cuda"), None,
                 torch.full((1,), 5, dtype=torch.int32, device="cuda"))
