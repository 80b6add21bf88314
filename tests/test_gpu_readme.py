"""The README's lines for new tokens over their past, run as they stand: queries and keys are
normed and turned once, and the attention is that of those."""

import os

import pytest
import torch

from gpu_util import W  # noqa: F401
from paged_util import batch, exact_attention, exact_heads, near, spread

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def lines():
    with open(os.path.join(ROOT, "README.md")) as f:
        code = f.read().split("```python")[1].split("```")[0]
    return code[code.index("turns ="):]


def test_self_attention_lines(W):
    B, Hq, Hk, D, page = 5, 8, 2, 64, 16
    lens = [40, 17, 1, 33, 100]
    b = batch([1] * B, lens, page, Hk, D)
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v, q_latent, k_latent, wqn, wkn = n(B, Hq, D), n(B, Hk, D), n(B, Hk, D), n(9, Hq, D), n(9, Hk, D), n(D), n(D)
    positions = torch.arange(9, dtype=torch.int32, device="cuda") * 7
    names = dict(W=W, D=D, q=q.clone(), k=k, v=v, q_latent=q_latent, k_latent=k_latent, positions=positions, wqn=wqn, wkn=wkn,
                 k_cache=b.k, v_cache=b.v, page_table=b.table, q_start=b.q_start, kv_len=b.kv_len)
    exec(lines(), names)
    torch.cuda.synchronize()
    W.poll_device_error()
    f = W.rope_frequencies(D).cuda()
    at = torch.tensor(lens, device="cuda") - 1
    assert near(names["q"], *exact_heads(q, wqn, spread(at, D // 2), f))
    cells = b.table[torch.arange(B, device="cuda"), at // page].long(), at % page
    assert near(b.k[cells], *exact_heads(k, wkn, spread(at, D // 2), f)) and torch.equal(b.v[cells], v)
    o, err, _ = exact_attention(b, names["q"])
    assert ((names["o"].double() - o).abs() <= err).all()
    for x, w, got in ((q_latent, wqn, names["q_turned"]), (k_latent, wkn, names["k_turned"])):
        assert near(got, *exact_heads(x, w, spread(positions, D // 2), f))
