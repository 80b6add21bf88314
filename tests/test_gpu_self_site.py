"""A self-attention site over a paged cache end to end: norm with the residual's
addition, projections, norms and rotation of the heads on the way into the cache,
attention over it, out-projection; prompts first, then single tokens.

Each step's own kernel is checked elsewhere; here the site's output is compared
with the same site in 32 bits throughout.  Four E4M3 roundings lie between the two
(tokens, weights, attention's output, and with a cache of codes its cells): each has
a relative error of at most 2^-4 a value, 2^-4 / sqrt(3) in the mean square.  Values of
independent signs add in squares; the products have two of them, so the output's relative error
(2-norm) stays below sqrt(7) 2^-4 / sqrt(3) < 0.1; the queries' and keys' errors
also pass through the softmax, whose scores here are of the order of one (0.12 with codes).
"""

import pytest
import torch

from gpu_util import W, dev_f32  # noqa: F401
from w8a16_linear_gb300.stack import SelfSite, SelfWeights

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def weights(W, hidden, heads, kv_heads, D, norms, codes, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def mat(n, k):
        w = torch.randn((n, k), generator=g, device="cuda") * k ** -0.5
        s = w.abs().amax(1) / 448
        return w, ((w / s[:, None]).to(F8).view(torch.uint8), s)

    def norm(n):
        return (1 + 0.1 * torch.randn((n,), generator=g, device="cuda")).bfloat16()

    q, k, v = mat(heads * D, hidden), mat(kv_heads * D, hidden), mat(kv_heads * D, hidden)
    o = torch.randn((hidden, heads * D), generator=g, device="cuda") * (heads * D) ** -0.5
    s_o = o.abs().max() / 448
    f = W.rope_frequencies(D)
    w = SelfWeights(norm(hidden), q[1], k[1], v[1], ((o / s_o).to(F8).view(torch.uint8), s_o.reshape(1)), dev_f32(3.0 / 448),
                    W.rope_turns(f), *((norm(D), norm(D)) if norms else (None, None)),
                    *((dev_f32(6.0 / 448), dev_f32(6.0 / 448)) if codes else (None, None)))
    return w, (q[0], k[0], v[0], o, f.cuda())


def plain(w, mats, xs, rs, past, heads, kv_heads, D):
    """Of each sequence (new x and residual, past hidden sums): the output of the new tokens."""
    def rms(t, n):
        return t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * (1 if n is None else n.float())

    out = []
    for x, r, p in zip(xs, rs, past):
        h = rms(torch.cat([p, x.float() + r.float()]), w.norm)
        q, k, v = (h @ m.T for m in mats[:3])
        pos = torch.arange(h.shape[0], device="cuda").double()[:, None] * mats[4]
        c, s = pos.cos().float()[:, None], pos.sin().float()[:, None]

        def turned(t, n):
            t = t.view(h.shape[0], -1, D)
            if n is not None:
                t = rms(t, n)
            a, b = t[..., :D // 2], t[..., D // 2:]
            return torch.cat([a * c - b * s, b * c + a * s], -1)

        q, k, v = turned(q, w.q_norm), turned(k, w.k_norm), v.view(h.shape[0], -1, D)
        k, v = (t.repeat_interleave(heads // kv_heads, 1) for t in (k, v))
        e = torch.einsum("lhd,thd->hlt", q[p.shape[0]:], k) * D ** -0.5
        later = torch.ones(e.shape[1:], dtype=torch.bool, device="cuda").triu(p.shape[0] + 1)
        a = torch.einsum("hlt,thd->lhd", torch.softmax(e.masked_fill(later, float("-inf")), -1), v)
        out.append(a.reshape(x.shape[0], -1) @ mats[3].T)
    return torch.cat(out)


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("hidden,heads,kv_heads,D,page,prompts", [(512, 8, 2, 64, 16, [150, 1, 37]), (512, 4, 4, 128, 32, [300, 90]),
                                                                  (1024, 16, 2, 128, 64, [20, 5, 700, 64])])
def test_site_matches_its_unquantized_form(W, hidden, heads, kv_heads, D, page, prompts, codes):
    w, mats = weights(W, hidden, heads, kv_heads, D, norms=D == 128, codes=codes, seed=D)
    g = torch.Generator(device="cuda").manual_seed(7)
    B, cols = len(prompts), (max(prompts) + 8 + page - 1) // page
    pages = B * cols + 2
    shape = (pages, page, kv_heads, D)
    cells = dict(dtype=torch.uint8 if codes else torch.bfloat16, device="cuda")
    kc, vc = (torch.full(shape, 0x7F if codes else float("nan"), **cells) for _ in range(2))   # never written: NaN
    table = torch.randperm(pages, generator=g, device="cuda")[:B * cols].view(B, cols).to(torch.int32)
    site = SelfSite(B, sum(prompts), max(prompts), hidden, heads, kv_heads, D, kc, vc, cols)
    step = SelfSite(B, B, 1, hidden, heads, kv_heads, D, kc, vc, cols)
    past = [torch.empty((0, hidden), device="cuda") for _ in prompts]
    lens = [0] * B
    for new in (prompts, [1] * B, [1] * B):
        lens = [a + n for a, n in zip(lens, new)]
        x, r = (torch.randn((sum(new), hidden), generator=g, device="cuda").bfloat16() for _ in range(2))
        start = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
        kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        y, res = (site if new is prompts else step).run(W, w, x, r, table, start, kv_len)
        torch.cuda.synchronize()
        W.poll_device_error()
        xs, rs = x.split(new), r.split(new)
        ref = plain(w, mats, xs, rs, past, heads, kv_heads, D)
        assert float((y.float() - ref).norm() / ref.norm()) < (0.12 if codes else 0.1)
        assert torch.equal(res, (x.float() + r.float()).bfloat16())
        past = [torch.cat([p, a.float() + b.float()]) for p, a, b in zip(past, xs, rs)]


def test_one_graph_serves_every_step(W):
    """Single tokens replayed from one graph: the lengths move on, and the bits are
    those of eager passes over the same cache."""
    B, hidden, heads, kv_heads, D, page, cols = 3, 512, 8, 2, 64, 16, 20
    w, _ = weights(W, hidden, heads, kv_heads, D, norms=True, codes=True)
    g = torch.Generator(device="cuda").manual_seed(9)
    shape = (B * cols, page, kv_heads, D)
    table = torch.randperm(B * cols, generator=g, device="cuda").view(B, cols).to(torch.int32)
    caches = [[torch.randint(0, 0x70, shape, generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]]
    caches.append([c.clone() for c in caches[0]])
    eager, captured = (SelfSite(B, B, 1, hidden, heads, kv_heads, D, *c, cols) for c in caches)
    x, r = (torch.randn((B, hidden), generator=g, device="cuda").bfloat16() for _ in range(2))
    kv_len = torch.tensor([300, 17, 1], dtype=torch.int32, device="cuda")
    lens = kv_len.clone()
    captured.run(W, w, x, r, table, None, lens)
    torch.cuda.synchronize()
    for a, b in zip(caches[0], caches[1]):
        b.copy_(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        captured.run(W, w, x, r, table, None, lens)
    for step in range(4):
        for t in (x, r):
            t.copy_(torch.randn((B, hidden), generator=g, device="cuda"))
        lens.copy_(kv_len + step)
        want = [t.clone() for t in eager.run(W, w, x, r, table, None, lens)]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured.y, want[0]) and torch.equal(captured.res, want[1])
        assert all(torch.equal(a, b) for a, b in zip(*caches))
    W.poll_device_error()
