"""GPU parity of paged_kv_append against the formula in 64 bits: the norm and
rotation as in test_gpu_rope.py, and a code's argument has two more roundings (the
scale's reciprocal and the product), 2^-23 of it.  Cells of other positions, pages and
heads keep their bits."""

import pytest
import torch

from gpu_util import W  # noqa: F401
from paged_util import batch, code_near, exact_heads, near, spread

pytestmark = pytest.mark.gpu


def tokens(b, Hq, Hk, D, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = (torch.randn((b.T, Hq + 2 * Hk, D), generator=g, device="cuda") * 1.5).to(b.dt)
    w = [(1 + 0.2 * torch.randn((D,), generator=g, device="cuda")).to(b.dt) for _ in range(2)]
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], *w


def places(b):
    """(token, page, cell, position) of every new token that has a page."""
    out, t = [], 0
    for i, (n, x) in enumerate(zip(b.new, b.lens)):
        for j in range(n):
            p = x - n + j
            if 0 <= p < b.cols * b.page and 0 <= int(b.table[i, p // b.page]) < b.k.shape[0]:
                out.append((t, int(b.table[i, p // b.page]), p % b.page, p))
            t += 1
    return torch.tensor(out, dtype=torch.long).reshape(-1, 4).T.cuda()


def positions(b):
    return torch.cat([torch.arange(x - n, x) for n, x in zip(b.new, b.lens)]).cuda()


def check(b, before, q, k, v, w, q_out, f, pos=None, **kw):
    torch.cuda.synchronize()
    pos = spread(positions(b) if pos is None else pos, len(f)) if f is not None else None
    f = None if f is None else f.cuda()
    y, e = exact_heads(k, w[1], pos, f, **kw)
    t, page, cell, _ = places(b)
    for name, want, err in (("k", y, e), ("v", v.double(), torch.zeros_like(v, dtype=torch.float64))):
        c, old = getattr(b, name), before[name]
        got = c[page, cell]
        if b.codes:
            s = float(getattr(b, name + "_scale"))
            want, err = want[t] / s, err[t] / s + want[t].abs() / s * 2.0 ** -23
            assert code_near(got, want, err), name
        elif name == "v":
            assert torch.equal(got, v[t])
        else:
            assert near(got, want[t], err[t])
        rest = torch.ones(c.shape[:2], dtype=torch.bool, device="cuda")
        rest[page, cell] = False
        assert torch.equal(c.view(torch.uint8)[rest], old.view(torch.uint8)[rest]), name
    if q is not None:
        assert near(q_out, *exact_heads(q, w[0], pos, f, **kw))


def run(W, b, q, k, v, w, f, **kw):
    before = {"k": b.k.clone(), "v": b.v.clone()}
    turns = None if f is None else W.rope_turns(f)
    q_out = W.paged_kv_append(k, v, b.k, b.v, b.table, kw.pop("q_start", b.q_start), b.kv_len, turns=turns, q=q, q_weight=w[0],
                              k_weight=w[1], k_scale=b.k_scale, v_scale=b.v_scale, **kw)
    return before, q_out


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new,lens,page,Hq,Hk,D,rot", [
    ([1], [1], 16, 4, 2, 128, 128), ([1] * 8, [2067, 1, 16, 17, 33, 500, 48, 1999], 16, 32, 8, 128, 128),
    ([333, 1, 0, 170], [999, 1, 5, 170], 48, 20, 4, 64, 64), ([700, 40], [700, 1000], 64, 3, 1, 80, 32),
    ([5, 5, 5], [9, 5, 300], 8, 6, 6, 96, 48), ([130], [131], 256, 1, 1, 16, 16)])
def test_shapes(W, new, lens, page, Hq, Hk, D, rot, dtype, codes):
    b = batch(new, lens, page, Hk, D, dtype, codes, seed=D)
    q, k, v, wq, wk = tokens(b, Hq, Hk, D)
    f = W.rope_frequencies(rot)
    for interleaved, norm, queries in ((False, True, True), (True, False, False), (True, True, True)):
        w = (wq if norm and queries else None, wk if norm else None)
        before, qo = run(W, b, q if queries else None, k, v, w, f, interleaved=interleaved)
        check(b, before, q if queries else None, k, v, w, qo, f, interleaved=interleaved)


def test_uniform_batches_without_starts(W):
    b = batch([3] * 5, [3, 40, 17, 300, 4], 16, 2, 64)
    q, k, v, wq, wk = tokens(b, 4, 2, 64)
    f = W.rope_frequencies(64)
    before, qo = run(W, b, q, k, v, (wq, wk), f, q_start=None)
    check(b, before, q, k, v, (wq, wk), qo, f)


@pytest.mark.parametrize("codes", [False, True])
def test_plain_append_and_given_positions(W, codes):
    b = batch([50, 7], [60, 400], 32, 2, 64, codes=codes)
    q, k, v, *_ = tokens(b, 4, 2, 64)
    before, _ = run(W, b, None, k, v, (None, None), None)
    check(b, before, None, k, v, (None, None), None, None)
    f = W.rope_frequencies(64)
    pos = torch.randint(0, 10 ** 6, (b.T,), device="cuda").to(torch.int32)
    before, qo = run(W, b, q, k, v, (None, None), f, positions=pos, amplitude=1.5)
    check(b, before, q, k, v, (None, None), qo, f, pos=pos, amplitude=1.5)


@pytest.mark.parametrize("codes", [False, True])
def test_positions_without_a_page_and_tokens_of_no_sequence(W, codes):
    """Pages outside the cache, positions beyond the table and below 0, and tokens
    before the first and behind the last sequence."""
    b = batch([6, 20, 3, 4], [6, 40, 90, 2], 16, 2, 64, codes=codes, cols=3)
    b.table[0, 0] = -1
    b.table[1, 1] = b.k.shape[0]
    b.lens[2] = 90                                           # of 48 that the table has
    q, k, v, wq, wk = tokens(b, 4, 2, 64)
    f = W.rope_frequencies(64)
    before, qo = run(W, b, q, k, v, (wq, wk), f)
    check(b, before, q, k, v, (wq, wk), qo, f)
    # two tokens before the first sequence and three behind the last
    pad = lambda x: torch.cat([x[:2], x, x[:3]])  # noqa: E731
    b2 = batch([6, 20, 3, 4], [6, 40, 90, 2], 16, 2, 64, codes=codes, cols=3)
    b2.table.copy_(b.table)
    before = {"k": b2.k.clone(), "v": b2.v.clone()}
    q_out = torch.full((b.T + 5, 4, 64), 7.0, dtype=b.dt, device="cuda")
    W.paged_kv_append(pad(k), pad(v), b2.k, b2.v, b2.table, b2.q_start + 2, b2.kv_len, turns=W.rope_turns(f), q=pad(q), q_weight=wq,
                      k_weight=wk, k_scale=b.k_scale, v_scale=b.v_scale, q_out=q_out)
    check(b2, before, q, k, v, (wq, wk), q_out[2:-3], f)
    assert torch.equal(q_out[2:-3], qo)
    assert (q_out[:2] == 7).all() and (q_out[-3:] == 7).all()


@pytest.mark.parametrize("codes", [False, True])
def test_layouts(W, codes):
    """Head-major pages, K and V of a page side by side, a table with longer rows."""
    b = batch([30, 1], [70, 33], 16, 2, 64, codes=codes)
    pages = b.k.shape[0]
    both = torch.zeros((pages, 2, 2, 16, 64), dtype=b.k.dtype, device="cuda")
    b.k, b.v = (both[:, i].transpose(1, 2) for i in range(2))
    wide = torch.full((2, b.cols + 5), -9, dtype=torch.int32, device="cuda")
    wide[:, :b.cols] = b.table
    b.table = wide[:, :b.cols]
    q, k, v, wq, wk = tokens(b, 4, 2, 64)
    f = W.rope_frequencies(64)
    before, qo = run(W, b, q, k, v, (wq, wk), f)
    check(b, before, q, k, v, (wq, wk), qo, f)


def test_nothing_to_append(W):
    b = batch([0, 0], [5, 6], 16, 2, 64)
    e = torch.empty((0, 2, 64), dtype=b.dt, device="cuda")
    before = b.k.clone()
    assert W.paged_kv_append(e, e, b.k, b.v, b.table, b.q_start, b.kv_len) is None
    none = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    x = torch.ones((3, 2, 64), dtype=b.dt, device="cuda")
    W.paged_kv_append(x, x, b.k, b.v, none, none.flatten()[:0].new_zeros(1), none.flatten())
    torch.cuda.synchronize()
    assert torch.equal(b.k, before)


def test_cells_past_32_bits(W):
    """A cache of more than 2^32 bytes (and 2^31 values): cells of its last page."""
    pages, page, Hk, D = 4097, 4096, 1, 128
    k = torch.zeros((pages, page, Hk, D), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    x = torch.full((1, Hk, D), 3.0, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([page], dtype=torch.int32, device="cuda")
    W.paged_kv_append(x, x, k, k, table, None, lens)
    torch.cuda.synchronize()
    assert (k[-1, -1] == 3).all() and int((k != 0).sum()) == D
