"""GPU parity of paged_attention against the formula in 64 bits.

The bound on the error is cross_attention's: with the weights P_j (sum 1) and
A = sum_j P_j |v_j|,
    |o^ - o| <= A E + h (|o| + A E),
    E = h + 2 (2 D 2^-24 scale max sum|q k| + 2^-22 max|s log2 e| + 2^-22) + 4 (x + 64) 2^-24
for x positions and h = half a step of the 16-bit type, and for f16, whose P is subnormal below 2^-14,
another x 2^-25 max|v|.  E4M3 cells are exact in 16 bits; their scales are one more rounding of the score's factor
and of the output's, which the 64 in E covers.  Beside them P is binary16, which is
off by 2^-25 below 2^-14 where the row's largest weight is 1 or more, or three E4M3 terms t0 + t1 / 16 +
t2 / 256: each rounds what the one before leaves, by 2^-4 of it or by half of
the smallest step, 2^-10, so that 2^-12 of a weight (less than h) or 2^-10 / 256 = 2^-18 is left, where the
row's largest weight is 2^6 or more.  Either is within 2^-24 of the largest weight, for
x positions x 2^-24 max|v|.
"""

import pytest
import torch

from gpu_util import W, dev_f32  # noqa: F401
from paged_util import DT, batch, code_near, exact_attention

pytestmark = pytest.mark.gpu


def queries(b, H, D, seed=3, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((b.T, H, D), generator=g, device="cuda") * std).to(b.dt)


def call(W, b, q, **kw):
    o = W.paged_attention(q, b.k, b.v, b.table, kw.pop("q_start", b.q_start), b.kv_len, k_scale=b.k_scale, v_scale=b.v_scale, **kw)
    torch.cuda.synchronize()
    W.poll_device_error()
    return o


def check(got, o, err, written, s_out=None):
    if s_out is not None:
        assert code_near(got[written], o[written] / float(s_out), err[written] / float(s_out))
        return
    bad = ~((got.double() - o).abs() <= err) & ~(torch.isnan(o) & torch.isnan(got))
    bad &= written[:, None, None]
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((got.double() - o).abs().nan_to_num(0.0).max()))


SHAPES = [  # new tokens, positions, page, query and key heads, D
    ([1], [1], 16, 1, 1, 64), ([1], [512], 16, 32, 8, 128), ([1], [513], 8, 4, 4, 128), ([1, 1, 1], [700, 1, 129], 16, 8, 2, 128),
    ([1], [5003], 64, 8, 1, 64), ([3], [129], 32, 5, 1, 80), ([128], [128], 128, 2, 2, 128), ([129], [129], 48, 2, 2, 64),
    ([256], [640], 16, 3, 3, 128), ([257], [1000], 256, 2, 1, 96), ([100, 30], [300, 30], 32, 14, 2, 128),
    ([385], [385], 16, 3, 3, 32), ([77, 5, 0, 40], [999, 5, 30, 700], 48, 20, 4, 64), ([1000], [1002], 64, 6, 2, 16),
    ([1], [300], 16, 128, 1, 128), ([2], [300], 24, 100, 1, 128), ([640, 1, 333, 2], [640, 900, 333, 333], 40, 2, 2, 48),
    ([20], [12000], 16, 16, 2, 128), ([5] * 7, [4133, 2000, 5, 6, 333, 1024, 4096], 48, 20, 4, 64), ([300] * 3, [300, 428, 3000], 32, 8, 1, 128)]


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new,lens,page,H,Hk,D", SHAPES)
def test_shapes(W, new, lens, page, H, Hk, D, dtype, codes):
    b = batch(new, lens, page, Hk, D, dtype, codes, seed=sum(lens))
    q = queries(b, H, D)
    for causal in (True, False):
        check(call(W, b, q, causal=causal, max_q=max(new)), *exact_attention(b, q, causal))


@pytest.mark.parametrize("D", [8, 24, 56, 72, 104, 120])
def test_heads_of_odd_sizes(W, D):
    b = batch([3, 200], [300, 260], 16, 2, D)
    q = queries(b, 6, D)
    check(call(W, b, q), *exact_attention(b, q))


@pytest.mark.parametrize("new,lens,H,Hk,D", [([1, 1, 1, 1], [600, 129, 1, 128], 4, 2, 128), ([300, 5, 130], [600, 5, 131], 2, 2, 64),
                                             ([2, 2], [3000, 66], 4, 1, 80), ([520], [900], 8, 2, 128)])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("kind", ["nan", "inf", "big"])
def test_anything_in_cells_behind_the_positions(W, new, lens, H, Hk, D, codes, kind):
    fill = {"nan": 0x7F, "inf": 0xFF, "big": 0x7E}[kind] if codes else {"nan": float("nan"), "inf": -float("inf"), "big": 3e38}[kind]
    b = batch(new, lens, 16, Hk, D, codes=codes, fill=fill)
    q = queries(b, H, D)
    for causal in (True, False):
        check(call(W, b, q, causal=causal), *exact_attention(b, q, causal))


@pytest.mark.parametrize("new,lens,H,Hk,D", [([300], [300], 2, 2, 64), ([40, 300], [333, 700], 8, 2, 128), ([3], [200], 4, 1, 128),
                                             ([1100], [1200], 1, 1, 96)])
@pytest.mark.parametrize("codes", [False, True])
def test_values_that_are_not_finite_reach_the_rows_that_see_them_alone(W, new, lens, H, Hk, D, codes):
    """NaN and infinities in K and V of new tokens: rows before them are as without."""
    b = batch(new, lens, 16, Hk, D, codes=codes)
    nan, inf = (0x7F, 0xFF) if codes else (float("nan"), float("inf"))
    for i, (n, x) in enumerate(zip(new, lens)):
        for p, c, d, value in ((x - 1, b.v, 3, nan), (x - n + n // 2, b.v, D - 1, inf), (x - n + 2 * n // 3, b.v, 7, inf),
                               (x - max(n // 4, 1), b.k, 5, nan)):
            c[b.table[i, p // 16].long(), p % 16, 0, d] = value
    q = queries(b, H, D)
    o, err, written = exact_attention(b, q)
    got = call(W, b, q)
    # a row that sees the NaN key is NaN everywhere
    t = 0
    for n in new:
        G = H // Hk
        o[t + n - max(n // 4, 1):t + n, :G] = float("nan")
        t += n
    finite = torch.isfinite(o)
    assert (got[~finite].double().isnan() | got[~finite].double().isinf()).all()
    check(got, o, err, finite.all(-1).all(-1) & written)
    bad = ~((got.double() - o).abs() <= err) & finite
    assert not bad.any(), bad.nonzero()[:4].tolist()


def test_rows_that_see_nothing(W):
    """Lengths of 0, below 0 and below the number of new tokens."""
    b = batch([4, 2, 300, 3], [2, 0, 10, 3], 16, 2, 64)
    b.kv_len[1], b.lens[1] = -7, -7
    q = queries(b, 4, 64)
    o, err, written = exact_attention(b, q)
    got = call(W, b, q)
    check(got, o, err, written)
    assert not got[:2].any() and not got[4:6].any() and not got[6:296].any()
    out = torch.full_like(q, 5.0)
    call(W, b, q, causal=False, out=out)
    assert not out[4:6].any()
    check(out, *exact_attention(b, q, False))


def test_rows_of_no_sequence_and_beyond_max_q_are_left_alone(W):
    b = batch([6, 300, 3], [60, 400, 90], 16, 2, 64)
    q = queries(b, 4, 64)
    o, err, written = exact_attention(b, q, max_q=100)
    out = torch.full_like(q, 5.0)
    call(W, b, q, max_q=100, out=out)
    check(out, o, err, written)
    assert (out[~written] == 5).all()
    pad = torch.cat([q[:2], q, q[:3]])
    out = torch.full_like(pad, 5.0)
    call(W, b, pad, q_start=b.q_start + 2, out=out)
    check(out[2:-3], *exact_attention(b, q))
    assert (out[:2] == 5).all() and (out[-3:] == 5).all()


def test_pages_that_are_none_and_positions_beyond_the_table(W):
    b = batch([3, 200, 2], [100, 260, 90], 16, 2, 64, cols=17)
    b.table[0, 2], b.table[1, 16], b.table[1, 3] = -1, b.k.shape[0], 2 ** 31 - 1
    b.kv_len[2], b.lens[2] = 17 * 16 + 50, 17 * 16 + 50      # 272 of 322 exist
    q = queries(b, 4, 64)
    for causal in (True, False):
        check(call(W, b, q, causal=causal), *exact_attention(b, q, causal))


@pytest.mark.parametrize("new", [1, 20, 200])
def test_a_table_without_columns(W, new):
    b = batch([new, 2], [50, 60], 16, 2, 64)
    b.table, b.cols = b.table[:, :0].contiguous(), 0
    q = queries(b, 4, 64)
    out = torch.full_like(q, 5.0)
    call(W, b, q, out=out)
    assert not out.any()


def test_uniform_batches_without_starts_and_shared_pages(W):
    b = batch([2] * 6, [300, 300, 40, 300, 2, 299], 16, 2, 128)
    b.table[1], b.table[3, :10] = b.table[0], b.table[0, :10]   # a prompt in common
    q = queries(b, 8, 128)
    check(call(W, b, q, q_start=None, max_q=2), *exact_attention(b, q))


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("new,lens", [([300], [700]), ([1, 1], [900, 33])])
def test_layouts(W, new, lens, codes):
    """Head-major pages with K and V side by side, strided q and out, a table with longer rows."""
    b = batch(new, lens, 32, 2, 64, codes=codes)
    both = torch.stack([b.k.transpose(1, 2), b.v.transpose(1, 2)], 1)
    b.k, b.v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    wide = torch.full((b.B, b.cols + 5), -9, dtype=torch.int32, device="cuda")
    wide[:, :b.cols] = b.table
    b.table = wide[:, :b.cols]
    big = torch.randn((b.T, 10, 72), device="cuda").to(b.dt)
    q = big[:, 1:9, :64]
    out = torch.full((8, b.T, 72), 9.0, dtype=b.dt, device="cuda").transpose(0, 1)
    call(W, b, q, out=out[..., :64])
    check(out[..., :64], *exact_attention(b, q))
    assert (out[..., 64:] == 9).all()


@pytest.mark.parametrize("new,lens", [([300, 7], [300, 900]), ([1] * 3, [2000, 50, 1])])
@pytest.mark.parametrize("codes", [False, True])
def test_codes_out(W, new, lens, codes):
    for H, Hk, D in ((8, 2, 128), (6, 2, 80), (4, 4, 64)):
        b = batch(new, lens, 16, Hk, D, codes=codes)
        q, s_out = queries(b, H, D), dev_f32(2.0 / 448)
        got = call(W, b, q, s_out=s_out)
        assert got.dtype == torch.uint8
        check(got, *exact_attention(b, q), s_out=s_out)


@pytest.mark.parametrize("new,lens", [([300], [700]), ([1], [3000])])
def test_scores_far_apart(W, new, lens):
    """Scores of some +-1000, and rows whose maximum comes last."""
    b = batch(new, lens, 16, 2, 64, std=4.0)
    q = queries(b, 4, 64, std=8.0)
    b.k.mul_(torch.linspace(0.1, 4.0, b.k.shape[0], device="cuda").to(b.dt)[:, None, None, None])
    check(call(W, b, q, scale=0.5), *exact_attention(b, q, scale=0.5))


def test_a_nan_query_spoils_its_own_row_only(W):
    b = batch([70, 1], [200, 90], 16, 2, 64)
    q = queries(b, 4, 64)
    want = call(W, b, q)
    q[11, 1, 3] = float("nan")
    got = call(W, b, q)
    assert torch.isnan(got[11, 1]).all()
    got[11, 1] = want[11, 1]
    o, err, written = exact_attention(b, q.nan_to_num(0.0))
    o[11, 1] = want[11, 1].double()
    check(got, o, err, written)


@pytest.mark.parametrize("new,lens,H,Hk,D", [([1] * 8, [9000] * 8, 8, 2, 128), ([1] * 100, [600] * 99 + [6000], 2, 1, 64),
                                             ([1] * 600, [300] * 600, 2, 2, 64), ([30] * 3, [5000, 100, 7000], 4, 1, 128),
                                             ([700, 5], [9000, 5], 4, 1, 128)])
def test_nothing_is_written_behind_the_workspace(W, new, lens, H, Hk, D):
    b = batch(new, lens, 64, Hk, D)
    q = queries(b, H, D)
    ws = W.paged_attention_workspace(q, b.k, b.table, max_q=max(new))
    room = torch.full((ws.numel() + 4096,), 3.0, device="cuda")
    got = call(W, b, q, max_q=max(new), ws=room[:ws.numel()])
    assert (room[ws.numel():] == 3).all()
    check(got, *exact_attention(b, q))
    if ws.numel():
        with pytest.raises(W.W8Error) as e:
            W.paged_attention(q, b.k, b.v, b.table, b.q_start, b.kv_len, max_q=max(new), ws=room[:ws.numel() - 1])
        assert e.value.status == 2


@pytest.mark.parametrize("B", [256, 257, 300])
@pytest.mark.parametrize("most,H,Hk,D", [(1, 8, 2, 64), (3, 10, 1, 64), (40, 10, 2, 128), (300, 2, 2, 64)])
@pytest.mark.parametrize("codes", [False, True])
def test_many_sequences_of_all_lengths(W, B, most, H, Hk, D, codes):
    """About as many as are kept in shared memory: some without a token, some without a past."""
    new = [most * (7 * i % 11) // 10 for i in range(B)]
    lens = [n + (37 * i % 101) * (i % 3) for i, n in enumerate(new)]
    b = batch(new, lens, 16, Hk, D, codes=codes)
    q = queries(b, H, D)
    for causal in (True, False):
        check(call(W, b, q, causal=causal, max_q=most), *exact_attention(b, q, causal))


@pytest.mark.parametrize("new,lens", [([1] * 4, [3000, 50, 2000, 1]), ([300, 40], [3000, 100])])
@pytest.mark.parametrize("codes", [False, True])
def test_equal_calls_give_equal_bits(W, new, lens, codes):
    """Again, after other work, on another stream, and replayed in a graph with
    the lengths of another step."""
    b = batch(new, lens, 16, 2, 128, codes=codes)
    q = queries(b, 8, 128)
    kw = dict(k_scale=b.k_scale, v_scale=b.v_scale, max_q=max(new))
    want = call(W, b, q, max_q=max(new)).clone()
    other = batch([64], [2500], 32, 2, 64)
    call(W, other, queries(other, 4, 64, std=30.0))
    assert torch.equal(call(W, b, q, max_q=max(new)), want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = W.paged_attention(q, b.k, b.v, b.table, b.q_start, b.kv_len, stream=st, **kw)
    st.synchronize()
    assert torch.equal(got, want)
    ws = W.paged_attention_workspace(q, b.k, b.table, max_q=max(new))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W.paged_attention(q, b.k, b.v, b.table, b.q_start, b.kv_len, out=got, ws=ws, **kw)
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    b.lens = [max(n, x // 2) for n, x in zip(b.new, b.lens)]
    b.kv_len.copy_(torch.tensor(b.lens, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    check(got, *exact_attention(b, q))


@pytest.mark.parametrize("D,dtype,codes", [(128, "bf16", False), (64, "f16", False), (128, "bf16", True)])
def test_long_contexts_of_few_queries_back_to_back(W, D, dtype, codes):
    b = batch([1, 2, 1], [20670, 16000, 12345], 64, 2, D, dtype, codes)
    q = queries(b, 8, D)
    outs = [W.paged_attention(q, b.k, b.v, b.table, b.q_start, b.kv_len, k_scale=b.k_scale, v_scale=b.v_scale) for _ in range(20)]
    torch.cuda.synchronize()
    W.poll_device_error()
    assert all(torch.equal(o, outs[0]) for o in outs)
    check(outs[0], *exact_attention(b, q))


def test_cells_past_32_bits(W):
    """A cache of more than 2^32 bytes (and 2^31 values): the last pages."""
    pages, page, D = 4100, 4096, 128
    k = torch.zeros((pages, page, 1, D), dtype=torch.bfloat16, device="cuda")
    k[-2:] = torch.randn((2, page, 1, D), device="cuda").bfloat16()
    b = batch([3], [5000], page, 1, D)
    b.k = b.v = k
    b.table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    q = queries(b, 4, D)
    check(call(W, b, q), *exact_attention(b, q))


def test_nothing_to_do(W):
    b = batch([0, 0], [5, 6], 16, 2, 64)
    q = torch.empty((0, 4, 64), dtype=b.dt, device="cuda")
    assert call(W, b, q).shape == (0, 4, 64)
    q = queries(batch([3], [3], 16, 2, 64), 4, 64)
    none = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 5.0)
    W.paged_attention(q, b.k, b.v, none, none.new_zeros(1), none.flatten(), out=out)
    torch.cuda.synchronize()
    assert (out == 5).all()
    assert DT["bf16"] == q.dtype


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("lens", [[1280], [1281], [1408], [1409], [1792], [1793], [1920], [1921], [1281] * 3, [1793, 1, 1281, 0, 2049]])
def test_single_tokens_around_the_lengths_at_which_units_are_cut(W, lens, codes):
    b = batch([min(x, 1) for x in lens], lens, 16, 2, 128, codes=codes)
    q = queries(b, 8, 128)
    check(call(W, b, q, max_q=1), *exact_attention(b, q))
