"""qk_norm_rope, paged_kv_append and paged_attention from several host threads at once (their
marshalling lets the interpreter go), as a thread's first CUDA call, and on a stream given to
the call with outputs and workspace of its own: the serial calls' bits."""

import threading

import pytest
import torch

from gpu_util import W, dev_f32  # noqa: F401
from paged_util import batch
from test_gpu_paged_attention import queries

pytestmark = pytest.mark.gpu


def normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def rope_case(W, M, D, interleaved):
    g = torch.Generator(device="cuda").manual_seed(M)
    q, k, w = normal(g, M, 6, D), normal(g, M, 2, D), normal(g, D)
    pos = torch.arange(M, device="cuda", dtype=torch.int32) * 31
    turns = W.rope_turns(W.rope_frequencies(D))

    def call(outs, **kw):
        W.qk_norm_rope(q, k, pos, turns, q_weight=w, k_weight=w, interleaved=interleaved, q_out=outs[0], k_out=outs[1], **kw)

    return call, lambda: [torch.zeros_like(q), torch.zeros_like(k)]


def append_case(W, new, lens, codes):
    b = batch(new, lens, 16, 2, 64, codes=codes)
    g = torch.Generator(device="cuda").manual_seed(len(new))
    k, v, q, w = normal(g, b.T, 2, 64), normal(g, b.T, 2, 64), normal(g, b.T, 8, 64), normal(g, 64)
    turns = W.rope_turns(W.rope_frequencies(64))

    def call(outs, **kw):
        W.paged_kv_append(k, v, outs[0], outs[1], b.table, b.q_start, b.kv_len, turns=turns, q=q, q_weight=w, k_weight=w,
                          k_scale=b.k_scale, v_scale=b.v_scale, q_out=outs[2], **kw)

    return call, lambda: [b.k.clone(), b.v.clone(), torch.zeros_like(q)]


def attention_case(W, new, lens, H, Hk, D, codes=False, s_out=None):
    b = batch(new, lens, 16, Hk, D, codes=codes)
    q = queries(b, H, D)
    kw = dict(max_q=max(new), k_scale=b.k_scale, v_scale=b.v_scale, s_out=s_out)
    ws = W.paged_attention_workspace(q, b.k, b.table, max_q=max(new))

    def call(outs, **more):
        W.paged_attention(q, b.k, b.v, b.table, b.q_start, b.kv_len, out=outs[0], ws=outs[1], **kw, **more)

    return call, lambda: [torch.zeros(q.shape, dtype=q.dtype if s_out is None else torch.uint8, device="cuda"), torch.empty_like(ws)]


def cases(W):
    return [rope_case(W, 700, 128, False), rope_case(W, 3, 64, True), append_case(W, [1] * 6, [90, 3, 4, 200, 17, 1], True),
            append_case(W, [300, 40], [300, 90], False), attention_case(W, [1], [3000], 8, 2, 128),
            attention_case(W, [1, 2], [2000, 90], 8, 2, 64, codes=True), attention_case(W, [30], [3000], 4, 1, 128, codes=True),
            attention_case(W, [300, 200], [700, 2500], 4, 2, 128, s_out=dev_f32(2.0 / 448))]


def same(got, want):
    """The outputs' bits (a workspace is last where there is one, and means nothing)."""
    n = 1 if len(got) == 2 and got[1].dtype == torch.float32 else len(got)
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got[:n], want[:n]))


def test_all_at_once(W):
    todo = []
    for call, make in cases(W):
        want, got = make(), make()
        call(want)
        todo.append((call, want, got))
    torch.cuda.synchronize()
    failures, start = [], threading.Barrier(len(todo))

    def work(i):
        call, want, got = todo[i]
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                start.wait()
                for _ in range(500):
                    call(got)
            stream.synchronize()
            if not same(got, want):
                failures.append((i, "bits"))
        except Exception as e:   # shown by the assertion below
            failures.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(todo))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    W.poll_device_error()
    assert not failures, failures


@pytest.mark.parametrize("marshalled", [True, False])
@pytest.mark.parametrize("which", range(8))
def test_first_call_of_a_thread(W, monkeypatch, which, marshalled):
    from w8a16_linear_gb300 import binding
    call, make = cases(W)[which]
    want, got = make(), make()
    call(want)
    torch.cuda.synchronize()
    errors = []
    if not marshalled:
        monkeypatch.setattr(binding, "_marshal", None)

    def work():
        try:
            call(got)
        except Exception as e:   # shown by the assertion below
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    W.poll_device_error()
    assert not errors, errors
    assert same(got, want)


@pytest.mark.parametrize("which", range(8))
def test_on_a_stream_given_to_the_call(W, which):
    call, make = cases(W)[which]
    want, got = make(), make()
    call(want)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    call(got, stream=stream)
    stream.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("new,lens,codes", [([1], [9000], False), ([1], [9000], True), ([40], [9000], False), ([300], [9000], False)])
def test_outputs_and_workspace_of_the_calls_own_on_its_stream(W, new, lens, codes):
    """What the call allocates belongs to its stream: tensors of the same sizes that the current
    stream goes on to make and fill are others."""
    b = batch(new, lens, 16, 2, 128, codes=codes)
    q = queries(b, 4, 128)
    args = (q, b.k, b.v, b.table, b.q_start, b.kv_len)
    kw = dict(max_q=max(new), k_scale=b.k_scale, v_scale=b.v_scale)
    want = W.paged_attention(*args, **kw)
    n = W.paged_attention_workspace(q, b.k, b.table, max_q=max(new)).numel()
    assert n > 0
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for _ in range(20):
        got = W.paged_attention(*args, stream=stream, **kw)
        others = [torch.full((n,), float(i), device="cuda") for i in range(4)]
        outs = [torch.full_like(q, 3.0) for _ in range(4)]
        torch.cuda.synchronize()
        W.poll_device_error()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        assert all(bool((t == float(i)).all()) for i, t in enumerate(others)) and all(bool((t == 3).all()) for t in outs)
