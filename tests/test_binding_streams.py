"""What a call allocates belongs to the stream that runs it: memory of
another stream's pool could be handed to that stream's next tensor while the
call's kernels still use it."""

import pytest
import torch

from fake_cuda import FakeStream, Recorder, fake


@pytest.fixture
def rec(monkeypatch):
    from w8a16_linear_gb300 import binding
    r = Recorder(monkeypatch, binding)
    r.b = binding
    return r


def _attention(b, stream):
    q, k = fake(1, 1, 4, 64), fake(1, 900, 2, 64)
    return b.cross_attention(q, k, k, stream=stream)


def _norm(b, stream):
    return b.add_rms_norm_quant(fake(3, 64), fake(3, 64), fake(64), stream=stream)


def _linear(b, stream):
    u8, f32 = torch.uint8, torch.float32
    return b.fp8_linear_w8a8_pertoken(fake(3, 64, dtype=u8), fake(3, dtype=f32), fake(32, 64, dtype=u8), fake(32, dtype=f32),
                                      stream=stream)


@pytest.mark.parametrize("call,n", [(_attention, 2), (_norm, 3), (_linear, 1)])
def test_allocations_are_made_on_the_calls_stream(rec, call, n):
    st = FakeStream()
    call(rec.b, st)
    assert [s for _, s in rec.allocations] == [st] * n
    assert rec.library.calls[-1][1][-1] == st.cuda_stream
    rec.allocations.clear()
    call(rec.b, None)                                  # the current stream's own pool
    assert [s for _, s in rec.allocations] == [None] * n
    assert rec.library.calls[-1][1][-1] == 0
