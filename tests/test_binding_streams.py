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


def _scale():
    return fake(1, dtype=torch.float32)


def _w8a8(b, stream):
    return b.fp8_linear_w8a8(fake(3, 64), fake(32, 64, dtype=torch.uint8), _scale(), _scale(), out=fake(3, 32), stream=stream)


def _group(b, stream):
    w = fake(32, 64, dtype=torch.uint8)
    return b.qkv_shared_quant_gemm(b.MODE_A8, fake(3, 64), _scale(), [w, w], [_scale(), _scale()], outs=[fake(3, 32), fake(3, 32)],
                                   stream=stream)


def _gate_up(b, stream):
    w, s = fake(32, 64, dtype=torch.uint8), _scale()
    return b.gate_up_swiglu_fp8(fake(3, 64), s, w, w, s, s, s, out=fake(3, 32, dtype=torch.uint8), stream=stream)


@pytest.mark.parametrize("call", [_w8a8, _group, _gate_up])
def test_temporary_codes_are_allocated_on_the_calls_stream(rec, call):
    st = FakeStream()
    call(rec.b, st)
    assert rec.allocations == [((3, 64), st)]
    rec.allocations.clear()
    call(rec.b, None)
    assert rec.allocations == [((3, 64), None)]
