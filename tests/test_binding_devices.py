"""The operators of a cross-attention site refuse tensors of another device
than the one that the call launches on: the kernels would read addresses of
another GPU."""

import pytest
import torch

from fake_cuda import FakeCuda, FakeLibrary


class On(FakeCuda):
    """A host tensor that names a CUDA device as its own."""
    index = 0

    @property
    def device(self):
        return torch.device("cuda", self.index)


class Elsewhere(On):
    index = 1


def on(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(On)


@pytest.fixture
def b(monkeypatch):
    from w8a16_linear_gb300 import binding
    library = FakeLibrary(0)
    monkeypatch.setattr(binding, "lib", lambda: library)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    binding.recorded = library.calls
    yield binding
    del binding.recorded


U8, F32 = torch.uint8, torch.float32


def norm_args():
    return dict(x=on(3, 64), residual=on(3, 64), weight=on(64), out=on(3, 64, dtype=U8), s_tok=on(3, dtype=F32),
                res_out=on(3, 64), h_out=on(3, 64))


def static_args():
    return dict(norm_args(), s_tok=None, s_in=on(1, dtype=F32))


def linear_args():
    return dict(qx=on(3, 64, dtype=U8), s_tok=on(3, dtype=F32), w=on(32, 64, dtype=U8), s_ch=on(32, dtype=F32), out=on(3, 32))


def attention_args():
    return dict(q=on(2, 1, 4, 64), k=on(2, 9, 2, 64), v=on(2, 9, 2, 64), kv_len=on(2, dtype=torch.int32),
                kv_mask=on(2, 9, dtype=torch.bool), s_out=on(1, dtype=F32), out=on(2, 1, 4, 64, dtype=U8), ws=on(64, dtype=F32))


CALLS = [("add_rms_norm_quant", norm_args), ("add_rms_norm_quant", static_args), ("fp8_linear_w8a8_pertoken", linear_args),
         ("cross_attention", attention_args)]


@pytest.mark.parametrize("name,args", CALLS)
def test_one_tensor_elsewhere(b, name, args):
    getattr(b, name)(**args())
    assert b.recorded[-1][1][-1] == 100            # the current device's stream
    for key, t in args().items():
        if t is None:
            continue
        n = len(b.recorded)
        with pytest.raises(b.W8Error) as e:
            getattr(b, name)(**dict(args(), **{key: t.as_subclass(Elsewhere)}))
        assert e.value.status == 1, key
        assert all(c[0] != name for c in b.recorded[n:]), key


@pytest.mark.parametrize("name,args", CALLS)
def test_all_tensors_elsewhere(b, name, args):
    """The library launches on the current device, whatever the tensors'."""
    with pytest.raises(b.W8Error) as e:
        getattr(b, name)(**{k: t if t is None else t.as_subclass(Elsewhere) for k, t in args().items()})
    assert e.value.status == 1


def test_a_stream_of_another_device(b):
    class Stream:
        cuda_stream, device = 7, torch.device("cuda", 1)

    with pytest.raises(b.W8Error) as e:
        b.add_rms_norm_quant(**norm_args(), stream=Stream())
    assert e.value.status == 1
    Stream.device = torch.device("cuda", 0)
    b.add_rms_norm_quant(**norm_args(), stream=Stream())
    assert b.recorded[-1][1][-1] == 7
