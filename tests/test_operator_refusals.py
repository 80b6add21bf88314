"""CPU tests of the arguments that add_rms_norm_quant,
fp8_linear_w8a8_pertoken and cross_attention refuse, before any CUDA call."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from w8a16_linear_gb300 import build as B
    from w8a16_linear_gb300 import binding
    B.build()
    return binding.lib()


P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
NUL = None


def test_add_rms_norm_quant(L):
    def f(x=P, res=P, dtype=0, M=4, K=64, w=P, eps=1e-6, s_in=NUL, s_tok=P, q=P, h=NUL, res_out=P):
        return L.add_rms_norm_quant(x, res, dtype, M, K, w, eps, s_in, s_tok, q, h, res_out, None)

    assert f(dtype=1) == 5 and f(dtype=7) == 5
    assert f(M=-1) == 2 and f(K=12) == 2 and f(K=0) == 2 and f(K=16392) == 2
    for eps in (-1e-6, float("nan"), float("inf")):
        assert f(eps=eps) == 11
    assert f(x=NUL) == 1 and f(w=NUL) == 1
    assert f(q=NUL, s_tok=NUL) == 1                   # no output
    assert f(s_tok=NUL) == 1                          # codes without a scale
    assert f(s_in=P) == 11                            # both scales
    assert f(q=NUL, h=P) == 1                         # a scale without codes
    assert f(res=NUL) == 1                            # a sum without a residual
    for name in ("x", "res", "w", "q", "h", "res_out"):
        assert f(**{name: ODD}) == 3, name
    assert f(s_tok=ctypes.c_void_p(0x10002)) == 3
    assert b"add_rms_norm_quant" in L.w8_last_error()
    assert f(M=0) == 0


def test_fp8_linear_w8a8_pertoken(L):
    def f(x=P, M=4, K=64, s_tok=P, G=2, w=(0x10000,) * 3, N=(32, 48, 16), s=(0x10000,) * 3, y=(0x10000,) * 3):
        arr = lambda v, t: None if v is None else (t * 3)(*v)  # noqa: E731
        return L.fp8_linear_w8a8_pertoken(x, M, K, s_tok, G, arr(w, ctypes.c_void_p), arr(N, ctypes.c_int64),
                                          arr(s, ctypes.c_void_p), arr(y, ctypes.c_void_p), None)

    assert f(G=0) == 2 and f(G=4) == 2
    assert f(w=None) == 1 and f(N=None) == 1 and f(s=None) == 1 and f(y=None) == 1
    assert f(M=-1) == 2 and f(K=24) == 2 and f(N=(32, 24, 16)) == 2 and f(N=(0, 16, 16)) == 2
    assert f(x=NUL) == 1 and f(s_tok=NUL) == 1
    assert f(w=(0x10000, 0, 0)) == 1 and f(s=(0x10000, 0, 0)) == 1 and f(y=(0x10000, 0, 0)) == 1
    assert f(x=ODD) == 3 and f(s=(0x10000, 0x10004, 0x10000)) == 3 and f(s_tok=ctypes.c_void_p(0x10001)) == 3
    assert f(M=0) == 0


def desc(**kw):
    from w8a16_linear_gb300 import binding as b
    d = dict(B=2, Lq=3, Lk=5, Hq=4, Hkv=2, D=64, qs=(768, 256, 64), ks=(640, 128, 64), vs=(640, 128, 64),
             os=(768, 256, 64), ms=5, dtype=0, scale=0.125)
    d.update(kw)
    t = ctypes.c_int64 * 3
    return b.AttentionDesc(d["B"], d["Lq"], d["Lk"], d["Hq"], d["Hkv"], d["D"], t(*d["qs"]), t(*d["ks"]), t(*d["vs"]),
                           t(*d["os"]), d["ms"], d["dtype"], d["scale"])


def test_cross_attention(L):
    def f(q=P, k=P, v=P, lens=NUL, mask=NUL, s_out=NUL, out=P, ws=NUL, n=0, **kw):
        return L.cross_attention(ctypes.byref(desc(**kw)), q, k, v, lens, mask, s_out, out, ws, n, None)

    assert L.cross_attention(None, P, P, P, NUL, NUL, NUL, P, NUL, 0, None) == 1
    assert f(dtype=1) == 5
    for bad in (dict(B=-1), dict(Lq=-1), dict(Lk=-1), dict(D=4), dict(D=136), dict(D=68), dict(Hq=3), dict(Hkv=0),
                dict(Hq=0), dict(Hq=258), dict(B=1 << 20, Lq=1 << 20),
                dict(Lk=(1 << 26) + 1)):
        assert f(**bad) == 2, bad
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert f(scale=scale) == 11
    assert f(qs=(768, 252, 64)) == 4                   # rows not 16-byte aligned
    assert f(ks=(640, 0, 64)) == 4 and f(vs=(640, 128, -64)) == 4 and f(os=(0, 256, 64)) == 4
    assert f(ms=-1) == 4
    assert f(k=P, out=NUL) == 1 and f(q=NUL) == 1
    assert f(out=ODD) == 3 and f(lens=ctypes.c_void_p(0x10002)) == 3
    assert b"cross_attention" in L.w8_last_error()
    # nothing to do: nothing is launched, and nothing but the descriptor is read
    assert f(B=0, q=NUL) == 0 and f(Lq=0, out=NUL) == 0
    n = ctypes.c_int64(-1)
    assert L.cross_attention_workspace(ctypes.byref(desc(Lq=0)), ctypes.byref(n)) == 0 and n.value == 0
    assert L.cross_attention_workspace(ctypes.byref(desc()), None) == 1


def test_the_binding_refuses_what_the_library_cannot_see(L):
    from w8a16_linear_gb300 import binding as b
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(b.W8Error) as e:
        b.add_rms_norm_quant(x, None, x[0])           # not on the device
    assert e.value.status == 1
    with pytest.raises(b.W8Error) as e:
        b.add_rms_norm_quant(x.float(), None, x[0])
    assert e.value.status in (1, 5)
    with pytest.raises(b.W8Error) as e:
        b.fp8_linear_w8a8_pertoken(x, None, None, None)
    assert e.value.status in (1, 5)
    q = torch.zeros((1, 2, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(b.W8Error) as e:
        b.cross_attention(q, q, q)
    assert e.value.status == 1
    with pytest.raises(b.W8Error) as e:
        b.cross_attention(q.float(), q, q)
    assert e.value.status == 5
