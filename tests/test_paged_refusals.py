"""CPU tests of what qk_norm_rope, paged_kv_append and paged_attention refuse,
before any CUDA call, and of the frequencies that are made on the host."""

import ctypes
import math
from fractions import Fraction

import pytest
import torch

from fake_cuda import FakeLibrary, fake
from test_binding_devices import Elsewhere, on


@pytest.fixture(scope="module")
def L():
    from w8a16_linear_gb300 import build as B
    from w8a16_linear_gb300 import binding
    B.build()
    return binding.lib()


P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
NUL = None
I2, I3 = ctypes.c_int64 * 2, ctypes.c_int64 * 3


def rope(**kw):
    from w8a16_linear_gb300 import binding as b
    d = dict(M=4, Hq=4, Hkv=2, D=64, qs=(512, 64), ks=(512, 64), vs=(512, 64), qos=(256, 64), kos=(128, 64), pitch=4, dtype=0,
             rot=64, inter=0, axes=1, pairs=(32, 0, 0), eps=1e-6, amplitude=1.0)
    d.update(kw)
    return b.RopeDesc(d["M"], d["Hq"], d["Hkv"], d["D"], I2(*d["qs"]), I2(*d["ks"]), I2(*d["vs"]), I2(*d["qos"]), I2(*d["kos"]),
                      d["pitch"], d["dtype"], d["rot"], d["inter"], d["axes"], (ctypes.c_int32 * 3)(*d["pairs"]), d["eps"],
                      d["amplitude"])


def cache(**kw):
    from w8a16_linear_gb300 import binding as b
    d = dict(B=2, pages=9, page=16, cols=4, table_stride=4, Hkv=2, D=64, cks=(2048, 128, 64), cvs=(2048, 128, 64), cells=0)
    d.update(kw)
    return b.PagedDesc(d["B"], d["pages"], d["page"], d["cols"], d["table_stride"], d["Hkv"], d["D"], I3(*d["cks"]), I3(*d["cvs"]),
                       d["cells"])


ROPE_BAD = [(dict(dtype=1), 5), (dict(M=-1), 2), (dict(Hq=-1), 2), (dict(Hkv=-1), 2), (dict(D=4), 2), (dict(D=264), 2),
            (dict(D=68), 2), (dict(rot=-16), 2), (dict(rot=24, pairs=(12, 0, 0)), 2), (dict(rot=80, pairs=(40, 0, 0)), 2),
            (dict(axes=0), 2), (dict(axes=4), 2), (dict(pairs=(31, 0, 0)), 2), (dict(axes=2, pairs=(40, -8, 0)), 2),
            (dict(axes=2, pairs=(16, 16, 0), pitch=0), 4), (dict(eps=-1.0), 11), (dict(eps=float("nan")), 11),
            (dict(amplitude=0.0), 11), (dict(amplitude=float("inf")), 11), (dict(qs=(508, 64)), 4), (dict(qs=(512, 0)), 4),
            (dict(ks=(-512, 64)), 4), (dict(qos=(256, 60)), 4)]


def test_qk_norm_rope(L):
    def f(q=P, k=P, pos=P, turns=P, wq=P, wk=P, qo=P, ko=P, **kw):
        return L.qk_norm_rope(ctypes.byref(rope(**kw)), q, k, pos, turns, wq, wk, qo, ko, None)

    assert L.qk_norm_rope(None, P, P, P, P, P, P, P, P, None) == 1
    for kw, status in ROPE_BAD + [(dict(Hq=0, Hkv=0), 2), (dict(kos=(0, 64)), 4)]:
        assert f(**kw) == status, kw
    assert f(rot=0, pairs=(0, 0, 0), wq=NUL, wk=NUL) == 11   # nothing to do
    for name in ("q", "k", "qo", "ko", "pos", "turns"):
        assert f(**{name: NUL}) == 1, name
    for name in ("q", "k", "qo", "ko", "wq", "wk"):
        assert f(**{name: ODD}) == 3, name
    assert f(pos=ctypes.c_void_p(0x10002)) == 3 and f(turns=ctypes.c_void_p(0x10004)) == 3
    assert b"qk_norm_rope" in L.w8_last_error()
    assert f(M=0, q=NUL) == 0


CACHE_BAD = [(dict(B=-1), 2), (dict(B=(1 << 20) + 1), 2), (dict(pages=0), 2), (dict(pages=1 << 31), 2), (dict(page=0), 2), (dict(page=12), 2),
             (dict(page=1 << 21), 2), (dict(cols=-1), 2), (dict(cols=1 << 23), 2), (dict(table_stride=-1), 4),
             (dict(cks=(2048, 124, 64)), 4), (dict(cvs=(0, 128, 64)), 4), (dict(cells=2), 5), (dict(cells=7), 5),
             (dict(cells=1, cks=(2056, 128, 64)), 4)]


def test_paged_kv_append(L):
    def f(q=P, k=P, v=P, pos=NUL, turns=P, wq=P, wk=P, kc=P, vc=P, table=P, start=P, lens=P, k_scale=NUL, v_scale=NUL, qo=P,
          c=(), **kw):
        ours = {x: y for x, y in kw.items() if x in ("B", "pages", "page", "cols", "table_stride", "cks", "cvs", "cells")}
        return L.paged_kv_append(ctypes.byref(rope(**kw)), ctypes.byref(cache(**ours, **dict(c))), q, k, v, pos, turns, wq, wk, kc,
                                 vc, table, start, lens, k_scale, v_scale, qo, None)

    assert L.paged_kv_append(None, ctypes.byref(cache()), *[P] * 15, None) == 1
    assert L.paged_kv_append(ctypes.byref(rope()), None, *[P] * 15, None) == 1
    for kw, status in ROPE_BAD + CACHE_BAD + [(dict(Hkv=0), 2), (dict(vs=(508, 64)), 4), (dict(c=dict(Hkv=3)), 2),
                                               (dict(c=dict(D=32)), 2)]:
        assert f(**kw) == status, kw
    for name in ("q", "k", "v", "turns", "kc", "vc", "table", "lens", "qo"):
        assert f(**{name: NUL}) == 1, name
    for name in ("q", "k", "v", "kc", "vc", "qo", "wk"):
        assert f(**{name: ODD}) == 3, name
    for name in ("table", "start", "lens"):
        assert f(**{name: ctypes.c_void_p(0x10002)}) == 3, name
    assert f(start=NUL, M=5) == 2                            # 5 tokens of 2 sequences
    assert f(k_scale=P, v_scale=P) == 11                     # scales of 16-bit cells
    assert f(cells=1) == 1 and f(k_scale=P, cells=1) == 1    # codes without both
    assert f(axes=2, pairs=(16, 16, 0)) == 2                 # axes without positions
    assert b"paged_kv_append" in L.w8_last_error()
    assert f(M=0, k=NUL) == 0 and f(B=0, k=NUL) == 0


def attention(**kw):
    from w8a16_linear_gb300 import binding as b
    d = dict(T=4, Hq=4, max_q=4, qs=(256, 64), os=(256, 64), dtype=0, causal=1, scale=0.125)
    d.update(kw)
    return b.PagedAttentionDesc(d["T"], d["Hq"], d["max_q"], I2(*d["qs"]), I2(*d["os"]), d["dtype"], d["causal"], d["scale"])


def test_paged_attention(L):
    own = ("T", "Hq", "max_q", "qs", "os", "dtype", "causal", "scale")

    def descs(kw):
        return (ctypes.byref(attention(**{k: v for k, v in kw.items() if k in own})),
                ctypes.byref(cache(**{k: v for k, v in kw.items() if k not in own})))

    def f(q=P, kc=P, vc=P, table=P, start=P, lens=P, ks=NUL, vs=NUL, s_out=NUL, out=P, ws=NUL, n=0, **kw):
        return L.paged_attention(*descs(kw), q, kc, vc, table, start, lens, ks, vs, s_out, out, ws, n, None)

    assert L.paged_attention(None, ctypes.byref(cache()), *[P] * 11, 0, None) == 1
    assert L.paged_attention(ctypes.byref(attention()), None, *[P] * 11, 0, None) == 1
    for kw, status in CACHE_BAD + [(dict(dtype=1), 5), (dict(T=-1), 2), (dict(Hq=3), 2), (dict(Hq=0), 2), (dict(Hq=258), 2),
                                   (dict(T=1 << 29), 2), (dict(max_q=0), 2), (dict(T=1 << 20, max_q=1 << 20, B=1 << 10), 2),
                                   (dict(D=136), 2), (dict(D=4), 2), (dict(D=72, cells=1), 2), (dict(Hkv=0), 2),
                                   (dict(qs=(252, 64)), 4), (dict(os=(256, -64)), 4), (dict(scale=0.0), 11),
                                   (dict(scale=float("nan")), 11)]:
        assert f(**kw) == status, kw
    for name in ("q", "kc", "vc", "table", "lens", "out"):
        assert f(**{name: NUL}) == 1, name
    for name in ("q", "kc", "vc", "out", "ws"):
        assert f(**{name: ODD}) == 3, name
    for name in ("table", "start", "lens", "s_out"):
        assert f(**{name: ctypes.c_void_p(0x10002)}) == 3, name
    assert f(start=NUL, T=5) == 2 and f(ks=P, vs=P) == 11 and f(cells=1, ks=P) == 1
    assert b"paged_attention" in L.w8_last_error()
    assert f(T=0, q=NUL) == 0 and f(B=0, q=NUL) == 0
    n = ctypes.c_int64(-1)
    assert L.paged_attention_workspace(*descs(dict(T=0)), ctypes.byref(n)) == 0 and n.value == 0
    assert L.paged_attention_workspace(*descs({}), None) == 1


F32, I32, U8 = torch.float32, torch.int32, torch.uint8


def rope_args():
    return dict(q=on(5, 4, 64), k=on(5, 2, 64), positions=on(5, dtype=I32), turns=on(32, dtype=torch.int64), q_weight=on(64),
                k_weight=on(64), q_out=on(5, 4, 64), k_out=on(5, 2, 64))


def append_args():
    return dict(k=on(5, 2, 64), v=on(5, 2, 64), k_cache=on(9, 16, 2, 64, dtype=U8), v_cache=on(9, 16, 2, 64, dtype=U8),
                page_table=on(2, 4, dtype=I32), q_start=on(3, dtype=I32), kv_len=on(2, dtype=I32), turns=on(32, dtype=torch.int64),
                q=on(5, 4, 64), q_weight=on(64), k_weight=on(64), positions=on(5, dtype=I32), k_scale=on(1, dtype=F32),
                v_scale=on(1, dtype=F32), q_out=on(5, 4, 64))


def attention_args():
    a = {k: v for k, v in append_args().items() if k in ("k_cache", "v_cache", "page_table", "q_start", "kv_len", "q", "k_scale",
                                                         "v_scale")}
    return dict(a, s_out=on(1, dtype=F32), out=on(5, 4, 64, dtype=U8), ws=on(64, dtype=F32))


CALLS = [("qk_norm_rope", rope_args), ("paged_kv_append", append_args), ("paged_attention", attention_args)]


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


@pytest.mark.parametrize("name,args", CALLS)
def test_tensors_of_another_device_or_type(b, name, args):
    getattr(b, name)(**args())
    assert b.recorded[-1][0] == name and b.recorded[-1][1][-1] == 100
    n = len(b.recorded)
    for key, t in args().items():
        for bad in (t.as_subclass(Elsewhere), t.double().as_subclass(type(t))):
            with pytest.raises(b.W8Error) as e:
                getattr(b, name)(**dict(args(), **{key: bad}))
            assert e.value.status in (1, 5), key
    assert all(c[0] != name for c in b.recorded[n:])
    with pytest.raises(b.W8Error) as e:
        getattr(b, name)(**{k: t.as_subclass(Elsewhere) for k, t in args().items()})
    assert e.value.status == 1


@pytest.mark.parametrize("name,args", CALLS)
def test_tensors_of_other_shapes(b, name, args):
    for key, t in args().items():
        if key in ("k_cache", "v_cache", "ws"):
            continue                                         # any number of pages; any room
        wrong = t.new_zeros((*t.shape[:-1], t.shape[-1] + 8)).as_subclass(type(t))
        if key == "page_table":
            wrong = t[0]
        if key == "turns":
            wrong = t[None]
        with pytest.raises(b.W8Error) as e:
            getattr(b, name)(**dict(args(), **{key: wrong}))
        assert e.value.status in (2, 5), key


def test_combinations(b):
    def status(name, **kw):
        args = dict(dict(CALLS)[name](), **kw)
        with pytest.raises(b.W8Error) as e:
            getattr(b, name)(**args)
        return e.value.status

    assert status("qk_norm_rope", positions=None) == 1       # a rotation without positions
    assert status("qk_norm_rope", turns=None) == 11          # positions without a rotation
    assert status("qk_norm_rope", k=None) == 1               # k_out without k
    assert status("qk_norm_rope", axes=()) == 2 and status("qk_norm_rope", axes=(8, 8, 8, 8)) == 2
    assert status("qk_norm_rope", axes=(16, 16)) == 2        # one row of positions for two axes
    assert status("qk_norm_rope", q=on(5, 4, 128)[..., ::2]) == 4
    assert status("qk_norm_rope", q=on(20, 64)) == 2
    assert status("paged_kv_append", q=None) == 1
    assert status("paged_kv_append", v_cache=on(8, 16, 2, 64, dtype=U8)) == 2
    assert status("paged_kv_append", v_cache=on(9, 16, 2, 64)) == 5   # K in codes, V not
    assert status("paged_kv_append", k_cache=on(9, 16, 2, 128, dtype=U8)[..., ::2]) == 4
    assert status("paged_attention", page_table=on(2, 8, dtype=I32)[:, ::2]) == 4
    assert status("paged_attention", out=on(5, 4, 64)) == 5  # codes wanted


def test_outputs_and_workspace_are_allocated_on_the_calls_stream(monkeypatch):
    from fake_cuda import FakeStream, Recorder
    from w8a16_linear_gb300 import binding
    rec = Recorder(monkeypatch, binding)
    plain = rec.library

    class Library(type(plain)):
        def __getattr__(self, name):
            call = super().__getattr__(name)

            def f(*args):
                if name == "paged_attention_workspace":
                    args[2]._obj.value = 64
                return call(*args)
            return f

    rec.library = Library()
    monkeypatch.setattr(binding, "lib", lambda: rec.library)
    c = fake(9, 16, 2, 64)
    i = lambda *s: fake(*s, dtype=I32)  # noqa: E731
    st = FakeStream()
    binding.paged_attention(fake(5, 4, 64), c, c, i(2, 4), i(3), i(2), stream=st)
    assert [s for _, s in rec.allocations] == [st] * 2
    rec.allocations.clear()
    binding.paged_kv_append(fake(5, 2, 64), fake(5, 2, 64), c, c, i(2, 4), i(3), i(2), q=fake(5, 4, 64), stream=st)
    binding.qk_norm_rope(fake(5, 4, 64), fake(5, 2, 64), q_weight=fake(64), stream=st)
    assert [s for _, s in rec.allocations] == [st] * 3


def test_turns_are_the_frequencies_in_parts_of_a_turn():
    from w8a16_linear_gb300 import binding as b
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021")
    f = b.rope_frequencies(128).tolist() + [0.0, -0.25, 7.5, 1e-9]
    turns = b.rope_turns(f, "cpu").tolist()
    for x, t in zip(f, turns):
        want = Fraction(x) * 2 ** 64 / two_pi % 2 ** 64
        off = abs(Fraction(t % 2 ** 64) - want)
        assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 1000)
    with pytest.raises(b.W8Error):
        b.rope_turns([float("inf")], "cpu")


def test_frequencies():
    from w8a16_linear_gb300 import binding as b
    f = b.rope_frequencies(64, 500.0)
    assert all(math.isclose(x, 500.0 ** (-2 * i / 64), rel_tol=1e-14) for i, x in enumerate(f.tolist()))
    assert torch.allclose(b.rope_frequencies(64, 500.0, factor=4.0), f / 4, rtol=1e-14)
    g = b.rope_frequencies(64, 10000.0, factor=8.0, trained=4096)
    f = b.rope_frequencies(64)
    turns = f * 4096 / (2 * math.pi)
    assert torch.equal(g[turns > 33], f[turns > 33])         # fast pairs are kept
    slow = turns < 0.75
    assert slow.any() and torch.allclose(g[slow], f[slow] / 8, rtol=1e-14)
    r = g / f
    assert (r[1:] <= r[:-1]).all() and (r > 0.12).all()      # and a ramp between
    for bad in (dict(dim=63), dict(dim=0), dict(dim=64, base=-1.0), dict(dim=64, factor=0.0), dict(dim=64, trained=0),
                dict(dim=64, trained=4096, fast=1.0, slow=2.0)):
        with pytest.raises(b.W8Error):
            b.rope_frequencies(**bad)
