"""The calls that csrc/marshal.cpp takes give what the binding's Python gives: the
same bits, and the same refusals of device tensors."""

import pytest
import torch

from gpu_util import W, dev_f32  # noqa: F401
from paged_util import batch

pytestmark = pytest.mark.gpu


@pytest.fixture
def b(W):
    from w8a16_linear_gb300 import binding
    binding.lib()
    assert binding._marshal is not None
    return binding


def rope_args(codes=False):
    g = torch.Generator(device="cuda").manual_seed(0)
    from w8a16_linear_gb300 import binding
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return dict(q=n(5, 6, 64), k=n(5, 2, 64), positions=torch.arange(5, device="cuda", dtype=torch.int32),
                turns=binding.rope_turns(binding.rope_frequencies(64)), q_weight=n(64), k_weight=n(64), q_out=n(5, 6, 64),
                k_out=n(5, 2, 64))


def append_args(codes=True):
    c = batch([3, 2], [40, 17], 16, 2, 64, codes=codes)
    r = rope_args()
    return dict(k=r["k"], v=r["k"].clone(), k_cache=c.k, v_cache=c.v, page_table=c.table, q_start=c.q_start, kv_len=c.kv_len,
                turns=r["turns"], q=r["q"], q_weight=r["q_weight"], k_weight=r["k_weight"], positions=r["positions"],
                k_scale=c.k_scale, v_scale=c.v_scale, q_out=r["q_out"])


def attention_args(codes=True):
    a = append_args(codes)
    keep = ("k_cache", "v_cache", "page_table", "q_start", "kv_len", "q", "k_scale", "v_scale")
    return dict({k: a[k] for k in keep}, s_out=dev_f32(0.01), out=torch.empty((5, 6, 64), dtype=torch.uint8, device="cuda"),
                ws=torch.empty((1 << 20,), device="cuda"))


CALLS = [("qk_norm_rope", rope_args), ("paged_kv_append", append_args), ("paged_attention", attention_args)]


def outputs(b, name, args):
    getattr(b, name)(**args)
    torch.cuda.synchronize()
    return [args[k].clone() for k in ("q_out", "k_out", "k_cache", "v_cache", "out") if k in args]


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("name,make", CALLS)
def test_same_bits(b, monkeypatch, name, make, codes):
    args = make(codes)
    taken = []
    m = b._marshal

    class Watch:
        def __getattr__(self, f):
            def call(*a):
                taken.append(getattr(m, f)(*a))
                return taken[-1]
            return call

    monkeypatch.setattr(b, "_marshal", Watch())
    got = outputs(b, name, dict(args))
    assert taken == [0]
    monkeypatch.setattr(b, "_marshal", None)
    args = make(codes)
    want = outputs(b, name, args)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(got, want))


@pytest.mark.parametrize("name,make", CALLS)
def test_same_refusals(b, monkeypatch, name, make):
    m = b._marshal

    def status(args):
        try:
            getattr(b, name)(**args)
        except b.W8Error as e:
            return e.status
        return 0

    args = make()
    cases = []
    for key, t in args.items():
        wide = t.new_zeros((*t.shape[:-1], t.shape[-1] + 8))
        cases += [{key: t.cpu()}, {key: t.double()}, {key: wide}]
        if t.dim() > 1:
            cases += [{key: wide[..., ::2]}, {key: t[0]}]
        if key in ("k_scale", "v_scale", "kv_len", "k_cache"):
            cases.append({key: None}) if key != "k_cache" else None
    if "axes" not in args and "turns" in args:
        cases += [dict(axes=(16, 16)), dict(axes=(31,)), dict(axes=(8, 8, 8, 8)), dict(eps=-1.0), dict(amplitude=0.0)]
    if name == "paged_attention":
        cases += [dict(max_q=0), dict(scale=0.0), dict(ws=args["ws"][:0])]
    for case in cases:
        a = dict(args, **case)
        monkeypatch.setattr(b, "_marshal", m)
        try:
            fast = status(a)
        except AttributeError as e:              # None where a tensor is wanted
            fast = type(e)
        monkeypatch.setattr(b, "_marshal", None)
        try:
            slow = status(a)
        except AttributeError as e:
            slow = type(e)
        assert fast == slow, (list(case), fast, slow)
    torch.cuda.synchronize()
