"""CrossSite keeps the addresses that a captured pass has taken in: a graph
of run() holds K, V and the workspace by address."""

import pytest
import torch

from w8a16_linear_gb300.stack import CrossSite, CrossWeights


class Library:
    """The calls of a site, recorded, with outputs that hold the call's number."""

    def __init__(self):
        self.n, self.attended = 0, []

    def add_rms_norm_quant(self, x, residual, weight, out=None, s_tok=None, res_out=None):
        return x, s_tok, res_out

    def fp8_linear_w8a8_pertoken(self, qx, s_tok, w, s_ch, out=None):
        return out

    def fp8_linear_w8a8_pertoken_group(self, qx, s_tok, weights, scales, outs=None):
        self.n += 1
        if outs is None:
            outs = [torch.empty((qx.shape[0], w.shape[0]), dtype=torch.bfloat16) for w in weights]
        for o in outs:
            o.fill_(self.n)
        return outs

    def cross_attention_workspace(self, q, k, v):
        return torch.empty((k.shape[1],))

    def cross_attention(self, q, k, v, kv_len=None, kv_mask=None, s_out=None, out=None, ws=None):
        self.attended.append((k, v, ws))

    def fp8_linear_w8a8(self, *args, out=None):
        return out


def addresses(site):
    return [t.data_ptr() for t in (site.k, site.v, site.ws)]


@pytest.fixture
def site(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return CrossSite(2, 3, 64, 4, 2, 16, torch.device("cpu"))


@pytest.fixture
def weights():
    n = torch.ones((64,), dtype=torch.bfloat16)
    w = lambda rows: (torch.zeros((rows, 64), dtype=torch.uint8), torch.ones((rows,)))  # noqa: E731
    return CrossWeights(n, n, w(64), w(32), w(32), w(64), torch.ones((1,)))


def states(T):
    return torch.zeros((2, T, 64), dtype=torch.bfloat16)


def run(site, W, w):
    site.run(W, w, torch.zeros((6, 64)), torch.zeros((6, 64)))


def test_encode_leaves_earlier_keys_alone(site, weights):
    """Without a graph each encode has memory of its own: a caller may have
    kept the keys and values of the states before."""
    W = Library()
    site.encode(W, weights, states(10))
    k, v = site.k, site.v
    site.encode(W, weights, states(10))
    assert (k == 1).all() and (v == 1).all() and (site.k == 2).all() and (site.v == 2).all()


def test_encode_writes_where_a_captured_pass_reads(site, weights, monkeypatch):
    W = Library()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    site.encode(W, weights, states(10))
    run(site, W, weights)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    captured = addresses(site)
    for n in (2, 3):
        site.encode(W, weights, states(10))
        run(site, W, weights)
        assert addresses(site) == captured == [t.data_ptr() for t in W.attended[-1]]
        assert (site.k == n).all() and (site.v == n).all()


def test_a_captured_pass_keeps_its_buffers(site, weights, monkeypatch):
    """Another length gets its own buffers; those of the captured pass stay
    alive, and are written again when states of its length come back."""
    W = Library()
    site.encode(W, weights, states(10))
    captured = addresses(site)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    run(site, W, weights)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    W.attended.clear()   # no references kept here
    others = []
    for T in (7, 11, 12):
        site.encode(W, weights, states(T))
        assert site.k.shape[1] == T
        others.append(torch.empty((2, 10, 2, 16), dtype=torch.bfloat16))   # would take freed memory
        assert set(addresses(site)).isdisjoint(captured)
        assert all(t.data_ptr() not in captured for t in others)
    site.encode(W, weights, states(10))
    assert addresses(site) == captured
    assert (site.k == 5).all()


def test_lengths_that_no_graph_holds_are_let_go(site, weights):
    W = Library()
    for T in (5, 6, 7, 8):
        site.encode(W, weights, states(T))
        run(site, W, weights)
        del W.attended[:]
    assert len(site.captured) == 0
    assert site.k.shape[1] == 8
