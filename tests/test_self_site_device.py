"""A self-attention site asks for its workspace with its own device as the current one, whichever
is current where it is made: the need goes by the SMs of the device that the passes run on."""

import contextlib

import torch

from w8a16_linear_gb300 import binding
from w8a16_linear_gb300.stack import SelfSite


def test_workspace_of_the_sites_device(monkeypatch):
    current, asked = [None], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d
        yield
        current[0] = before

    def workspace(q, k_cache, page_table, max_q=None):
        asked.append((current[0], max_q))
        assert q.shape == (300, 4, 64) and page_table.shape == (3, 7)
        return torch.empty((max_q if max_q <= 64 else 5,))

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(binding, "paged_attention_workspace", workspace)
    cells = torch.zeros((9, 16, 2, 64), dtype=torch.bfloat16)
    site = SelfSite(3, 300, 250, 128, 4, 2, 64, cells, cells, 7)
    assert {d for d, _ in asked} == {cells.device}
    assert {n for _, n in asked} >= {8, 64, 250} and site.ws.numel() == 64     # 16 and 128 rows, and the most; the largest need
