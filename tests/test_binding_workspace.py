"""cross_attention_workspace answers for every q, k and v that cross_attention
takes, and refuses others in the binding's own way."""

import pytest
import torch

from fake_cuda import fake


@pytest.fixture(scope="module")
def b():
    from w8a16_linear_gb300 import binding, build
    build.build()
    return binding


def status(b, *args):
    """0, or the status of the W8Error."""
    try:
        b.cross_attention_workspace(*args)
    except b.W8Error as e:
        return e.status
    return 0


def test_queries_that_all_samples_share(b):
    """Their sample's stride is 0, which an output's may not be."""
    q, k = fake(1, 1, 4, 64).expand(3, -1, -1, -1), fake(3, 900, 2, 64)
    assert q.stride(0) == 0
    # without a GPU the library gets as far as asking for the device
    assert status(b, q, k, k) in (0, 9)
    assert status(b, q[:1], k[:1], k[:1]) in (0, 9)


def test_refusals(b):
    q, k = fake(3, 1, 4, 64), fake(3, 900, 2, 64)
    assert status(b, q[0], k, k) == 2                  # not four dimensions
    assert status(b, q, k[0], k) == 2
    assert status(b, q.float(), k, k) == 5
    assert status(b, q, k.half(), k) == 5              # not q's type
    assert status(b, q, k, k[:, :800]) == 2            # K and V of different lengths
    assert status(b, q, k[:2], k[:2]) == 2             # not q's samples
    assert status(b, q, k[..., :32], k[..., :32]) == 2
