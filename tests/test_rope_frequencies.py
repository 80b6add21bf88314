"""rope_frequencies by parts: every pair is held to the ramp by its own number of turns
over the trained length, wherever the ramp's ends lie, also beyond the head's first and last pair."""

import math

import pytest
import torch


@pytest.fixture(scope="module")
def b():
    from w8a16_linear_gb300 import binding
    return binding


def ramp(dim, base, trained, n):
    """The (fractional) pair that turns n times: base^(-i / half) trained = 2 pi n."""
    return dim / 2 * math.log(trained / (2 * math.pi * n), base)


@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("base", [500.0, 1e4, 1e6])
@pytest.mark.parametrize("trained", [5, 100, 202, 4096, 8192, 47000, 54000, 65536, 131072, 10 ** 7])
@pytest.mark.parametrize("factor", [4.0, 8.0])
def test_every_pair_stands_on_the_ramp(b, dim, base, trained, factor):
    plain = b.rope_frequencies(dim, base)
    got = (b.rope_frequencies(dim, base, factor, trained) / plain).tolist()
    low, high = math.floor(ramp(dim, base, trained, 32.0)), math.ceil(ramp(dim, base, trained, 1.0))
    for i, (r, f) in enumerate(zip(got, plain.tolist())):
        turns = f * trained / (2 * math.pi)
        divided = min(max((i - low) / (high - low), 0.0), 1.0)
        assert math.isclose(r, 1 - divided + divided / factor, rel_tol=1e-12), (i, turns)
        if turns > 32.0001:
            assert math.isclose(r, 1.0, rel_tol=1e-12), (i, turns)
        if turns < 0.9999:
            assert math.isclose(r, 1 / factor, rel_tol=1e-12), (i, turns)
        elif turns > 1.0001 and i < high:
            assert r > 1 / factor * (1 + 1e-9), (i, turns)


def test_long_training_leaves_the_last_pair_on_the_ramp(b):
    """The last pair of 128 dimensions turns 2.41 times over 131072 positions."""
    r = (b.rope_frequencies(128, 1e4, 8.0, 131072) / b.rope_frequencies(128, 1e4))[63]
    assert math.isclose(float(r), 1 - 18 / 25 * 7 / 8, rel_tol=1e-12)   # the ramp goes from pair 45 to pair 70
    assert (b.rope_frequencies(64, 1e4, 8.0, 10 ** 9) == b.rope_frequencies(64, 1e4)).all()   # all are fast
    assert torch.allclose(b.rope_frequencies(64, 1e4, 8.0, 5), b.rope_frequencies(64, 1e4) / 8, rtol=1e-14)   # all are slow


@pytest.mark.parametrize("bad", [dict(base=1.0), dict(base=0.5), dict(base=math.inf), dict(base=math.nan), dict(trained=math.inf),
                                 dict(factor=math.inf), dict(fast=math.inf), dict(slow=0.0), dict(trained=-1)])
def test_refusals_by_parts(b, bad):
    """A base of 1 or less has no pair that turns a given number of times, or has them the other way round."""
    with pytest.raises(b.W8Error) as e:
        b.rope_frequencies(**dict(dict(dim=64, base=1e4, factor=4.0, trained=4096), **bad))
    assert e.value.status == 11
    assert len(b.rope_frequencies(64, base=1.0)) == 32 and len(b.rope_frequencies(64, base=0.5)) == 32
