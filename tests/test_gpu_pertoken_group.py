"""A group of W8A8 linears with a scale for each token equals its members by
themselves, bit for bit, where all partial sums are integers below 2^24 and
the scales powers of two (in general the order of the sum depends on the
group's size)."""

import pytest
import torch

from gpu_util import W  # noqa: F401

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.mark.parametrize("M", [1, 20, 200, 1100])
def test_group_equals_its_members(W, M):
    g = torch.Generator(device="cuda").manual_seed(M)
    K, Ns = 1024, (256, 528, 2064)

    def whole(*shape):
        return torch.randint(-4, 5, shape, generator=g, device="cuda").float().to(F8).view(torch.uint8)

    def powers(n):
        return 2.0 ** torch.randint(-6, 3, (n,), generator=g, device="cuda").float()

    x, s_tok, ws, cs = whole(M, K), powers(M), [whole(n, K) for n in Ns], [powers(n) for n in Ns]
    for G in (2, 3):
        group = W.fp8_linear_w8a8_pertoken_group(x, s_tok, ws[:G], cs[:G])
        for y, w, c in zip(group, ws, cs):
            one = W.fp8_linear_w8a8_pertoken(x, s_tok, w, c)
            torch.cuda.synchronize()
            assert torch.equal(y.view(torch.int16), one.view(torch.int16))
