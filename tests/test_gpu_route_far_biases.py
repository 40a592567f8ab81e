"""Groups of experts whose two best add up to more than fp32 holds, on the GPU."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_gb300 import mmvq
from tests import _layer
from tests._gpu import host

pytestmark = pytest.mark.gpu


def check(x, bias, k, groups, top, scoring):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, w = mmvq.route_topk(x, k, scoring=scoring, bias=bias, n_groups=groups, top_groups=top, status=st)
    want, ww = _layer.route(x.double().cpu().numpy(), k, scoring, bias.double().cpu().numpy(), groups, top, True, 1.0)
    assert np.array_equal(host(ids), want), np.argwhere(host(ids) != want)[:5]
    # logits within 8 of one another: exp of a rounded difference, a sum of 8 terms, a quotient: below 64 half units
    assert (np.abs(host(w) - ww) <= ww * 64 * 2.0 ** -24).all()
    assert int(st[0]) == 0


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top", [(64, 8, 3), (256, 8, 4), (60, 4, 1), (96, 32, 2), (1000, 5, 2), (24, 12, 5)])
def test_sums_of_two_beyond_fp32(scoring, E, groups, top):
    size = E // groups
    gen = torch.Generator("cuda").manual_seed(E)
    x = torch.randn((9, E), device="cuda", generator=gen)
    g = torch.arange(E, device="cuda") // size
    rising = 1 + g / 128.0
    for sign in (1.0, -1.0):
        # the last groups' sums are the largest; all of them, or half of them, beyond fp32
        for bias in (sign * 2.5e38 * rising, torch.where(g % 2 == 0, sign * 2.5e38 * rising, torch.randn(E, device="cuda", generator=gen))):
            check(x, bias.float(), min(8, size), groups, top, scoring)
    # infinite biases: such groups first, in order of their ids
    bias = torch.randn(E, device="cuda", generator=gen) * 0.1
    bias[size + 1] = bias[3 * size] = float("inf")
    check(x, bias, min(8, size), groups, top, scoring)
    bias[::size] = float("-inf")                    # groups with one expert less, some with one alone
    check(x, bias, 1, groups, top, scoring)
