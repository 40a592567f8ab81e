"""Softmax scores far below the best one, on the GPU: their logits' distances to it round to the same fp32 number, and
their order is still that of 64 bits."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_gb300 import mmvq
from tests import _layer
from tests._gpu import host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,groups,top,k", [(16, 4, 2, 8), (24, 12, 5, 8), (32, 2, 1, 12), (64, 8, 3, 10), (256, 8, 4, 32), (1024, 16, 5, 32)])
def test_scores_that_32_bits_cannot_tell_apart(E, groups, top, k):
    rng = np.random.default_rng(E)
    rows = []
    for best in (33.0, 63.0, 65.0, 70.0, 85.0, 99.0, 110.0):
        for spread in (1, 2, 9, 40, 300):                # in units of 2^-23; a distance's unit is 2^-18 to 2^-17
            x = np.float32(1) + rng.integers(0, spread + 1, E).astype(np.float32) * np.float32(2.0 ** -23)
            x[rng.integers(E)] = best
            rows.append(x)
    x = torch.from_numpy(np.stack(rows))
    for b in (None, torch.zeros(E)):
        ids, _ = mmvq.route_topk(x.cuda(), k, n_groups=groups, top_groups=top, bias=None if b is None else b.cuda())
        want, _ = _layer.route(x.double().numpy(), k, "softmax", None if b is None else b.double().numpy(), groups, top, True, 1.0)
        assert np.array_equal(host(ids), want), np.argwhere(host(ids) != want)[:5]
