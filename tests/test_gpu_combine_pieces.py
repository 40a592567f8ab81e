"""The experts' rows combined on the GPU where a thread has several places of a row at once (few rows a token), against a
plain 64-bit implementation."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_gb300 import mmvq
from tests import _layer
from tests._gpu import host

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("k", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("n,H", [
    (320, 6564), (320, 2054), (320, 1027), (320, 2048), (320, 1030), (320, 515),   # by four, two and one columns; pieces over in the last round
    (120, 6564), (120, 1542), (310, 1000), (310, 258), (305, 129),                   # a token's columns shared out; two rounds of threads
])
def test_several_places_of_a_row_at_once(dtype, k, n, H):
    """k + 2 products added in fp32, each to half a unit of the largest sum on the way; the gate's exp, sum and quotient:
    (k + 12) half units of the sum of sizes, then one rounding."""
    E = 12
    gen = torch.Generator("cuda").manual_seed(n + H + k)
    topk = torch.rand((n, E), device="cuda", generator=gen).argsort(1)[:, :k].to(torch.int32).contiguous()
    topk[1, 0] = topk[n - 1, k - 1] = -1            # slots of no expert
    _, offs, _, slot, _ = mmvq.route_groups(topk, E)
    y, w = torch.randn((n * k, H), device="cuda", generator=gen), torch.randn((n, k), device="cuda", generator=gen)
    y[int(offs[E]):] = float("nan")                 # rows that no slot stands for
    r, s = (torch.randn((n, H), device="cuda", generator=gen).to(TYPES[dtype]) for _ in range(2))
    g = torch.randn(n, device="cuda", generator=gen) * 4
    room = torch.full((n * H + 64,), -7.0, device="cuda").to(TYPES[dtype])
    out = room[32:32 + n * H].view(n, H)
    got = mmvq.combine_experts(y, topk, w, offs, slot, residual=r, shared=s, shared_gate=g, out=out)
    assert got is out and bool((room[:32] == -7).all()) and bool((room[-32:] == -7).all())
    want, size = _layer.combine(host(y), host(topk), host(w), host(offs), host(slot), r.double().cpu().numpy(), s.double().cpu().numpy(), host(g), H)
    info = torch.finfo(got.dtype)
    bound = size * (k + 12) * 2.0 ** -24
    bound = bound + (np.abs(want) + bound) * info.eps / 2 + info.smallest_normal * info.eps
    err = np.abs(host(got.double()) - want)
    assert (err <= bound).all(), (err / bound).max()
    # over the residual, and the experts' rows alone
    assert torch.equal(mmvq.combine_experts(y, topk, w, offs, slot, residual=r, shared=s, shared_gate=g, out=r), got)
    want, size = _layer.combine(host(y), host(topk), host(w), host(offs), host(slot), None, None, None, H)
    alone = mmvq.combine_experts(y, topk, w, offs, slot, dtype=TYPES[dtype])
    bound = size * (k + 12) * 2.0 ** -24
    bound = bound + (np.abs(want) + bound) * info.eps / 2 + info.smallest_normal * info.eps
    assert (np.abs(host(alone.double()) - want) <= bound).all()
