"""Calls of the 4-bit cache at the edges of what their arguments allow: streams, windows, lengths, many
sequences, long sums, values at a code's border."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_gb300 import mmvq
from tests import _kv4
from tests._gpu import dev, host
from tests.test_gpu_kv4 import bound, check_attention, where

pytestmark = pytest.mark.gpu


def test_defaults_on_another_stream():
    """Outputs and workspace made by the call, on a side stream, while the current stream is busy and its pool's
    free memory holds ones: items split over many CTAs still find zeroed counters."""
    bt = _kv4.Batch(128, 1, 64, [5000, 900], [1, 1], seed=40)
    bt.fill_random()
    q = torch.from_numpy(bt.rng.normal(size=(2, 8, 128))).float()
    want, _, a, s = _kv4.attention(bt, q.double().numpy(), 128 ** -0.5)
    w, qc, all_of_0 = where(bt), q.cuda(), dev(np.array([0, 5000, 5000], np.int32))
    (k, *_), (v, *_) = bt.sequence(0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        dirty = [torch.full((n,), -1, dtype=torch.int32, device="cuda") for n in (1 << 22, 1 << 20, 4096)]
        del dirty
        torch.cuda._sleep(2_000_000)          # about a millisecond of the current stream
        y = mmvq.kv4_attention(qc, *w, stream=side)
        kr, vr = mmvq.kv4_read(*w[:2], all_of_0, w[3], 5000, stream=side)
        dirty = torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda")
        side.synchronize()
        assert (np.abs(host(y) - want) <= bound("f32", want, a, s)).all()
        assert np.array_equal(host(kr), k.astype(np.float32)) and np.array_equal(host(vr), v.astype(np.float32))
        del dirty


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 6, 1 << 30])
@pytest.mark.parametrize("sinks", [0, 2])
def test_windows_up_to_the_largest_number(window, sinks):
    """As good as none, also where a sequence has more rows than tokens, whose first position is negative."""
    bt = _kv4.Batch(64, 2, 16, [3, 0, 20, 5], [5, 2, 8, 8], seed=41)
    bt.fill_random()
    check_attention(bt, 4, "f32", window=window, sinks=sinks)
