"""Calls of the 4-bit cache at the edges of what their arguments allow: streams, windows, lengths, many
sequences, long sums, values at a code's border."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_gb300 import mmvq
from tests import _kv4
from tests._gpu import dev, host
from tests.test_gpu_kv4 import bound, check_attention, expected_cache, where

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


@pytest.mark.parametrize("rows", [5, 40])   # the kernel for few rows a sequence, and the one for tiles
def test_append_next_to_the_border_of_the_last_code(rows):
    """Steps so small that fp16 rounds them by much: the quotient of a block's largest (or smallest) value lies next
    to 8, where adding 7.5 rounds to 15.5.  At every place of a block, among zeros and among values like it."""
    D = 64
    bt = _kv4.Batch(D, 2, 16, [rows], [rows], seed=42)
    k = np.zeros((rows, 2, D), np.float32)
    v = bt.rng.uniform(-4, 4, (rows, 2, D)).astype(np.float32) * np.float32(2.0 ** -24)
    below = np.nextafter(np.float32(8), np.float32(0))
    for r in range(rows):
        for h in range(2):
            for b in range(2):
                at = (7 * r + 5 * h + 3 * b + np.array([0, 9])) % 32 + 32 * b
                step = np.float32((1 + r % 5) * 2.0 ** -24)
                for x in (k, v):
                    x[r, h, at[0]], x[r, h, at[1]] = below * step, -below * step
    assert (_kv4.quantise(k.astype(np.float64))[0] == 15).any()
    w = where(bt)
    mmvq.kv4_append(dev(k), dev(v), *w)
    assert np.array_equal(host(w[0]), expected_cache(bt, k.astype(np.float64), v.astype(np.float64)))
