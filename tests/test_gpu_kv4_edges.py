"""Calls of the 4-bit cache at the edges of what their arguments allow: streams, windows, lengths, many
sequences, long sums, values at a code's border."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_gb300 import mmvq
from tests import _kv4
from tests._gpu import dev, host
from tests.test_gpu_kv4 import TYPES, bound, check_attention, expected_cache, where

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


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 20), (2 ** 31 - 1, 0)])
def test_attention_of_lengths_far_past_the_table(window, sinks):
    """Only the table's tokens are looked at, however long the sequence says it is; the others are as if masked."""
    bt = _kv4.Batch(64, 2, 16, [96, 40, 64], [2, 1, 8], seed=43, table_spare=0)   # 6 pages a row of the table
    bt.fill_random()
    q = torch.from_numpy(bt.rng.normal(size=(bt.n, 16, 64))).float()
    lens = np.array([2 ** 31 - 1, 40, 2 ** 31 - 9], np.int32)
    table = bt.table.copy()
    table[1, 3:], table[2, 4:] = 0, bt.n_pages                                     # sequence 2: two pages that are not there
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, lse = mmvq.kv4_attention(q.cuda(), dev(bt.cache), dev(table), dev(bt.offsets), dev(lens), window=window,
                                sinks=sinks, status=status, with_lse=True)
    y, lse = host(y).astype(np.float64), host(lse)
    assert int(host(status)[0]) == mmvq.ERR_ROUTING
    far = window == 100                     # the window lies past the table: the sinks alone are seen
    for b, rows in ((0, range(0, 2)), (2, range(3, 11))):
        (k, kz, kd, _), (v, vz, vd, vc) = bt.sequence(b)
        n = 20 if far else bt.lens[b]
        for r in rows:
            x = np.einsum("hgd,nhd->hgn", q[r].double().numpy().reshape(2, 8, 64), k[:n]) / 8
            p = np.exp(x - x.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            want, a = (np.einsum("hgn,nhd->hgd", p, w[:n]).reshape(16, 64) for w in (v, vz + vd * vc))
            s = np.einsum("hgd,nhd->hgn", np.abs(q[r].double().numpy().reshape(2, 8, 64)), kz[:n] + 15 * kd[:n]).max(-1).reshape(16) / 8
            assert (np.abs(y[r] - want) <= bound("f32", want, a, s)).all()
    bt.lens, bt.news, bt.offsets = [40], [1], np.array([0, 1], np.int32)
    bt.table = bt.table[1:2]
    want, _, a, s = _kv4.attention(bt, q[2:3].double().numpy(), 0.125, window, sinks)
    assert (np.abs(y[2:3] - want) <= bound("f32", want, a, s)).all()


@pytest.mark.parametrize("rows", [4, 40])
def test_negative_lengths_hold_nothing(rows):
    """Down to the least number: no row is written, reads as anything but zeros, or counts as an error."""
    bt = _kv4.Batch(64, 2, 16, [rows, rows], [rows, rows], seed=44)
    bt.fill_random()
    w = (*where(bt)[:3], dev(np.array([-2 ** 31, rows], np.int32)))
    k, v = (dev(bt.rng.normal(size=(bt.n, 2, 64)).astype(np.float32)) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kr, vr = mmvq.kv4_read(*w, bt.n, status=status)
    assert not host(kr)[:rows].any() and not host(vr)[:rows].any() and host(kr)[rows:].any(-1).all()
    assert int(host(status)[0]) == 0
    mmvq.kv4_append(k, v, *w, status=status)
    bt.lens = [-2 ** 31, rows]
    assert np.array_equal(host(w[0]), expected_cache(bt, host(k).astype(np.float64), host(v).astype(np.float64)))
    y, lse = mmvq.kv4_attention(dev(bt.rng.normal(size=(2, 4, 64)).astype(np.float32)), *w[:2], dev(np.array([0, 1, 2], np.int32)), w[3],
                                with_lse=True, status=status)
    assert not host(y)[0].any() and np.isneginf(host(lse)[0]).all() and np.isfinite(host(lse)[1]).all()
    assert int(host(status)[0]) == 0


@pytest.mark.parametrize("D,kv,group,dtype", [(128, 3, 2, "bf16"), (128, 2, 8, "f32"), (256, 2, 2, "f32"), (64, 2, 8, "f16")])
def test_more_sequences_than_a_cta_has_threads(D, kv, group, dtype):
    """400 and more, so that a thread takes several; empty ones between them, and a few long enough to be split."""
    n = 400 if D == 256 else 1030
    lens = [(7 * i) % 29 if i % 5 else 0 for i in range(n)]
    lens[3], lens[n // 2], lens[n - 1] = 2500, 1111, 3000
    news = [0 if i % 7 == 2 else 1 + i % 2 for i in range(n)]
    bt = _kv4.Batch(D, kv, 32, lens, news, seed=45)
    bt.fill_random()
    check_attention(bt, kv * group, dtype)


def shared_rows(bt, q, rows):
    """Attention of `rows` sequences that share bt's one sequence and its query: y in float64."""
    w = (dev(bt.cache), dev(np.repeat(bt.table, rows, 0)), dev(np.arange(rows + 1, dtype=np.int32)), dev(np.full(rows, bt.lens[0], np.int32)))
    return host(mmvq.kv4_attention(q.cuda().expand(rows, -1, -1), *w).double())


@pytest.mark.parametrize("D,group", [(64, 4), (128, 12), (256, 6), (256, 12)])
def test_long_sums_keep_their_precision(D, group):
    """Enough sequences of 65536 tokens that a warp adds up a hundred tiles and more, under nearly even probabilities,
    values with an offset: within the bound of a short sequence, whose chains of products are those of one tile."""
    bt = _kv4.Batch(D, 1, 256, [65536], [1], seed=46)
    bt.fill_random()
    z = bt.cache.view(np.float16)[..., 9 * D + D // 2:]
    z[:] = np.where(np.isfinite(z), np.abs(z) + np.float16(0.25), z)
    q = torch.from_numpy(bt.rng.normal(size=(1, group, D)) * 0.01).float()
    want, _, a, s = _kv4.attention(bt, q.double().numpy(), D ** -0.5)
    got = shared_rows(bt, q, 64)
    off = np.abs(got - want)
    assert (off <= bound("f32", want, a, s)).all(), f"{(off / bound('f32', want, a, s)).max():.2f} of the bound"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_long_sums_that_cancel(dtype):
    """Values of both signs under nearly even probabilities, a hundred tiles and more a warp: what the kernel adds
    stays below three quarters of the output's own rounding."""
    bt = _kv4.Batch(256, 1, 256, [65536], [1], seed=47)
    bt.fill_random()
    q = torch.from_numpy(bt.rng.normal(size=(1, 12, 256)) * 0.05).to(TYPES[dtype])
    want = _kv4.attention(bt, q.double().numpy(), 1 / 16)[0]
    rounding = np.linalg.norm(torch.from_numpy(want).to(TYPES[dtype]).double().numpy() - want)
    assert max(np.linalg.norm(row - want[0]) for row in shared_rows(bt, q, 64)) <= 1.25 * rounding


@pytest.mark.parametrize("D,group", [(64, 4), (128, 4), (256, 12)])
def test_long_sums_that_cancel_carry_no_offset(D, group):
    """The same in fp32, several hundred tiles a warp.  Sums that stay as small as their result: its 2-norm is off by
    2^-22 for each of p, p d, the sums within tiles and sum(p), and by sqrt(1000) 2^-25 for the additions: below 2^-19."""
    bt = _kv4.Batch(D, 1, 256, [65536], [1], seed=50)
    bt.fill_random()
    q = torch.from_numpy(bt.rng.normal(size=(1, group, D)) * 0.05).float()
    want = _kv4.attention(bt, q.double().numpy(), D ** -0.5)[0]
    off = max(np.linalg.norm(row - want[0]) for row in shared_rows(bt, q, 256)) / np.linalg.norm(want)
    assert off <= 2.0 ** -19, f"{off:.2e}"


@pytest.mark.parametrize("n,longest", [(33, 90), (300, 2), (1100, 60), (1100, 3)])
@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 128), ("f16", 256)])
def test_append_and_read_of_many_sequences(n, longest, dtype, D):
    """More than a warp has lanes, so that a row's sequence is found in two steps or three, empty ones between them;
    with few rows each, and with tiles of them."""
    news = [(5 * i) % (longest + 1) if i % 4 else 0 for i in range(n)]
    lens = [t + (3 * i) % 19 for i, t in enumerate(news)]
    bt = _kv4.Batch(D, 1, 16, lens, news, seed=48, fill=0)
    x = torch.from_numpy(bt.rng.normal(size=(2, bt.n, 1, D))).to(TYPES[dtype])
    w = where(bt)
    mmvq.kv4_append(x[0].cuda(), x[1].cuda(), *w)
    k, v = mmvq.kv4_read(*w, bt.n, dtype=TYPES[dtype])
    for got, rows in ((k, x[0]), (v, x[1])):
        want = _kv4.values(*_kv4.quantise(rows.double().numpy())).astype(np.float32)
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(TYPES[dtype]))


@pytest.mark.parametrize("D,kv,group,dtype", [(128, 2, 5, "f16"), (64, 2, 4, "f16"), (64, 1, 16, "bf16"), (256, 2, 3, "f16"),
                                              (256, 1, 12, "bf16"), (256, 1, 12, "f32")])
@pytest.mark.parametrize("window,sinks", [(40, 4), (130, 0), (1000, 17)])
def test_windows_of_every_head_size_and_type(D, kv, group, dtype, window, sinks):
    bt = _kv4.Batch(D, kv, 32, [700, 40, 5, 0, 171, 64], [1, 2, 3, 1, 1, 8], seed=49)
    bt.fill_random()
    check_attention(bt, kv * group, dtype, window=window, sinks=sinks)
