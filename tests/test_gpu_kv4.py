"""The 4-bit key/value cache on the GPU: append and read byte for byte, attention against a
plain 64-bit implementation, at the sizes, masks, strides and contents where they can go wrong."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_gb300 import mmvq
from tests import _kv4
from tests._gpu import dev, host

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def where(bt, cache=None):
    return (dev(bt.cache) if cache is None else cache, dev(bt.table), dev(bt.offsets), dev(np.array(bt.lens, np.int32)))


def kv_inputs(bt, dtype, heads=None):
    x = bt.rng.normal(size=(2, bt.n, heads or bt.kv, bt.D))
    x[0, :, :, :3] *= 20
    x = torch.from_numpy(x).to(TYPES[dtype])
    return x[0], x[1]


def expected_cache(bt, k, v):
    """bt.cache with rows k, v (float64 [n, kv, D]) written."""
    want = bt.cache.copy()
    qk, qv = _kv4.quantise(k), _kv4.quantise(v)
    for r, (b, p) in enumerate(bt.positions()):
        if p < 0:
            continue
        pg, ti, t = bt.at(b, p)
        for h in range(bt.kv):
            _kv4.put(want[pg, h, ti], t, bt.D, [x[r, h] for x in qk], [x[r, h] for x in qv])
    return want


# ------------------------------------------------------------------- append --

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D,kv,page,lens,news", [
    (64, 3, 16, [1], [1]),                             # one token
    (128, 2, 32, [5, 0, 33, 40], [5, 0, 1, 9]),        # an empty sequence, tiles begun and ended inside
    (256, 1, 64, [131, 16, 17], [131, 16, 1]),         # whole tiles and ragged ends
    (128, 5, 16, [70, 20], [68, 18]),                  # starting at an odd place
])
def test_append_writes_the_format_and_nothing_else(dtype, D, kv, page, lens, news):
    bt = _kv4.Batch(D, kv, page, lens, news, seed=D + kv)
    k, v = kv_inputs(bt, dtype)
    w = where(bt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mmvq.kv4_append(k.cuda(), v.cuda(), *w, status=status)
    assert np.array_equal(host(w[0]), expected_cache(bt, k.double().numpy(), v.double().numpy()))
    assert int(host(status)[0]) == 0


def test_append_takes_strided_and_broadcast_inputs():
    bt = _kv4.Batch(128, 4, 32, [37, 19], [20, 19], seed=3)
    qkv = torch.from_numpy(bt.rng.normal(size=(bt.n, 1 + 2 + 12, 128))).float()   # heads of q, k, v in one row
    odd = torch.from_numpy(bt.rng.normal(size=(bt.n, 4, 133))).float()            # rows not aligned to 16 bytes
    one = torch.from_numpy(bt.rng.normal(size=(bt.n, 1, 128))).float()            # one head for all
    for k, v in ((qkv[:, 1:5], qkv[:, 5:13:2]), (odd[:, :, 3:131], odd[:, :, 1:129]), (one.expand(-1, 4, -1), qkv[:, 2:6])):
        w = where(bt)
        g = [dev(t.numpy()) for t in (qkv, odd, one)]
        view = lambda t: torch.as_strided(g[[i for i, b in enumerate((qkv, odd, one)) if b.data_ptr() <= t.data_ptr() < b.data_ptr() + 4 * b.numel()][0]],  # noqa: E731
                                          t.shape, t.stride(), t.storage_offset())
        mmvq.kv4_append(view(k), view(v), *w)
        assert np.array_equal(host(w[0]), expected_cache(bt, k.double().numpy(), v.double().numpy()))


def test_append_clamps_what_is_not_finite_and_says_so():
    bt = _kv4.Batch(64, 1, 16, [3], [3], seed=4)
    k, v = kv_inputs(bt, "f32")
    k[1, 0, 5], k[1, 0, 40], v[2, 0, 0] = float("inf"), float("-inf"), float("nan")
    w = where(bt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mmvq.kv4_append(k.cuda(), v.cuda(), *w, status=status)
    assert np.array_equal(host(w[0]), expected_cache(bt, k.double().numpy(), v.double().numpy()))
    assert int(host(status)[0]) == mmvq.ERR_VALUE
    k, v = kv_inputs(bt, "f32")
    k[0] = 1e30    # finite, beyond fp16: clamped without a word
    v[0] = 3e-8    # d rounds to zero
    v[1, 0, :32] = 7.0
    status.zero_()
    mmvq.kv4_append(k.cuda(), v.cuda(), *w, status=status)
    assert np.array_equal(host(w[0]), expected_cache(bt, k.double().numpy(), v.double().numpy()))
    assert int(host(status)[0]) == 0


def test_append_ties_and_extreme_blocks():
    """Values at and next to the places where the code changes, steps from subnormal to the largest."""
    D, n = 256, 40
    bt = _kv4.Batch(D, 1, 64, [n], [n], seed=5)
    d = np.float32(2.0) ** np.arange(-24, 16).repeat(1)[:, None, None]
    x = (bt.rng.integers(0, 31, (n, 1, D)) / 2 - 7.5).astype(np.float32)       # whole and half steps
    x[..., 0::32], x[..., 1::32] = -7.5, 7.5                                   # d = the power of two, z = 0
    k = np.clip(x * d, -65504, 65504).astype(np.float32)
    v = np.nextafter(k, np.float32(np.inf)) + d * np.float32(bt.rng.integers(-3, 4))
    w = where(bt)
    mmvq.kv4_append(dev(k), dev(v.astype(np.float32)), *w)
    assert np.array_equal(host(w[0]), expected_cache(bt, k.astype(np.float64), v.astype(np.float32).astype(np.float64)))


def test_append_skips_bad_pages_and_negative_positions():
    bt = _kv4.Batch(128, 2, 16, [40, 3, 30], [40, 5, 4], seed=6)   # sequence 1: two rows before its beginning
    k, v = kv_inputs(bt, "f32")
    bad = bt.table.copy()
    bad[0, 1], bad[2, 1] = bt.n_pages, -1
    w = (dev(bt.cache), dev(bad), dev(bt.offsets), dev(np.array(bt.lens, np.int32)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mmvq.kv4_append(k.cuda(), v.cuda(), *w, status=status)
    want = expected_cache(bt, k.double().numpy(), v.double().numpy())
    for b, pi in ((0, 1), (2, 1)):
        want[bt.table[b, pi]] = bt.cache[bt.table[b, pi]]
    assert np.array_equal(host(w[0]), want)
    assert int(host(status)[0]) == mmvq.ERR_ROUTING
    # a length past the table, and a table too short for it
    status.zero_()
    w = (dev(bt.cache), dev(bt.table), dev(bt.offsets), dev(np.array([40, 3, 16 * bt.table.shape[1] + 2], np.int32)))
    mmvq.kv4_append(k.cuda(), v.cuda(), *w, status=status)
    assert int(host(status)[0]) == mmvq.ERR_ROUTING


# --------------------------------------------------------------------- read --

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D,kv,page,lens,news", [
    (64, 1, 16, [1], [1]), (128, 3, 32, [50, 0, 33], [50, 0, 2]), (256, 2, 128, [200, 7], [63, 7]), (64, 12, 16, [18], [18])])
def test_read_gives_the_rounded_values(dtype, D, kv, page, lens, news):
    bt = _kv4.Batch(D, kv, page, lens, news, seed=7 * D + kv)
    bt.fill_random()
    k, v = mmvq.kv4_read(*where(bt), bt.n, dtype=TYPES[dtype])
    wk, wv = np.zeros((bt.n, kv, D)), np.zeros((bt.n, kv, D))
    for r, (b, p) in enumerate(bt.positions()):
        (sk, *_), (sv, *_) = bt.sequence(b)
        wk[r], wv[r] = sk[p], sv[p]
    for got, want in ((k, wk), (v, wv)):
        want = torch.from_numpy(want).float().to(TYPES[dtype])   # z + d (c - 7.5) rounded to fp32, then to the type
        assert torch.equal(got.cpu(), want)


def test_read_of_missing_places_is_zero():
    bt = _kv4.Batch(128, 2, 16, [40, 3], [40, 5], seed=9)
    bt.fill_random()
    bad = bt.table.copy()
    bad[0, 1] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = mmvq.kv4_read(dev(bt.cache), dev(bad), dev(bt.offsets), dev(np.array(bt.lens, np.int32)), bt.n, status=status)
    k = host(k)
    assert int(host(status)[0]) == mmvq.ERR_ROUTING
    assert not k[16:32].any() and not k[40:42].any() and k[:16].any(-1).all() and k[42:].any(-1).all()


def test_append_then_read_is_the_quantised_value():
    bt = _kv4.Batch(256, 2, 64, [77, 300], [77, 129], seed=10, fill=0)
    k, v = kv_inputs(bt, "f32")
    w = where(bt)
    mmvq.kv4_append(k.cuda(), v.cuda(), *w)
    for got, x in zip(mmvq.kv4_read(*w, bt.n), (k, v)):
        assert np.array_equal(host(got), _kv4.values(*_kv4.quantise(x.double().numpy())).astype(np.float32))


# ---------------------------------------------------------------- attention --
# Bounds, from the arithmetic alone.  A score is a sum of products of q and of a code's value:
# q to 2^-23 of itself, at most four chained fp32 accumulations a block that may each drop 2^-23 of
# the magnitudes, eight blocks added in fp32 (2^-24 each), the scale: below 2^-19 of s = scale *
# sum |q| (|z| + 15 d).  A probability is then off by 2^-19 s (twice: once in the sum, once in the
# weight) and 2^-20 for exp2 and its fp32 argument; weighted sums of the values by as much of a =
# sum p (|z| + d |c - 7.5|), plus 2^-20 for their accumulation.  (For fp16 and bf16 queries the codes enter as
# subnormals, whose sums drop 2^-18 of the largest product instead of 2^-23 of the magnitudes: inside the same bound.)  Types whose probabilities are kept to
# 11 bits (bf16) add 2^-12 for each of two roundings; the output is rounded once.

def bound(dtype, y, a, s):
    b = a * (2.0 ** -18 * s[..., None] + 2.0 ** -19) + 1e-30
    if dtype == "bf16":
        b = b + a * 2.0 ** -11
    return b + np.abs(y) * {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype] + {"f32": 0.0, "f16": 2.0 ** -24, "bf16": 0.0}[dtype]


def check_attention(bt, heads, dtype, scale=None, window=0, sinks=0, gain=1.0, q=None, cache=None, table=None, lens=None, **kw):
    scale = bt.D ** -0.5 if scale is None else scale
    if q is None:
        q = torch.from_numpy(bt.rng.normal(size=(bt.n, heads, bt.D)) * gain).to(TYPES[dtype])
    want, wl, a, s = _kv4.attention(bt, q.double().numpy(), scale, window, sinks)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = where(bt, cache)
    if table is not None:
        w = (w[0], dev(table), *w[2:])
    y, lse = mmvq.kv4_attention(q.cuda(), *w, scale=scale, window=window, sinks=sinks, with_lse=True, status=status, **kw)
    got, gl = host(y.double()), host(lse).astype(np.float64)
    assert int(host(status)[0]) == 0
    assert np.isfinite(got).all(), "non-finite outputs"
    lim = bound(dtype, want, a, s)
    off = np.abs(got - want)
    assert (off <= lim).all(), f"worst {np.nanmax(off / lim):.3g} of the bound at {np.unravel_index(np.nanargmax(off / lim), off.shape)}"
    none = np.isneginf(wl)
    assert np.array_equal(np.isneginf(gl), none) and not got[none].any()
    assert (np.abs(gl[~none] - wl[~none]) <= 2.0 ** -18 * s[~none] + 2.0 ** -20 * (1 + np.abs(wl[~none]))).all()
    return y


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv,group,page,lens,news", [
    (2, 4, 16, [1], [1]),                                   # one token, seen by itself
    (1, 12, 64, [77], [1]),                                 # the odd head ratio of the dense shapes
    (2, 1, 32, [15, 16, 17, 0, 31, 33], [1, 1, 1, 0, 1, 1]),  # tile edges, an empty sequence
    (3, 5, 16, [100, 8, 5, 260], [8, 8, 5, 3]),             # verify windows, one as long as its sequence
    (1, 16, 128, [515], [8]),                               # the most rows
])
def test_attention(dtype, D, kv, group, page, lens, news):
    bt = _kv4.Batch(D, kv, page, lens, news, seed=D + group + len(lens))
    bt.fill_random()
    check_attention(bt, kv * group, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (17, 1), (40, 4), (64, 16), (100, 33), (2000, 3), (5, 1000)])
def test_attention_window_and_sinks(dtype, window, sinks):
    bt = _kv4.Batch(128, 2, 32, [300, 40, 5, 0, 170, 64], [1, 8, 3, 1, 5, 8], seed=window + sinks)
    bt.fill_random()
    # entries of pages that no query sees are not valid
    table = bt.table.copy()
    for b, (n, t) in enumerate(zip(bt.lens, bt.news)):
        for pi in range(-(-n // 32)):
            p = np.arange(32 * pi, min(n, 32 * pi + 32))
            if not ((p > n - t - window) | (p < sinks)).any():
                table[b, pi] = -5
    check_attention(bt, 8, dtype, window=window, sinks=sinks, table=table)


def test_rows_before_the_beginning_see_nothing():
    bt = _kv4.Batch(64, 2, 16, [3, 0, 20], [5, 2, 8], seed=11)
    bt.fill_random()
    check_attention(bt, 4, "f32")


@pytest.mark.parametrize("gain,scale", [(30.0, None), (1e-6, None), (1e4, 1e-3), (300.0, -0.05), (1.0, 0.0)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_attention_score_ranges(dtype, gain, scale):
    """Peaked and flat softmaxes, scores that grow along the sequence, a negative and a zero scale."""
    bt = _kv4.Batch(128, 1, 32, [400, 129], [2, 1], seed=12)
    bt.fill_random()
    check_attention(bt, 4, dtype, gain=gain, scale=scale)


@pytest.mark.parametrize("spread", [1e-4, 1e-2, 50.0, 3000.0])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_attention_cache_ranges(dtype, spread):
    """Steps from fp16's subnormals up to thousands; f16 outputs stay in their range."""
    if dtype == "f16" and spread > 1000:
        spread = 1000.0
    bt = _kv4.Batch(128, 2, 16, [200, 31], [3, 1], seed=13)
    bt.fill_random(spread=spread)
    check_attention(bt, 6, dtype, scale=0.05 / spread)


def test_attention_steps_that_grow_within_a_sequence():
    bt = _kv4.Batch(64, 1, 16, [320], [1], seed=14)
    bt.fill_random()
    half = bt.cache.view(np.float16)
    for i in range(20):                        # value steps and midpoints 4^-5 .. 4^5, rising with the position
        pg, ti, _ = bt.at(0, 16 * i)
        half[pg, 0, ti, 9 * 64:] *= np.float16(2.0 ** (i - 8))
    check_attention(bt, 4, "f32", gain=0.3)


def test_attention_scores_rise_and_fall():
    """The running maximum moves at every tile, then never again."""
    bt = _kv4.Batch(64, 1, 16, [640], [1], seed=15)
    bt.fill_random()
    half = bt.cache.view(np.float16)
    for i in range(40):
        pg, ti, _ = bt.at(0, 16 * i)
        half[pg, 0, ti, 8 * 64 + 32:9 * 64] = np.float16(0.2 * i if i < 20 else 0.2 * (40 - i))
    q = torch.full((1, 2, 64), 0.9)
    q[0, 1] = -0.9
    check_attention(bt, 2, "f32", scale=1.0, q=q)


def test_attention_strided_q_and_given_outputs():
    bt = _kv4.Batch(256, 2, 64, [70, 150], [5, 2], seed=16)
    bt.fill_random()
    both = torch.from_numpy(bt.rng.normal(size=(bt.n, 24, 512))).float()   # queries and their gates side by side
    q = both[:, :, :256]
    want, wl, a, s = _kv4.attention(bt, q.double().numpy(), 1 / 16)
    g = both.cuda()
    y = torch.full((bt.n, 24, 256), 7.0, device="cuda")
    lse = torch.zeros((bt.n, 24), device="cuda")
    ws = mmvq.kv4_attention_workspace(256, "cuda")
    out, l2 = mmvq.kv4_attention(g[:, :, :256], *where(bt), out=y, lse=lse, workspace=ws)
    assert out is y and l2 is lse
    assert (np.abs(host(y) - want) <= bound("f32", want, a, s)).all()
    first = host(y).copy()
    for _ in range(3):   # the workspace is left ready, the results are the same bits
        assert np.array_equal(host(mmvq.kv4_attention(g[:, :, :256], *where(bt), workspace=ws)).view(np.uint32), first.view(np.uint32))


@pytest.mark.parametrize("D,kv,group,lens,news", [(128, 1, 8, [9000], [1]), (256, 1, 3, [5003, 7], [2, 1]), (64, 2, 2, [3001, 6000, 1, 2222], [1, 4, 1, 8])])
def test_attention_long_and_uneven(D, kv, group, lens, news):
    """Sequences split over many CTAs next to ones of a tile."""
    bt = _kv4.Batch(D, kv, 64, lens, news, seed=17)
    bt.fill_random()
    check_attention(bt, kv * group, "f32")
    check_attention(bt, kv * group, "bf16", window=1500, sinks=5)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_even_probabilities_over_many_tokens_cost_no_more_than_the_outputs_rounding(dtype):
    """Values of both signs under nearly equal probabilities cancel to 1/256 of themselves.  What the kernel
    adds to the output's own rounding stays below three quarters of that (1.25 squared is 1 + 0.75 squared).
    Four sequences share the pages, so that a warp adds up a dozen tiles."""
    bt = _kv4.Batch(256, 1, 256, [65536], [1], seed=19)
    bt.fill_random()
    q = torch.from_numpy(bt.rng.normal(size=(1, 12, 256)) * 0.05).to(TYPES[dtype])
    want = _kv4.attention(bt, q.double().numpy(), 1 / 16)[0]
    w = (dev(bt.cache), dev(np.repeat(bt.table, 4, 0)), dev(np.arange(5, dtype=np.int32)), dev(np.full(4, 65536, np.int32)))
    got = host(mmvq.kv4_attention(q.cuda().expand(4, -1, -1), *w).double())
    rounding = np.linalg.norm(torch.from_numpy(want).to(TYPES[dtype]).double().numpy() - want)
    assert max(np.linalg.norm(row - want[0]) for row in got) <= 1.25 * rounding


def test_attention_of_a_large_batch():
    """More sequences than one search step, lengths of every residue."""
    n = 300
    bt = _kv4.Batch(64, 1, 16, [i % 53 for i in range(n)], [min(1 + i % 3, 2) for i in range(n)], seed=18)
    bt.fill_random()
    check_attention(bt, 2, "f32")


def test_attention_refuses_long_windows_and_bad_tables_on_the_device():
    bt = _kv4.Batch(64, 1, 16, [40, 20, 30], [9, 1, 2], seed=19)
    bt.fill_random()
    q = torch.from_numpy(bt.rng.normal(size=(bt.n, 2, 64))).float()
    want, _, a, s = _kv4.attention(bt, q.double().numpy(), 0.125)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((bt.n, 2, 64), 7.0, device="cuda")
    mmvq.kv4_attention(q.cuda(), *where(bt), out=y, status=status)
    assert int(host(status)[0]) == mmvq.ERR_NCOLS
    assert (host(y)[:9] == 7.0).all() and (np.abs(host(y) - want) <= bound("f32", want, a, s))[9:].all()
    # a page that is not there is not attended to: as if its tokens were masked
    bt = _kv4.Batch(64, 1, 16, [40], [1], seed=20)
    bt.fill_random()
    bad = bt.table.copy()
    bad[0, 1] = bt.n_pages + 3
    status.zero_()
    y, lse = mmvq.kv4_attention(q[:1].cuda(), dev(bt.cache), dev(bad), dev(bt.offsets), dev(np.array([40], np.int32)), status=status, with_lse=True)
    assert int(host(status)[0]) == mmvq.ERR_ROUTING
    (k, *_), (v, *_) = bt.sequence(0)
    j = np.r_[0:16, 32:40]
    x = np.einsum("hd,nd->hn", q[0].double().numpy(), k[j, 0]) / 8
    e = np.exp(x - x.max(-1, keepdims=True))
    assert np.abs(host(y)[0] - np.einsum("hn,nd->hd", e / e.sum(-1, keepdims=True), v[j, 0])).max() < 1e-4
    # every page missing: zeros and -inf
    bad[:] = -1
    y, lse = mmvq.kv4_attention(q[:1].cuda(), dev(bt.cache), dev(bad), dev(bt.offsets), dev(np.array([40], np.int32)), status=status, with_lse=True)
    assert not host(y).any() and np.isneginf(host(lse)).all()


def test_nan_queries_stay_in_their_row():
    bt = _kv4.Batch(128, 1, 32, [50], [4], seed=21)
    bt.fill_random()
    q = torch.from_numpy(bt.rng.normal(size=(4, 4, 128))).float()
    clean = host(mmvq.kv4_attention(q.cuda(), *where(bt)))
    q[1, 2, 7], q[3, 0, 0] = float("nan"), float("inf")
    got = host(mmvq.kv4_attention(q.cuda(), *where(bt)))
    bad = np.zeros((4, 4), bool)
    bad[1, 2] = bad[3, 0] = True
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], clean[~bad])


def test_step_on_another_stream():
    """Append and attention of one step, on a side stream, on tensors made on the default one."""
    bt = _kv4.Batch(128, 2, 32, [33, 64], [2, 1], seed=22)
    bt.fill_random()
    k, v = kv_inputs(bt, "f32")
    want = expected_cache(bt, k.double().numpy(), v.double().numpy())
    w, kc, vc = where(bt), k.cuda(), v.cuda()
    q = torch.from_numpy(bt.rng.normal(size=(bt.n, 8, 128))).float()
    qc, ws = q.cuda(), mmvq.kv4_attention_workspace(128, "cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    mmvq.kv4_append(kc, vc, *w, stream=st)
    y = mmvq.kv4_attention(qc, *w, workspace=ws, stream=st)
    st.synchronize()
    bt.cache = want
    yw, _, a, s = _kv4.attention(bt, q.double().numpy(), 128 ** -0.5)
    assert np.array_equal(host(w[0]), want) and (np.abs(host(y) - yw) <= bound("f32", yw, a, s)).all()


def test_offsets_past_32_bits():
    """A cache of over 4 GiB whose used pages lie at its end."""
    D, kv, page = 256, 8, 256
    pages = (1 << 32) // mmvq.kv4_page_bytes(kv, D, page) + 9
    bt = _kv4.Batch(D, kv, page, [300], [2], seed=23, spare=1)
    bt.fill_random()
    cache = mmvq.kv4_cache(pages, kv, D, page, "cuda")
    cache[pages - bt.n_pages:] = dev(bt.cache)
    bt2 = np.where(bt.table >= 0, bt.table + pages - bt.n_pages, bt.table)
    check_attention(bt, 16, "f32", cache=cache, table=bt2.astype(np.int32))
    k, v = kv_inputs(bt, "f32")
    mmvq.kv4_append(k.cuda(), v.cuda(), cache, dev(bt2.astype(np.int32)), dev(bt.offsets), dev(np.array([300], np.int32)))
    assert np.array_equal(host(cache[pages - bt.n_pages:]), expected_cache(bt, k.double().numpy(), v.double().numpy()))
    del cache
    torch.cuda.empty_cache()


def test_graph_replay_with_new_tokens_and_lengths():
    """A captured step (append, attention) replayed after the lengths, inputs and queries changed on the device."""
    D, kv, heads = 128, 2, 8
    bt = _kv4.Batch(D, kv, 32, [400, 90], [1, 1], seed=24)
    bt.fill_random()
    w = where(bt)
    k, v, q = (torch.zeros(2, h, D, device="cuda") for h in (kv, kv, heads))
    y, ws = torch.empty(2, heads, D, device="cuda"), mmvq.kv4_attention_workspace(D, "cuda")

    def step():
        mmvq.kv4_append(k, v, *w)
        mmvq.kv4_attention(q, *w, out=y, workspace=ws)
    for length in ([400, 90], [37, 90]):
        w[3].copy_(torch.tensor(length, dtype=torch.int32))
        step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for length in ([5, 90], [400, 1], [333, 47], [16, 17]):
        for t in (k, v, q):
            t.copy_(torch.from_numpy(bt.rng.normal(size=tuple(t.shape))))
        w[3].copy_(torch.tensor(length, dtype=torch.int32))
        before = host(w[0]).copy()
        graph.replay()
        bt.cache, bt.lens = before, length
        bt.cache = expected_cache(bt, k.double().cpu().numpy(), v.double().cpu().numpy())
        assert np.array_equal(host(w[0]), bt.cache)
        want, _, a, s = _kv4.attention(bt, q.double().cpu().numpy(), D ** -0.5)
        assert (np.abs(host(y) - want) <= bound("f32", want, a, s)).all()


def test_one_workspace_for_calls_of_every_shape():
    """Split and whole items, few rows and many, one after the other in one workspace: the bits of a fresh one."""
    ws = mmvq.kv4_attention_workspace(64, "cuda")
    calls = []
    for i, (kv, group, lens, news) in enumerate([(1, 2, [4000], [1]), (2, 8, [30, 2000, 5], [2, 1, 1]), (1, 16, [900], [8]), (3, 1, [16] * 40, [1] * 40)]):
        bt = _kv4.Batch(64, kv, 16, lens, news, seed=30 + i)
        bt.fill_random()
        q = torch.from_numpy(bt.rng.normal(size=(bt.n, kv * group, 64))).float().cuda()
        calls.append((q, where(bt)))
    fresh = [host(mmvq.kv4_attention(q, *w)).copy() for q, w in calls]
    for _ in range(2):
        outs = [mmvq.kv4_attention(q, *w, workspace=ws) for q, w in calls]   # nothing waits in between
        for got, want in zip(outs, fresh):
            assert np.array_equal(host(got).view(np.uint32), want.view(np.uint32))
    assert not host(ws[:7680]).any()   # the join counters are left at zero
