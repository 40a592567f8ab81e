"""Log probabilities, entropy and alternatives on the GPU against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_gb300 import mmvq
from tests import _layer
from tests._gpu import host

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
I32 = dict(dtype=torch.int32, device="cuda")


def check(logits, tokens=None, top=0, scale=1.0, status=0):
    """Alternatives equal.  A term exp(d) is off by half a unit for each unit of d, of which the sum of p |d| (at most
    the entropy) counts, by 16 for exp itself, and by the additions of its thread, its warp and the rows' parts, at
    most 600 for a vocabulary of 300000; a log probability besides by three roundings of d."""
    st = torch.zeros(1, **I32)
    got = mmvq.token_logprobs(logits, tokens, top=top, scale=scale, status=st)
    n, V = logits.shape
    tok = np.zeros((n, 0), np.int32) if tokens is None else tokens.cpu().numpy()
    want = _layer.logprobs(logits.double().cpu().numpy(), tok, top, float(np.float32(scale)))
    assert np.array_equal(host(got["top_ids"]), want["top_ids"])
    with np.errstate(invalid="ignore"):
        unit = 2.0 ** -24
        rel = 2 * unit * (20 + min(600, V) + 4 * want["entropy"])  # of S and of the entropy
        slack = np.minimum(1, want["entropy"]) * rel    # S / (1 + S) <= H
        for name in ("lse", "entropy", "logprobs", "top_logprobs"):
            g, w = host(got[name]).astype(np.float64), want[name]
            assert np.array_equal(np.isnan(g), np.isnan(w)) and np.array_equal(g[np.isinf(w)], w[np.isinf(w)]), name
            s = want["entropy"] * rel if name == "entropy" else slack if w.ndim == 1 else slack[:, None]
            f = np.isfinite(w)
            bound = np.broadcast_to(s, w.shape)[f] + 4 * unit * np.abs(w[f]) + 1e-37
            err = np.abs(g[f] - w[f])
            assert (err <= bound).all(), (name, (err / bound).max())
    assert int(st[0]) == status
    return got


def rows(n, V, dtype, seed, spread=2.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn((n, V), device="cuda", generator=gen) * spread
    x[::2, V // 3] += 18                           # rows that are all but certain
    tokens = torch.randint(0, V, (n, 3), generator=gen, **I32)
    tokens[:, 0] = V // 3
    return x.to(TYPES[dtype]), tokens


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,V,top,scale", [(1, 1, 1, 1.0), (3, 2, 4, 1.0), (2, 31, 32, 0.7), (5, 1000, 20, 1.0), (1, 151936, 20, 0.8),
                                           (8, 151936, 5, 1.0), (40, 4099, 8, 1.3), (301, 513, 1, 1.0), (17, 32771, 32, 1.0), (2, 262147, 7, 1.0),
                                           (700, 8209, 3, 1.0)])
def test_against_64_bits(dtype, n, V, top, scale):
    x, tokens = rows(n, V, dtype, n + V)
    check(x, tokens, top, scale)
    check(x, None, 0, scale)
    check(x, tokens, 0, scale)


def test_many_rows_of_a_long_vocabulary():
    x, tokens = rows(320, 151937, "bf16", 5)
    check(x, tokens, 20)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_equal_logits_go_to_the_lowest_ids(dtype):
    for V in (5, 700, 40001):
        got = check(torch.full((3, V), -1.5, device="cuda", dtype=TYPES[dtype]), None, min(V, 32))
        assert np.array_equal(host(got["top_ids"]), np.tile(np.arange(min(V, 32), dtype=np.int32), (3, 1)))
    coarse = torch.randint(-2, 3, (30, 20011), generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(TYPES[dtype])
    check(coarse, None, 32)


def test_rows_in_order():
    """Rising rows bring a new largest logit at every step, falling ones never."""
    up = torch.arange(50000, device="cuda").float() / 5000
    x = torch.stack((up, up.flip(0), torch.cat((up[::2], up[::2].flip(0))), -up * 50, (up * 1e4).floor()))
    for dtype in (torch.float32, torch.bfloat16):
        check(x.to(dtype), torch.tensor([[0, 49999]] * 5, **I32), 32)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_masks(dtype):
    V = 9001
    x, tokens = rows(12, V, dtype, 7)
    low = torch.finfo(TYPES[dtype]).min
    x[0] = float("-inf")                            # nothing left
    x[1] = float("-inf")
    x[1, 4321] = 2.0                                # one left
    x[2, torch.arange(V, device="cuda") % 1000 != 7] = float("-inf")  # ten left, twenty asked for
    x[3] = low                                      # the type's lowest value everywhere
    x[4, 10:] = low
    x[5, 1:] = low
    x[6, :V - 3] = float("-inf")
    x[7, 3:] = float("-inf")
    tokens[1, 1], tokens[6, 1], tokens[7, 1] = 4321, V - 2, 1
    check(x, tokens, 20)
    check(x, tokens, 20, scale=1e-3)
    if dtype == "f32":
        x[8, 5], x[8, 6] = 3e38, -3e38              # a difference that has no fp32 number: no probability at all
        got = mmvq.token_logprobs(x[8:9].contiguous(), torch.tensor([[5, 6]], **I32), top=1)
        assert host(got["logprobs"]).tolist() == [[0.0, float("-inf")]] and int(got["top_ids"][0, 0]) == 5


def test_rows_that_hold_what_is_no_number():
    x, tokens = rows(9, 5000, "f32", 8)
    x[1, 77], x[4, 4999], x[6, 0] = float("nan"), float("inf"), float("nan")
    check(x, tokens, 5, status=mmvq.ERR_VALUE)
    x, tokens = rows(3, 151936, "bf16", 8)
    x[1, 151935] = float("nan")
    check(x, tokens, 5, status=mmvq.ERR_VALUE)


def test_tokens_that_are_none():
    x, tokens = rows(6, 3001, "f16", 9)
    tokens[0, 0], tokens[3, 2], tokens[5, 1] = -1, 3001, 2 ** 31 - 1
    check(x, tokens, 2, status=mmvq.ERR_ROUTING)


def test_strides_outputs_and_streams():
    wide = torch.randn((40, 5003), device="cuda", generator=torch.Generator("cuda").manual_seed(3)) * 3
    for dtype in TYPES.values():
        for first in range(0, 9):
            check(wide.to(dtype)[::3, first:first + 4990], None, 4)
    x = wide[:, :5000].contiguous()
    tokens = torch.zeros((40, 1), **I32)
    want = mmvq.token_logprobs(x, tokens, top=3)
    part = dict(logprobs=torch.empty((40, 1), device="cuda"), top_ids=torch.empty((40, 3), **I32), top_logprobs=torch.empty((40, 3), device="cuda"))
    got = mmvq.token_logprobs(x, tokens, top=3, out=part)
    assert got is part and all(torch.equal(part[name], want[name]) for name in part)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = mmvq.token_logprobs(x, tokens, top=3, stream=side)
    side.synchronize()
    assert all(torch.equal(got[name], want[name]) for name in want)
    assert mmvq.token_logprobs(x[:0], tokens[:0], top=3)["top_ids"].shape == (0, 3)


def test_two_streams_at_once_and_replays():
    """Calls share nothing: two streams' calls side by side and replays of one graph give the same bits."""
    x = [torch.randn((n, 151936), device="cuda") for n in (1, 5)]
    want = [mmvq.token_logprobs(t, None, top=20) for t in x]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in x]
    got = [[mmvq.token_logprobs(t, None, top=20, stream=s) for t, s in zip(x, side)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert all(torch.equal(a[name], b[name]) for name in b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mmvq.token_logprobs(x[1], None, top=20)
    for _ in range(3):
        x[1].normal_()
        g.replay()
        have = {name: t.clone() for name, t in out.items()}
        again = mmvq.token_logprobs(x[1], None, top=20)
        assert all(torch.equal(have[name], again[name]) for name in again)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,V", [(1, 1000003), (400, 262144), (700, 150001), (3, 5000)])
def test_even_rows_keep_their_sums(dtype, n, V):
    """All logits but eight equal: every addition rounds the same way.  A batch's sums are at most 32 additions of a
    thread, a row's at most 123 batches of it (one CTA of 512 threads to 1000003 fp32), then 10 of its warp and 8 of the
    CTAs: below 180 half units in all, and the same again for exp and its argument's rounding (up to 8)."""
    x = torch.full((n, V), 0.3, device="cuda").to(TYPES[dtype])
    x[:, V // 2:V // 2 + 8] = 1.0                 # the rest lies below the list's last
    got = mmvq.token_logprobs(x, None, top=8)
    a, b = (float(t) for t in (x[0, 0], x[0, V // 2]))
    total = 8 + (V - 8) * np.exp(a - b)           # of exp(x - the largest)
    lse, entropy = b + np.log(total), np.log(total) - (V - 8) * np.exp(a - b) * (a - b) / total
    for name, want in (("lse", lse), ("entropy", entropy)):
        err = np.abs(host(got[name]).astype(np.float64) - want)
        assert err.max() <= 200 * 2.0 ** -24 + 2 * 2.0 ** -24 * want, (name, err.max() / 2.0 ** -24)
    assert np.array_equal(host(got["top_ids"]), np.tile(np.arange(V // 2, V // 2 + 8, dtype=np.int32), (n, 1)))


def test_nothing_beside_the_outputs_is_written():
    n, V, m, top = 5, 4001, 3, 4
    x, tokens = rows(n, V, "bf16", 4)
    want = mmvq.token_logprobs(x, tokens, top=top)
    room = {name: torch.full((t.numel() + 64,), -7, dtype=t.dtype, device="cuda") for name, t in want.items()}
    out = {name: room[name][32:32 + t.numel()].view(t.shape) for name, t in want.items()}
    mmvq.token_logprobs(x, tokens, top=top, out=out)
    for name, t in want.items():
        assert torch.equal(out[name], t) and bool((room[name][:32] == -7).all()) and bool((room[name][-32:] == -7).all())
