"""Log probabilities on the GPU of rows in which a hundred logits carry everything: a window that goes over the whole
vocabulary, so that a logit lost or counted twice anywhere shows, whatever the rows are shared out by."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_gb300 import mmvq

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
I32 = dict(dtype=torch.int32, device="cuda")
WINDOW, TOP = 100, 20


def windows(n, V, dtype, first, fill):
    """Rows whose windows take turns: every place of the vocabulary is in one.  Of a window the likeliest TOP are listed and
    the other eighty are summed, among logits of no weight (-inf, or exp(-60) for each one).

    A logit has at least exp(-2) / 100 of the sum.  The sum of all but the largest is of at most 99 additions that are
    not of such small ones, after a rounded exponent of at most 3 (3 half units), ex2 (4) and up to ten changes of the
    reference (5 each): below 200 half units, which log1p makes no larger; the entropy's sum is of terms up to 3 times as
    large, stated for up to three references at once: 1000.  What is written besides: 4 half units of the value."""
    size = min(WINDOW, V)
    gen = torch.Generator("cpu").manual_seed(V + first)
    values = (torch.rand(size, generator=gen) * 2 - 1).to(TYPES[dtype])
    v = values.double().numpy()
    order = np.argsort(-v, kind="stable")[:min(TOP, size)]
    p = np.exp(v - v.max())
    lse = v.max() + np.log(p.sum())
    entropy = lse - (p * v).sum() / p.sum()
    small = V * np.exp(-60.0)                       # 2e-21 of it, and of the entropy at most 60 times that
    assert small < 1e-18
    dev = values.cuda()
    buffer = torch.full((n, V + 9), fill, device="cuda", dtype=TYPES[dtype])
    x = buffer[:, first:first + V]                  # rows begin at every address in turn
    buffer[:, :first] = buffer[:, first + V:] = 50.0  # what lies beside the rows is not theirs
    starts = torch.arange(0, -(-V // size), device="cuda") * size
    starts = starts.clamp(max=V - size)
    at = torch.arange(size, device="cuda")
    order = torch.from_numpy(order).cuda()
    unit = 2.0 ** -24
    worst = torch.zeros(4, device="cuda", dtype=torch.float64)
    equal = torch.ones((), dtype=torch.bool, device="cuda")
    for call in range(-(-len(starts) // n)):
        s = starts[(torch.arange(n, device="cuda") + call * n) % len(starts)]
        where = s[:, None] + at
        x.scatter_(1, where, dev.expand(n, -1))
        tokens = torch.stack((s, s + size - 1), 1).to(torch.int32)
        got = mmvq.token_logprobs(x, tokens, top=TOP)
        off = ((got["lse"].double() - lse).abs(), (got["entropy"].double() - entropy).abs(),
               (got["logprobs"].double() - (dev[[0, -1]].double() - lse)).abs(), (got["top_logprobs"][:, :len(order)].double() - (dev[order].double() - lse)).abs())
        worst = torch.maximum(worst, torch.stack([o.max() for o in off]))
        ids = got["top_ids"]
        equal &= (ids[:, :len(order)] == s[:, None] + order).all()
        if V < TOP:
            equal &= (ids[:, V:] == -1).all()
        x.scatter_(1, where, torch.full((n, size), fill, device="cuda", dtype=x.dtype))
    assert bool(equal)
    off = worst.cpu().numpy() / unit
    assert off[0] <= 200 + 4 * abs(lse) and off[1] <= 1000 + 4 * entropy and off[2] <= 200 + 4 * (abs(lse) + 1) and off[3] <= 200 + 4 * (abs(lse) + 1), off


# rows and vocabulary: shared out to clusters of 16, 8, 4 and 2 CTAs and one of 16 warps; by CTAs of 4 warps and of one
SHAPES = [(1, 151936), (3, 151936), (5, 151936), (20, 151936), (40, 151936), (80, 151936), (2, 33000), (40, 50021), (15, 50021), (200, 20011), (100, 4099), (200, 4099),
          (700, 20011), (1, 1001), (700, 8209), (700, 1265), (700, 1001), (700, 633), (700, 601), (2000, 257), (700, 100), (700, 5), (700, 1)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,V", SHAPES)
@pytest.mark.parametrize("fill", [float("-inf"), -60.0])
def test_every_place_of_the_vocabulary_counts_once(dtype, n, V, fill):
    for first in range(9 if V < 60000 else 3):
        windows(n, V, dtype, first, fill)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,V", [(700, 1), (700, 5), (700, 300), (700, 601), (700, 1265), (2000, 601)])
def test_many_short_rows(dtype, n, V):
    """The list, the sums, masks and what is no number, of rows that a warp takes by itself."""
    from tests import _layer
    gen = torch.Generator("cuda").manual_seed(V)
    x = (torch.randn((n, V), device="cuda", generator=gen) * 3).to(TYPES[dtype])
    x[::7, ::2] = float("-inf")
    x[5] = float("-inf")
    x[6] = torch.finfo(TYPES[dtype]).min
    x[8, V // 2], x[9, V - 1] = float("nan"), float("inf")
    x[10] = 1.5                                     # all equal
    x[11] = x[11].sort().values                     # rising: a new largest at every step
    tokens = torch.randint(0, V, (n, 2), generator=gen, **I32)
    tokens[12, 1] = V
    st = torch.zeros(1, **I32)
    for top in (0, 5, 32):
        got = mmvq.token_logprobs(x, tokens, top=top, status=st)
        want = _layer.logprobs(x.double().cpu().numpy(), tokens.cpu().numpy(), top, 1.0)
        assert np.array_equal(got["top_ids"].cpu().numpy(), want["top_ids"])
        # additions: a lane's 40 values at most, 5 of its warp, 4 of the join; exp and its argument (up to 24 for what counts);
        # the entropy's terms up to 16 times as large
        for name, units in (("lse", 100), ("entropy", 1600), ("logprobs", 100), ("top_logprobs", 100)):
            g, w = got[name].double().cpu().numpy(), want[name]
            assert np.array_equal(np.isnan(g), np.isnan(w)) and np.array_equal(g[np.isinf(w)], w[np.isinf(w)]), name
            f = np.isfinite(w)
            assert (np.abs(g[f] - w[f]) <= (units + 4 * np.abs(w[f])) * 2.0 ** -24).all(), (name, np.abs(g[f] - w[f]).max() * 2.0 ** 24)
    assert int(st[0]) in (mmvq.ERR_VALUE, mmvq.ERR_ROUTING)
