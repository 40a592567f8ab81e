"""Log probabilities on the GPU of logits far from zero, where neighbouring numbers of fp32 are whole units apart."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_gb300 import mmvq
from tests import _layer

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
I32 = dict(dtype=torch.int32, device="cuda")


def check(x, scale, top=20, distinct=None):
    """Of rows that are the first `distinct` of them over and over.  A sum is of at most 130 additions of a thread, 20 of its CTA and cluster (half a unit each), of terms whose exponent's
    rounding (24) and ex2 (4) count: below 200 half units, which log1p makes no larger.  The entropy's sum is of terms that
    are up to 16 times as large where they count: 1600 more.  What is written: 4 half units of the value."""
    st = torch.zeros(1, **I32)
    n, V = x.shape
    tokens = torch.tensor([[0, V // 2, V - 1]], **I32).expand(n, 3).contiguous()
    got = mmvq.token_logprobs(x, tokens, top=top, scale=scale, status=st)
    d = min(n, distinct or n)
    want = _layer.logprobs(x[:d].double().cpu().numpy(), tokens[:d].cpu().numpy(), top, float(np.float32(scale)))
    want = {name: w[np.arange(n) % d] for name, w in want.items()}
    assert np.array_equal(got["top_ids"].cpu().numpy(), want["top_ids"])
    for name, units in (("lse", 200), ("entropy", 1800), ("logprobs", 200), ("top_logprobs", 200)):
        g, w = got[name].double().cpu().numpy(), want[name]
        w = np.where(np.abs(w) > 3.402823567e38, np.copysign(np.inf, w), w)   # what fp32 has no number for
        assert np.array_equal(g[np.isinf(w)], w[np.isinf(w)]), name
        f = np.isfinite(w)
        off = np.abs(g[f] - w[f]) / 2.0 ** -24
        assert (off <= units + 4 * np.abs(w[f])).all(), (name, np.nanmax(off), np.isnan(off).sum())
    assert int(st[0]) == 0


def rows(V, base, dtype, gen):
    """At a distance: all equal; two levels; a few next to one another; steps of the type's own, and of several."""
    one = torch.tensor(base, device="cuda").to(TYPES[dtype])
    one = one.float()
    unit = torch.finfo(TYPES[dtype]).eps * 2.0 ** np.floor(np.log2(abs(float(one))))
    steps = [torch.zeros(V, device="cuda"), -(torch.arange(V, device="cuda") % 2).float(), -(torch.arange(V, device="cuda") % 7).float(),
             -torch.randint(0, 12, (V,), device="cuda", generator=gen).float(), torch.randint(-50, 1, (V,), device="cuda", generator=gen).float() * 3]
    x = torch.stack([one + s * unit for s in steps]).to(TYPES[dtype])
    assert bool(torch.isfinite(x).all())
    return x


# powers of two that scale * log2(e) * logit lies near: 24, from which on a number of that size is a whole unit off, 31, 32 and
# 35, from which on its half unit is an exponent that fp32 does not hold, 99 to 101 and further
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("power", [12, 22, 23.6, 24.2, 27, 30.6, 31.2, 32, 35, 50, 76, 99, 100.5, 110])
@pytest.mark.parametrize("n,V", [(1, 40), (1, 5003), (700, 300)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_logits_at_a_distance(dtype, n, V, power, sign):
    gen = torch.Generator("cuda").manual_seed(V)
    bases = [40000.0] if dtype == "f16" else [3000.0, 1e6, 1e9, 1e20, 1e30, 1e38]
    for base in bases:
        scale = 2.0 ** power / (base * 1.4427)
        if not 2.0 ** -60 < scale < 2.0 ** 60:
            continue
        x = rows(V, sign * base, dtype, gen)
        x = x.repeat(-(-n // len(x)), 1)
        check(x, scale, distinct=5)
        check(x, scale, 0, distinct=5)
        check(x[:, 1:], scale, distinct=5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V", [(1, 151936), (20, 50021), (400, 20011), (700, 8209)])
def test_long_rows_at_a_distance(dtype, n, V):
    """Ties carry the sums: values that the list has no room for lie at its last."""
    gen = torch.Generator("cuda").manual_seed(1)
    for base, scale in ((1e9, 1.0), (-1e9, 1.0), (3e7, 1.0), (1e30, 1e-4), (-3e30, 0.01), (-1e9, 1 / 64), (1e9, 1 / 64)):
        x = rows(V, base, dtype, gen)
        if n == 1:
            for i in range(5):
                check(x[i:i + 1], scale)
        else:
            check(x.repeat(n // 5, 1), scale, distinct=5)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("mask", [-1e4, -6e4, -1e9, -1e30, -3e38])
def test_a_few_tokens_above_a_finite_mask(dtype, mask):
    """Fewer allowed than the list holds: its last, and so the sums' reference, is the mask."""
    if dtype == "f16" and mask < -65504:
        mask = -65504.0
    gen = torch.Generator("cuda").manual_seed(2)
    for n, V in ((1, 151936), (40, 20011), (700, 8209), (700, 300)):
        d = min(n, 10)
        for allowed in (1, 3, 7, 19, 25):
            x = torch.full((d, V), mask, device="cuda")
            at = torch.randint(0, V, (d, allowed), device="cuda", generator=gen)
            x.scatter_(1, at, torch.randn((d, allowed), device="cuda", generator=gen) * 3)
            check(x.to(TYPES[dtype]).repeat(n // d, 1), 1.0, distinct=d)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("power", [10, 19, 30, 50, 63])
@pytest.mark.parametrize("n,V", [(1, 349), (3, 50021), (700, 300), (200, 2600)])
def test_differences_that_fp32_does_not_hold(dtype, power, n, V):
    """Scales that put the next number below infinitely far: what is not equal to the largest has no probability."""
    gen = torch.Generator("cuda").manual_seed(V)
    low = torch.finfo(TYPES[dtype]).min
    x = torch.randn((5, V), device="cuda", generator=gen)
    x[1] *= 6e3 if dtype == "f16" else 1e30
    x[2] = x[2].masked_fill(torch.rand(V, device="cuda", generator=gen) < 0.7, low)
    x[3] = x[1].masked_fill(torch.rand(V, device="cuda", generator=gen) < 0.5, low)
    x[4] = low * 0.9
    x = x.to(TYPES[dtype]).repeat(-(-n // 5), 1)[:n]
    for top in (1, 20):
        if n > 1:
            check(x, 2.0 ** power, top, distinct=5)
    if n == 1:
        for i in range(5):
            check(rows_of(dtype, V, i, low), 2.0 ** power)


def rows_of(dtype, V, i, low):
    gen = torch.Generator("cuda").manual_seed(V + i)
    x = torch.randn((1, V), device="cuda", generator=gen) * (6e3 if dtype == "f16" else 1e30) ** (i % 2)
    if i > 1:
        x = x.masked_fill(torch.rand(V, device="cuda", generator=gen) < 0.7, low)
    return x.to(TYPES[dtype])
