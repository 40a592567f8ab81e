"""The quotients of the 4-bit cache's quantiser, step by step in fp32 on the CPU, against the division."""
import numpy as np

F, L = np.float32, np.longdouble


def fma(a, b, c):
    """a b + c rounded once.  Exact before that: the callers' sums span at most 60 bits."""
    return (L(a) * L(b) + L(c)).astype(F)


def test_longdouble_holds_the_sums():
    assert np.finfo(L).nmant >= 63


def test_a_fifteenth_of_every_significand():
    """q = x c, c = fp32(1/15), corrected once by its exact remainder, as divide15 does it."""
    c = F(1) / F(15)
    for k in range(8):
        x = (np.arange(k << 20, (k + 1) << 20, dtype=np.uint32) + np.uint32(0x3f800000)).view(F)
        q = x * c
        got = fma(fma(np.full_like(x, -15), q, x), np.full_like(x, c), q)
        assert np.array_equal(got.view(np.uint32), (x / F(15)).view(np.uint32))


def test_quotients_by_every_step():
    """(x - z) / d by the rounded reciprocal of d, corrected once, for every fp16 significand of d: random numerators,
    and those next to the middle between two fp32 quotients, where the rounding is decided."""
    rng = np.random.default_rng(1)
    d = np.arange(1024, 2048, dtype=F)[:, None]
    r = F(1) / d
    mid = (rng.integers(1 << 23, 1 << 24, (1024, 4096)) + 0.5) * d.astype(np.float64)      # exact: 25 + 11 bits
    for e in (rng.uniform(0.5, 16000, (1024, 4096)).astype(F), mid.astype(F), np.nextafter(mid.astype(F), F(0)), np.nextafter(mid.astype(F), F(np.inf))):
        q = e * r
        got = fma(fma(-d, q, e), r, q)
        assert np.array_equal(got.view(np.uint32), (e / d).view(np.uint32))
