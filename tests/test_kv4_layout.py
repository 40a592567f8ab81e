"""The 4-bit key/value cache's format and layout on the CPU (the plain implementation that the
GPU tests compare with), the sizes the library reports, and its refusals before any CUDA call."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_gb300 import build, mmvq
from tests import _kv4


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mmvq.lib()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_every_bit_of_a_tile_has_one_owner(D):
    kb, ksh, vb, vsh, ks, vs = _kv4.places(D)
    used = np.zeros(20 * D * 8, int)
    owner = {}
    for t in range(16):
        for by, sh in ((kb[t], ksh[t]), (vb[t], vsh[t])):
            for i in range(D):
                used[8 * by[i] + sh[i]:8 * by[i] + sh[i] + 4] += 1
                assert owner.setdefault(int(by[i]), t) == t  # no two tokens share a byte
        for s in (ks[t], vs[t]):
            for x in s:
                used[8 * x:8 * x + 16] += 1
                used[8 * (x + D):8 * (x + D) + 16] += 1
    assert (used == 1).all()


def test_put_and_get_are_inverse():
    rng = np.random.default_rng(1)
    D = 128
    tile = np.full(20 * D, 0xff, np.uint8)
    toks = [tuple(_kv4.quantise(rng.normal(size=D)) for _ in range(2)) for _ in range(16)]
    for t in rng.permutation(16):
        _kv4.put(tile, t, D, *toks[t])
    k, v = _kv4.get(tile[None], D)
    for t in range(16):
        for got, want in ((k, toks[t][0]), (v, toks[t][1])):
            for g, w in zip(got, want):
                assert np.array_equal(g[0, t], w)


def test_format_values():
    x = np.linspace(-3, 3, 32)
    c, d, z = _kv4.quantise(x)
    assert d[0] == np.float16(0.4) and z[0] == 0 and c[0] == 0 and c[31] == 15
    assert np.abs(_kv4.values(c, d, z) - x).max() <= 0.2 * 1.01
    c, d, z = _kv4.quantise(np.full(32, 1.5))     # a constant block: its midpoint
    assert d[0] == 0 and z[0] == 1.5 and not c.any() and (_kv4.values(c, d, z) == 1.5).all()
    c, d, z = _kv4.quantise(np.full(32, np.inf))
    assert z[0] == 65504
    x = np.zeros(32)
    x[3] = np.nan
    assert (_kv4.quantise(x)[2] == 0).all()


def test_sizes(lib):
    assert mmvq.kv4_page_bytes(2, 256, 64) == 2 * 4 * 20 * 256
    assert mmvq.kv4_page_bytes(8, 128, 16) * 8 == 8 * 128 * 16 * 2 * 5  # 5 bits a value, keys and values
    for bad in ((0, 128, 64), (8, 96, 64), (8, 128, 0), (8, 128, 24), (1025, 128, 64), (8, 128, 1 << 17)):
        with pytest.raises(mmvq.MMVQError):
            mmvq.kv4_page_bytes(*bad)
    for D in (64, 128, 256):
        assert lib.mmvq_kv4_attention_workspace_bytes(D) > 0
    assert lib.mmvq_kv4_attention_workspace_bytes(96) == -1


A = 0x10000  # an aligned fake device address: never dereferenced


def change(base, **kw):
    names = list(base)
    assert set(kw) <= set(names)
    return [kw.get(n, base[n]) for n in names]


CACHE = dict(cache=A, n_pages=4, page=64, kv=2, D=128, table=A, ld=2, offsets=A, lens=A, seqs=3, n=5)
APPEND = dict(dtype=0, k=A, ldk=256, hk=128, v=A, ldv=256, hv=128, **CACHE, status=None, stream=None)
READ = dict(dtype=0, k=A, v=A, **CACHE, status=None, stream=None)
ATTEND = dict(dtype=0, q=A, ldq=1024, hq=128, heads=8, scale=0.1, window=0, sinks=0, y=A, lse=None, **CACHE,
              workspace=A, status=None, stream=None)
COMMON = [(dict(dtype=14), mmvq.ERR_TYPE), (dict(dtype=2), mmvq.ERR_TYPE), (dict(cache=None), mmvq.ERR_NULL),
          (dict(table=None), mmvq.ERR_NULL), (dict(offsets=None), mmvq.ERR_NULL), (dict(lens=None), mmvq.ERR_NULL),
          (dict(D=96), mmvq.ERR_SHAPE), (dict(D=0), mmvq.ERR_SHAPE), (dict(page=40), mmvq.ERR_SHAPE),
          (dict(page=0), mmvq.ERR_SHAPE), (dict(n_pages=0), mmvq.ERR_SHAPE), (dict(n_pages=1 << 31), mmvq.ERR_SHAPE),
          (dict(ld=0), mmvq.ERR_SHAPE), (dict(ld=1 << 26), mmvq.ERR_SHAPE), (dict(seqs=0), mmvq.ERR_SHAPE),
          (dict(seqs=4097), mmvq.ERR_SHAPE), (dict(n=-1), mmvq.ERR_SHAPE), (dict(cache=A + 8), mmvq.ERR_ALIGN),
          (dict(table=A + 2), mmvq.ERR_ALIGN), (dict(lens=A + 1), mmvq.ERR_ALIGN), (dict(status=A + 2), mmvq.ERR_ALIGN)]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(kv=0), mmvq.ERR_SHAPE), (dict(k=None), mmvq.ERR_NULL), (dict(v=None), mmvq.ERR_NULL),
    (dict(ldk=-1), mmvq.ERR_SHAPE), (dict(hv=-128), mmvq.ERR_SHAPE), (dict(k=A + 2), mmvq.ERR_ALIGN),
    (dict(dtype=1, v=A + 1), mmvq.ERR_ALIGN), (dict(n=0), mmvq.OK), (dict(n=0, k=None, v=None), mmvq.OK)])
def test_append_rejects_on_host(lib, kw, code):
    assert lib.mmvq_kv4_append(*change(APPEND, **kw)) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(kv=0), mmvq.ERR_SHAPE), (dict(k=None), mmvq.ERR_NULL), (dict(v=A + 8), mmvq.ERR_ALIGN), (dict(n=0), mmvq.OK)])
def test_read_rejects_on_host(lib, kw, code):
    assert lib.mmvq_kv4_read(*change(READ, **kw)) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(q=None), mmvq.ERR_NULL), (dict(y=None), mmvq.ERR_NULL), (dict(workspace=None), mmvq.ERR_NULL),
    (dict(heads=7), mmvq.ERR_SHAPE), (dict(heads=0), mmvq.ERR_SHAPE), (dict(heads=258), mmvq.ERR_SHAPE),
    (dict(window=-1), mmvq.ERR_SHAPE), (dict(sinks=-1), mmvq.ERR_SHAPE), (dict(scale=float("nan")), mmvq.ERR_SHAPE),
    (dict(scale=float("inf")), mmvq.ERR_SHAPE), (dict(ldq=-1), mmvq.ERR_SHAPE), (dict(n=25), mmvq.ERR_NCOLS),
    (dict(y=A + 8), mmvq.ERR_ALIGN), (dict(q=A + 2), mmvq.ERR_ALIGN), (dict(lse=A + 2), mmvq.ERR_ALIGN),
    (dict(workspace=A + 128), mmvq.ERR_ALIGN), (dict(n=0), mmvq.OK)])
def test_attention_rejects_on_host(lib, kw, code):
    assert lib.mmvq_kv4_attention(*change(ATTEND, **kw)) == code


def test_binding_rejects_tensors_that_are_not_a_batch():
    cpu = torch.zeros((2, 2, 4, 2560), dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        mmvq.kv4_read(cpu, i32(1, 2), i32(2), i32(1), 1)
    assert "clamped" in mmvq.strerror(mmvq.ERR_VALUE)
