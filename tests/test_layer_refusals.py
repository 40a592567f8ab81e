"""norm_rope refuses rows that would be written over one another.  On the CPU: nothing is launched."""
import itertools

import pytest
import torch

from block_quantized_matvec_gb300 import build, mmvq
from tests.test_kv4_binding import tensor
from tests.test_layer_binding import ROPE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mmvq.lib()


def overlap(ld, h, n, heads, dim):
    """Whether two of the rows share a value, by trying all."""
    at = sorted(t * ld + i * h for t in range(n) for i in range(heads))
    return any(b - a < dim for a, b in zip(at, at[1:]))


def test_rows_that_would_be_written_twice_are_refused(lib):
    """Every layout of a few tokens and heads: refused where rows overlap and nowhere else.  (q is NULL, which is looked
    at after the shapes, so that nothing can be launched.)"""
    seen = set()
    for n, heads in itertools.product((1, 2, 3, 5), (1, 2, 3, 7)):
        for ld, h in itertools.product((0, 64, 100, 128, 129, 192, 256, 320, 384, 448, 640, 1024), repeat=2):
            bad = overlap(ld, h, n, heads, 64)
            want = mmvq.ERR_SHAPE if bad else mmvq.ERR_NULL
            one = dict(ROPE, q=None, head_dim=64, rot_dim=32, n_tokens=n, n_heads=heads, n_kv_heads=0, ldyq=ld, hyq=h)
            assert lib.mmvq_norm_rope(*one.values()) == want, (n, heads, ld, h)
            one = dict(ROPE, q=None, head_dim=64, rot_dim=32, n_tokens=n, n_heads=1, n_kv_heads=heads, ldyq=64, hyq=64, ldyk=ld, hyk=h)
            assert lib.mmvq_norm_rope(*one.values()) == want, (n, heads, ld, h)
            seen.add((bad, n > 1 and heads > 1))
    assert len(seen) == 4
    far = dict(ROPE, q=None, n_tokens=2 ** 21, n_heads=1024, n_kv_heads=0, ldyq=2 ** 62, hyq=2 ** 62)  # products beyond 64 bits
    assert lib.mmvq_norm_rope(*far.values()) == mmvq.ERR_SHAPE
    far.update(hyq=128)
    assert lib.mmvq_norm_rope(*far.values()) == mmvq.ERR_NULL


def test_the_binding_refuses_such_an_out(lib, monkeypatch):
    monkeypatch.setattr(mmvq, "_current_device", lambda: 0)
    monkeypatch.setattr(mmvq, "_stream", lambda s: None)
    monkeypatch.setattr(mmvq, "_raw_stream", None)
    f32 = torch.float32
    q, k, pos, table = tensor((3, 4, 64), f32), tensor((3, 2, 64), f32), tensor((3,), torch.int32), tensor((2, 16), torch.int64)
    room = tensor((3 * 4 * 64,), f32)
    twice = room.as_strided((3, 4, 64), (64, 64, 1))
    for args in ((q, None, twice, None), (q, q, q.clone().as_subclass(type(q)), twice), (k, q, k, twice)):
        with pytest.raises(mmvq.MMVQError) as e:
            mmvq.norm_rope(args[0], args[1], pos, table, out=args[2:])
        assert e.value.code == mmvq.ERR_SHAPE
