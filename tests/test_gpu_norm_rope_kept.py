"""Values that the rotation does not turn, on the GPU: they stay as they are whatever stands in their neighbours."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_gb300 import mmvq
from tests import _layer
from tests._gpu import host

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
I32 = dict(dtype=torch.int32, device="cuda")
INF, NAN = float("inf"), float("nan")


def same(got, want):
    """Equal, NaN in the same places, zeros of the same sign."""
    g, w = host(got.double()), np.asarray(want, np.float64)
    num = ~np.isnan(w)
    assert np.array_equal(np.isnan(g), np.isnan(w)) and np.array_equal(g[num], w[num])
    assert np.array_equal(np.signbit(g[num]), np.signbit(w[num]))


def heads(n, dim, dtype, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    q = torch.randn((n, 5, dim), device="cuda", generator=gen)
    wild = torch.rand(q.shape, device="cuda", generator=gen)
    for i, x in enumerate((INF, -INF, NAN, 0.0, -0.0)):
        q[(wild > i * 0.04) & (wild < i * 0.04 + 0.04)] = x
    return q.to(TYPES[dtype])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim,rot,interleaved", [(64, 16, False), (128, 64, False), (256, 64, False), (256, 128, False), (64, 18, False), (128, 6, False),
                                                 (64, 8, True), (64, 2, True), (128, 74, True), (256, 100, True)])
@pytest.mark.parametrize("n", [3, 900])
def test_values_behind_the_turning_ones_stay(dtype, dim, rot, interleaved, n):
    q = heads(n, dim, dtype, dim + rot)
    f = [1e4 ** (-2 * i / rot) for i in range(rot // 2)]
    y, _ = mmvq.norm_rope(q, None, torch.arange(1, n + 1, **I32), mmvq.rope_table(f), eps=None, interleaved=interleaved)
    same(y[..., rot:], host(q.double())[..., rot:])
    # what turns is finite where both of the pair are
    x = host(q.double())[..., :rot]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:])
    g = host(y.double())[..., :rot]
    ga = g[..., 0::2] if interleaved else g[..., :rot // 2]
    ok = np.isfinite(a) & np.isfinite(b)
    assert np.isfinite(ga[ok]).all() and not np.isfinite(ga[np.isnan(a) | np.isnan(b)]).any()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim,rot,interleaved", [(64, 64, False), (128, 64, False), (64, 18, False), (64, 64, True), (256, 30, True)])
def test_pairs_of_no_axis_stay(dtype, dim, rot, interleaved):
    n, half = 4, rot // 2
    q = heads(n, dim, dtype, 3)
    axis_of = [i % 2 for i in range(half)]          # axis 1 has no positions
    tab = mmvq.rope_table([1e4 ** (-i / half) for i in range(half)], axis_of=axis_of)
    status = torch.zeros(1, **I32)
    y, _ = mmvq.norm_rope(q, None, torch.arange(1, n + 1, **I32), tab, eps=None, interleaved=interleaved, status=status)
    assert int(status[0]) == mmvq.ERR_SHAPE
    pairs = [(2 * i, 2 * i + 1) if interleaved else (i, i + half) for i in range(half) if axis_of[i]]
    stay = [i for p in pairs for i in p] + list(range(rot, dim))
    same(y[..., stay], host(q.double())[..., stay])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim,rot,interleaved", [(64, 16, False), (256, 64, False), (64, 18, False), (128, 32, True)])
def test_an_infinity_behind_the_turning_ones_under_the_norm(dtype, dim, rot, interleaved):
    """The mean square is infinite: finite values become 0, the infinity itself is no number; nothing else is lost."""
    n = 6
    q = (torch.randn((n, 3, dim), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).abs() + 0.5).to(TYPES[dtype])
    q[:, 1, rot + 1], q[:, 2, dim - 1] = INF, -INF
    w = torch.rand(dim, device="cuda", generator=torch.Generator("cuda").manual_seed(2)) + 0.5
    f = [1e4 ** (-2 * i / rot) for i in range(rot // 2)]
    pos = torch.arange(n, **I32)
    y, _ = mmvq.norm_rope(q, None, pos, mmvq.rope_table(f), q_weight=w, eps=1e-6, interleaved=interleaved)
    want, _ = _layer.norm_rope(q[:, 1:].double().cpu().numpy(), w.cpu().numpy(), 1e-6, pos.cpu().numpy()[None], f, [0] * (rot // 2), rot, interleaved)
    g = host(y.double())
    assert np.array_equal(np.isnan(g[:, 1:]), np.isnan(want)) and np.isnan(want).sum() == 2 * n
    assert (g[:, 1:][~np.isnan(want)] == 0).all() and np.isfinite(g[:, 0]).all()
