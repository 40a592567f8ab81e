"""Head norm with rotation on the GPU against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_gb300 import mmvq
from tests import _layer
from tests._gpu import host

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
I32 = dict(dtype=torch.int32, device="cuda")


def freqs(rot, base=1e4):
    return [base ** (-2 * i / rot) for i in range(rot // 2)]


def check(got, x, weight, eps, positions, f, axis_of, interleaved):
    """The statistics in fp32 (13 additions of a lane and its warp, halved by the root; the root, the weight and the
    product: 12 half units), sine and cosine (4) and the rotation (3) stay below 2^-19 of the pair; then one rounding."""
    want, size = _layer.norm_rope(x.double().cpu().numpy(), None if weight is None else weight.cpu().numpy(), eps,
                                  np.atleast_2d(positions.cpu().numpy()), f, axis_of, 2 * len(f), interleaved)
    info = torch.finfo(got.dtype)
    bound = size * 2.0 ** -19 + (np.abs(want) + size * 2.0 ** -19) * info.eps / 2 + info.smallest_normal * info.eps
    err = np.abs(host(got.double()) - want)
    assert got.shape == x.shape and (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim,rot,interleaved,heads,kv,n", [
    (64, 64, False, 3, 1, 1), (64, 2, True, 1, 1, 7), (64, 18, False, 12, 12, 33), (128, 128, False, 8, 2, 65),
    (128, 32, True, 5, 3, 9), (128, 126, False, 2, 1, 11), (256, 64, False, 24, 2, 5), (256, 256, True, 2, 2, 17), (256, 6, False, 1, 4, 3),
    (256, 254, False, 1, 1, 40), (64, 64, True, 40, 8, 161),
])
def test_against_64_bits(dtype, dim, rot, interleaved, heads, kv, n):
    gen = torch.Generator("cuda").manual_seed(dim + rot + n)
    q = (torch.randn((n, heads, dim), device="cuda", generator=gen) * 3).to(TYPES[dtype])
    k = (torch.randn((n, kv, dim), device="cuda", generator=gen) * 0.01).to(TYPES[dtype])
    k[0] = 0  # a head of zeros stays one
    wq, wk = (torch.rand(dim, device="cuda", generator=gen) + 0.5 for _ in range(2))
    pos = torch.randint(0, 200000, (n,), generator=gen, **I32)
    f = freqs(rot)
    status = torch.zeros(1, **I32)
    yq, yk = mmvq.norm_rope(q, k, pos, mmvq.rope_table(f), q_weight=wq, k_weight=wk, eps=1e-5, interleaved=interleaved, status=status)
    assert yq.is_contiguous() and yq.dtype == q.dtype
    check(yq, q, wq, 1e-5, pos, f, [0] * (rot // 2), interleaved)
    check(yk, k, wk, 1e-5, pos, f, [0] * (rot // 2), interleaved)
    assert int(status[0]) == 0


@pytest.mark.parametrize("axis_of", [[0] * 12 + [1] * 10 + [2] * 10, [i % 3 for i in range(32)], [3, 1] * 16])
def test_several_axes(axis_of):
    gen = torch.Generator("cuda").manual_seed(5)
    n = 29
    q = torch.randn((n, 4, 128), device="cuda", generator=gen)
    pos = torch.randint(-50, 5000, (4, 64), generator=gen, **I32)[:, 3:3 + n]  # rows of a larger array, some before zero
    f = freqs(64)
    yq, yk = mmvq.norm_rope(q, None, pos, mmvq.rope_table(f, axis_of=axis_of))
    assert yk is None
    check(yq, q, None, 1e-6, pos, f, axis_of, False)
    one = mmvq.rope_table(f, sections=(12, 10, 10)), mmvq.rope_table(f, axis_of=[0] * 12 + [1] * 10 + [2] * 10)
    assert torch.equal(*one)
    # the same positions on every axis turn as one axis does
    same = pos[:1].expand(4, n)
    assert torch.equal(mmvq.norm_rope(q, None, same, mmvq.rope_table(f, axis_of=axis_of))[0],
                       mmvq.norm_rope(q, None, pos[0], mmvq.rope_table(f))[0])


def test_far_positions_keep_their_angles():
    """Up to the ends of int32 and at frequencies of 1 and more, whose turns 32 bits would lose altogether."""
    pos = torch.tensor([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 123456789, 2 ** 30 + 12345], **I32)
    f = [1.0, 0.3, 7.25, 1e-3, 2 ** -20, 100.1, 1e-9, 0.0, -0.7, 3.0] + freqs(44)
    q = torch.randn((8, 3, 64), device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    y, _ = mmvq.norm_rope(q, None, pos, mmvq.rope_table(f), eps=None)
    check(y, q, None, None, pos, f, [0] * 32, False)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_strides_gates_and_places(dtype):
    """Queries next to their gates, heads of one wide row, rows that no 16-byte load may start at, a head shared by
    all, and results over their inputs."""
    gen = torch.Generator("cuda").manual_seed(3)
    n, f = 19, freqs(96)
    tab = mmvq.rope_table(f)
    pos = torch.randint(0, 9000, (n,), generator=gen, **I32)
    rows = (torch.randn((n, 6, 300), device="cuda", generator=gen)).to(TYPES[dtype])
    gated, odd = rows[:, :4, :128], rows[:, ::2, 3:131]
    shared = rows[:, :1, 16:144].expand(-1, 5, -1)
    for q in (gated, odd, shared):
        y, yk = mmvq.norm_rope(q, rows[:, 4:, 8:136], pos, tab)
        check(y, q, None, 1e-6, pos, f, [0] * 48, False)
        check(yk, rows[:, 4:, 8:136], None, 1e-6, pos, f, [0] * 48, False)
    for q in (gated, odd):
        there = rows.clone()
        place = torch.as_strided(there, q.shape, q.stride(), q.storage_offset())
        y, _ = mmvq.norm_rope(place, None, pos, tab, out=(place, None))
        assert y.data_ptr() == place.data_ptr()
        check(y, q, None, 1e-6, pos, f, [0] * 48, False)
        torch.as_strided(there, q.shape, q.stride(), q.storage_offset()).copy_(q)
        assert torch.equal(there, rows)  # nothing beside the heads was written


def test_values_that_are_not_finite_stay_in_their_head():
    f = freqs(64)
    q = torch.randn((4, 6, 64), device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    pos = torch.arange(4, **I32)
    want, _ = mmvq.norm_rope(q, None, pos, mmvq.rope_table(f))
    q[1, 2, 5], q[2, 0, 63], q[3, 5, 0] = float("nan"), float("inf"), float("-inf")
    got, _ = mmvq.norm_rope(q, None, pos, mmvq.rope_table(f))
    hit = torch.zeros((4, 6), dtype=torch.bool, device="cuda")
    hit[1, 2] = hit[2, 0] = hit[3, 5] = True
    assert torch.equal(got[~hit], want[~hit]) and bool(torch.isnan(got[1, 2]).all())


def test_a_wrong_axis_is_reported_and_leaves_its_pairs():
    q = torch.randn((3, 2, 64), device="cuda", generator=torch.Generator("cuda").manual_seed(6))
    pos = torch.arange(1, 4, **I32)
    tab = mmvq.rope_table(freqs(64), axis_of=[0] * 30 + [1, 2])
    status = torch.zeros(1, **I32)
    y, _ = mmvq.norm_rope(q, None, pos, tab, eps=None, status=status)
    assert int(status[0]) == mmvq.ERR_SHAPE
    assert torch.equal(y[..., [30, 31, 62, 63]], q[..., [30, 31, 62, 63]]) and not torch.equal(y[..., 29], q[..., 29])


def test_no_tokens_and_another_stream():
    tab = mmvq.rope_table(freqs(64))
    q = torch.randn((0, 2, 64), device="cuda")
    assert mmvq.norm_rope(q, q, torch.zeros(0, **I32), tab)[1].shape == (0, 2, 64)
    q, pos = torch.randn((700, 24, 64), device="cuda"), torch.arange(700, **I32)
    want, _ = mmvq.norm_rope(q, None, pos, tab)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, _ = mmvq.norm_rope(q, None, pos, tab, stream=side)
    with torch.cuda.stream(side):
        again, _ = mmvq.norm_rope(q, None, pos, tab)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(again, want)


def test_graph_replay_with_new_inputs():
    tab, n = mmvq.rope_table(freqs(128)), 6
    q, k, pos = torch.randn((n, 8, 128), device="cuda"), torch.randn((n, 2, 128), device="cuda"), torch.arange(n, **I32)
    out = torch.empty_like(q), torch.empty_like(k)
    mmvq.norm_rope(q, k, pos, tab, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mmvq.norm_rope(q, k, pos, tab, out=out)
    for i in range(3):
        q.normal_(), k.normal_(), pos.add_(1000)
        g.replay()
        for a, b in zip(out, mmvq.norm_rope(q, k, pos, tab)):
            assert torch.equal(a, b)
