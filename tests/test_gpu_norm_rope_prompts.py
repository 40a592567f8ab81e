"""Head norm with rotation of many tokens on the GPU, where a warp takes several steps of a token's heads, against a
plain 64-bit implementation at tokens of the beginning, the end and between."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_gb300 import mmvq
from tests import _layer
from tests._gpu import host

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
I32 = dict(dtype=torch.int32, device="cuda")


def check(got, x, weight, eps, positions, f, axis_of, interleaved):
    """A lane adds 16 squares (8 of them at most where they are fp32), its row's lanes 5 times more: 21 roundings of the
    sum, halved by the root; division, eps, root (2), the weight's two products, sine and cosine (2 ulp: 4 half units), the
    rotation's 3: below 32 half units of the pair's size, 2^-19; then one rounding to the type."""
    want, size = _layer.norm_rope(x.double().cpu().numpy(), None if weight is None else weight.cpu().numpy(), eps,
                                  positions.cpu().numpy(), f, axis_of, 2 * len(f), interleaved)
    info = torch.finfo(got.dtype)
    bound = size * 2.0 ** -19 + (np.abs(want) + size * 2.0 ** -19) * info.eps / 2 + info.smallest_normal * info.eps
    err = np.abs(host(got.double()) - want)
    assert (err <= bound).all(), (err / bound).max()


# head_dim, turning, neighbours, query heads, key heads, tokens; a step is 64 * V / head_dim heads of one tensor (V: 8 of
# 16 bits, 4 of 32), and from 3648 steps in all on a warp has several
SHAPES = [
    (64, 64, False, 40, 8, 911), (64, 32, False, 61, 3, 1201), (64, 64, True, 33, 17, 777), (64, 6, True, 70, 9, 601),
    (128, 128, False, 32, 8, 541), (128, 64, False, 29, 3, 1013), (128, 128, True, 40, 40, 301), (128, 50, True, 23, 5, 700),
    (256, 256, False, 33, 2, 499), (256, 64, False, 24, 2, 1021), (256, 256, True, 17, 16, 400), (256, 98, True, 24, 1, 509),
    (256, 128, False, 24, 0, 620), (128, 128, False, 1024, 512, 11), (128, 128, False, 4, 2, 7001),
]


def sample(n):
    return sorted({0, 1, n // 3, n // 2, n - 2, n - 1})


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim,rot,interleaved,heads,kv,n", SHAPES)
def test_prompts_against_64_bits(dtype, dim, rot, interleaved, heads, kv, n):
    V = 4 if dtype == "f32" else 8
    rows = 64 * V // dim
    assert (-(-heads // rows) + -(-kv // rows)) * n > 3648
    gen = torch.Generator("cuda").manual_seed(dim + rot + n)
    q = (torch.randn((n, heads, dim), device="cuda", generator=gen) * 3).to(TYPES[dtype])
    k = (torch.randn((n, kv, dim), device="cuda", generator=gen) * 0.01).to(TYPES[dtype])
    wq, wk = (torch.rand(dim, device="cuda", generator=gen) + s for s in (0.5, 4.0))
    f = [1e4 ** (-2 * i / rot) for i in range(rot // 2)]
    axis_of = [i % 2 for i in range(rot // 2)]
    pos = torch.randint(0, 200000, (2, n), generator=gen, **I32)
    tab = mmvq.rope_table(f, axis_of=axis_of)
    args = dict(q_weight=wq, k_weight=wk, eps=1e-5, interleaved=interleaved)
    yq, yk = mmvq.norm_rope(q, k, pos, tab, **args)
    at = sample(n)
    for y, x, w in ((yq, q, wq), (yk, k, wk)):
        check(y[at], x[at], w, 1e-5, pos[:, at], f, axis_of, interleaved)
    # every token's result is that of the token by itself, where a warp has one step: all of them, bit by bit
    for lo in range(0, n, n // 3):
        part = slice(lo, min(n, lo + max(1, 3648 // (heads + kv))))
        a, b = mmvq.norm_rope(q[part], k[part], pos[:, part], tab, **args)
        assert torch.equal(a, yq[part]) and torch.equal(b, yk[part])
    # over its inputs, and without norm
    both = q.clone(), k.clone()
    got = mmvq.norm_rope(*both, pos, tab, out=both, **args)
    assert got[0] is both[0] and torch.equal(both[0], yq) and torch.equal(both[1], yk)
    yq, yk = mmvq.norm_rope(q, k, pos, tab, eps=None, interleaved=interleaved)
    for y, x in ((yq, q), (yk, k)):
        check(y[at], x[at], None, None, pos[:, at], f, axis_of, interleaved)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_a_prompts_heads_in_wider_rows(dtype):
    """Queries next to their gates, keys among values; nothing beside the heads is written."""
    n, f = 801, [1e4 ** (-2 * i / 128) for i in range(64)]
    gen = torch.Generator("cuda").manual_seed(1)
    rows = torch.randn((n, 50, 256), device="cuda", generator=gen).to(TYPES[dtype])
    pos = torch.arange(n, **I32)[None]
    tab = mmvq.rope_table(f)
    q, k = rows[:, :40, :128], rows[:, 40:49:2, 128:]
    want = mmvq.norm_rope(q.contiguous(), k.contiguous(), pos, tab)
    at = sample(n)
    check(want[0][at], q[at], None, 1e-6, pos[:, at], f, [0] * 64, False)
    check(want[1][at], k[at], None, 1e-6, pos[:, at], f, [0] * 64, False)
    there = rows.clone()
    place = there[:, :40, :128], there[:, 40:49:2, 128:]
    mmvq.norm_rope(*place, pos, tab, out=place)
    assert torch.equal(place[0], want[0]) and torch.equal(place[1], want[1])
    place[0].copy_(q), place[1].copy_(k)
    assert torch.equal(there, rows)
    there = torch.full_like(rows, -7)
    place = there[:, :40, :128], there[:, 40:49:2, 128:]
    mmvq.norm_rope(q, k, pos, tab, out=place)
    assert torch.equal(place[0], want[0]) and torch.equal(place[1], want[1])
    place[0].fill_(-7), place[1].fill_(-7)
    assert bool((there == -7).all())
