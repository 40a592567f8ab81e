"""Expert routing and the combining of the experts' rows on the GPU, each against a plain 64-bit implementation, and
the two around the routing calls they belong to."""
import numpy as np
import pytest
import torch

from block_quantized_matvec_gb300 import mmvq
from tests import _layer
from tests._gpu import dev, host

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
I32 = dict(dtype=torch.int32, device="cuda")


def check_route(logits, k, scoring="softmax", bias=None, n_groups=1, top_groups=None, renormalize=True, scale=1.0):
    """Experts equal.  A weight is exp of a rounded difference (half a unit for each unit of it), two such over a sum
    of up to 1024 in 32 lanes (37 additions) and a quotient: (|x - best| + 64) half units."""
    status = torch.zeros(1, **I32)
    ids, w = mmvq.route_topk(logits, k, scoring=scoring, bias=bias, n_groups=n_groups, top_groups=top_groups,
                             renormalize=renormalize, scale=scale, status=status)
    x = logits.double().cpu().numpy()
    want, ww = _layer.route(x, k, scoring, None if bias is None else bias.double().cpu().numpy(), n_groups,
                            n_groups if top_groups is None else top_groups, renormalize, scale)
    ids, w = host(ids), host(w).astype(np.float64)
    assert np.array_equal(ids, want), np.argwhere(ids != want)[:5]
    far = np.where(np.isfinite(x), x, 0)
    far = 2 * np.abs(far).max(-1, keepdims=True)
    assert (np.abs(w - ww) <= np.abs(ww) * (far + 64) * 2.0 ** -24 + 2.0 ** -126 * (1 + abs(scale))).all()
    assert (w[want < 0] == 0).all()
    assert int(status[0]) == (0 if not (np.isnan(x) | (x == np.inf)).any() else mmvq.ERR_VALUE)
    return ids


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,E,k,groups,top,scoring,bias,renormalize", [
    (1, 1, 1, 1, 1, "softmax", False, True), (5, 7, 7, 1, 1, "sigmoid", False, True), (33, 32, 4, 1, 1, "softmax", False, False),
    (17, 64, 6, 8, 3, "softmax", False, True), (9, 60, 5, 4, 1, "sigmoid", False, False), (301, 256, 8, 8, 4, "sigmoid", True, True),
    (130, 128, 32, 1, 1, "softmax", True, True), (7, 1024, 32, 32, 16, "sigmoid", True, False), (40, 1000, 11, 5, 2, "softmax", True, True),
    (64, 512, 10, 1, 1, "softmax", False, True), (12, 96, 3, 32, 2, "sigmoid", True, True), (6, 300, 12, 3, 3, "sigmoid", True, True),
    (5, 24, 6, 24, 6, "softmax", True, True), (1000, 40, 8, 1, 1, "sigmoid", True, True),
])
def test_route_against_64_bits(dtype, n, E, k, groups, top, scoring, bias, renormalize):
    gen = torch.Generator("cuda").manual_seed(n + E)
    x = (torch.randn((n, E), device="cuda", generator=gen) * 2).to(TYPES[dtype])
    b = torch.randn(E, device="cuda", generator=gen) * 0.2 if bias else None
    check_route(x, k, scoring, b, groups, top, renormalize, 2.5)


def test_equal_logits_go_to_the_lowest_ids():
    for E in (8, 256, 1024):
        x = torch.full((3, E), 0.25, device="cuda", dtype=torch.bfloat16)
        zero = torch.zeros(E, device="cuda")
        k = min(8, E)
        for bias in (None, zero):
            for scoring in ("softmax", "sigmoid"):
                assert np.array_equal(check_route(x, k, scoring, bias), np.tile(np.arange(k, dtype=np.int32), (3, 1)))
                check_route(x, k, scoring, bias, 4, 2) if k <= E // 2 else None
    # coarse logits: many ties in and out of the chosen
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.randint(-3, 4, (200, 256), device="cuda", generator=gen).to(torch.float16)
    for bias in (None, torch.randint(-2, 3, (256,), device="cuda", generator=gen).float() / 4):
        check_route(x, 8, "sigmoid", bias)
        check_route(x, 8, "softmax", bias, 8, 3)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_values_that_32_bits_cannot_tell_apart(scoring):
    """Biases that bring every score to a common value but for differences far below a unit of fp32: the order is
    that of the differences in 64 bits."""
    rng = np.random.default_rng(7)
    for E, groups, top in ((16, 1, 1), (64, 8, 2), (256, 1, 1), (1024, 16, 5)):
        x = torch.from_numpy(rng.normal(size=(40, E)).astype(np.float32))
        xd = x[:1].double().numpy()
        s = 1 / (1 + np.exp(-xd)) if scoring == "sigmoid" else np.exp(xd) / np.exp(xd).sum()
        b = torch.from_numpy((0.75 - s[0]).astype(np.float32))  # row 0: all values 0.75 to within half a unit of the bias
        check_route(x.cuda(), 8, scoring, b.cuda(), groups, top)
        # and logits next to one another
        near = torch.from_numpy(np.float32(1.5) + rng.integers(0, 3, (40, E)).astype(np.float32) * np.float32(2.0 ** -23))
        check_route(near.cuda(), 8, scoring, None, groups, top)
        check_route(near.cuda(), 8, scoring, torch.zeros(E).cuda(), groups, top)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_values_alike_of_scores_that_are_not(scoring):
    """Half of the experts with small scores and exact values, half with large scores that a bias brings to the same
    values: the errors of the second lie between the gaps of the first."""
    rng = np.random.default_rng(11)
    for E in (16, 64, 256):
        x = rng.normal(size=(60, E)).astype(np.float32)
        x[:, ::2] = np.float32(-7) + rng.integers(0, 4, (60, E // 2)).astype(np.float32) * np.float32(2.0 ** -21)
        xd = x.astype(np.float64)
        s = 1 / (1 + np.exp(-xd)) if scoring == "sigmoid" else np.exp(xd) / np.exp(xd).sum(-1, keepdims=True)
        for row in range(0, 60, 12):
            b = np.where(np.arange(E) % 2, s[row, 0] - s[row], 0.0).astype(np.float32)
            check_route(torch.from_numpy(x).cuda(), min(8, E // 2), scoring, torch.from_numpy(b).cuda())
            check_route(torch.from_numpy(x).cuda(), 4, scoring, torch.from_numpy(b).cuda(), 4, 2)


def test_masked_experts_and_rows():
    gen = torch.Generator("cuda").manual_seed(3)
    x = torch.randn((12, 64), device="cuda", generator=gen)
    x[0] = float("-inf")                        # nothing left
    x[1, 3:] = float("-inf")                    # three left, eight asked for
    x[2, ::2] = float("-inf")
    x[3] = -3.4028234663852886e38               # the type's lowest value everywhere
    x[4, 5:] = -3.4028234663852886e38           # and nearly everywhere
    x[5] = -200.0                               # sigmoids that 32 bits have no number for
    x[6] = 200.0 + torch.arange(64, device="cuda")  # and that are all 1
    x[7, :8] = float("-inf")                    # a whole group of eight
    bias = torch.randn(64, device="cuda", generator=gen) * 0.1
    for scoring in ("softmax", "sigmoid"):
        for b in (None, bias):
            for groups, top in ((1, 1), (8, 3)):
                for renormalize in (True, False):
                    ids = check_route(x, 8, scoring, b, groups, top, renormalize)
                    assert (ids[0] == -1).all()
    # what is not a number is never chosen, and said
    x[8, 1], x[9, 2], x[10, 3] = float("nan"), float("inf"), float("-inf")
    for b in (None, bias):
        ids = check_route(x, 8, "sigmoid", b)
        assert not (ids[8] == 1).any() and not (ids[9] == 2).any()
    # biases that keep experts out, or bring them in
    wild = bias.clone()
    wild[5], wild[6], wild[7] = float("-inf"), float("nan"), 1e30
    ids = check_route(x[:8], 4, "sigmoid", wild)
    assert not np.isin(ids, (5, 6)).any() and (ids[3] == 7).any()


def test_route_takes_rows_of_wider_ones_and_other_streams():
    wide = torch.randn((50, 301), device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    for dtype in TYPES.values():
        check_route(wide.to(dtype)[:, 7:263], 8, "softmax")
        check_route(wide.to(dtype)[::3, 1:257], 8, "sigmoid", torch.zeros(256, device="cuda"), 8, 4)
    x = wide[:, :256].contiguous()
    want = mmvq.route_topk(x, 8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = mmvq.route_topk(x, 8, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert mmvq.route_topk(x[:0], 8)[0].shape == (0, 8)


def test_route_writes_nothing_beside_its_outputs():
    for n, E, k in ((3, 40, 5), (1, 1000, 32), (6, 8, 1)):
        x = torch.randn((n, E), device="cuda", generator=torch.Generator("cuda").manual_seed(n))
        ids, w = mmvq.route_topk(x, k)
        rooms = [torch.full((n * k + 64,), -7, dtype=t.dtype, device="cuda") for t in (ids, w)]
        out = [r[32:32 + n * k].view(n, k) for r in rooms]
        mmvq.route_topk(x, k, out=tuple(out))
        for r, o, t in zip(rooms, out, (ids, w)):
            assert torch.equal(o, t) and bool((r[:32] == -7).all()) and bool((r[-32:] == -7).all())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_more_equal_values_than_a_warp_has_lanes(scoring):
    """Ties of more than 32 experts at the last choice, in and out of groups, and as many choices as there can be."""
    for E, k, groups, top in ((256, 8, 1, 1), (1024, 32, 1, 1), (96, 32, 1, 1), (512, 32, 4, 2), (40, 32, 1, 1), (33, 32, 1, 1)):
        x = torch.zeros((6, E), device="cuda")
        x[1, E // 2:] = 1.0
        x[2, ::3] = -1.0
        x[3, E - 1] = 5.0
        x[4] = (torch.arange(E, device="cuda") // 7).float()
        x[5, :] = float("-inf")
        x[5, E - 3:] = 0.5
        for bias in (None, torch.zeros(E, device="cuda"), (torch.arange(E, device="cuda") % 2) * 0.25):
            check_route(x, k, scoring, bias, groups, top)


# ------------------------------------------------------------------ combine --

def lists(topk, E):
    _, offs, _, slot, _ = mmvq.route_groups(topk, E)
    return offs, slot


def check_combine(y, topk, weights, offs, slot, residual=None, shared=None, gate=None, status=0, **kw):
    """k + 2 products added in fp32, each to half a unit of the largest sum on the way; the gate's exp, sum and
    quotient: (k + 12) half units of the sum of sizes, then one rounding."""
    st = torch.zeros(1, **I32)
    keep = [None if t is None else t.double().cpu().numpy() for t in (residual, shared)]
    got = mmvq.combine_experts(y, topk, weights, offs, slot, residual=residual, shared=shared, shared_gate=gate, status=st, **kw)
    want, size = _layer.combine(host(y), host(topk), host(weights), host(offs), host(slot), *keep,
                                None if gate is None else host(gate), y.shape[1])
    info = torch.finfo(got.dtype)
    bound = size * (topk.shape[1] + 12) * 2.0 ** -24
    bound = bound + (np.abs(want) + bound) * info.eps / 2 + info.smallest_normal * info.eps
    err = np.abs(host(got.double()) - want)
    assert (err <= bound).all(), (err / bound).max()
    assert int(st[0]) == status
    return got


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,k,E,H", [(1, 1, 1, 1), (1, 8, 256, 2560), (8, 8, 256, 2560), (37, 3, 5, 33), (5, 10, 16, 1030),
                                     (129, 4, 60, 514), (300, 6, 6, 96), (3, 64, 64, 40)])
def test_combine_against_64_bits(dtype, n, k, E, H):
    gen = torch.Generator("cuda").manual_seed(n + H)
    topk = torch.rand((n, E), device="cuda", generator=gen).argsort(1)[:, :k].to(torch.int32).contiguous()
    offs, slot = lists(topk, E)
    y, w = torch.randn((n * k, H), device="cuda", generator=gen), torch.rand((n, k), device="cuda", generator=gen)
    r, s = (torch.randn((n, H), device="cuda", generator=gen).to(TYPES[dtype]) for _ in range(2))
    g = torch.randn(n, device="cuda", generator=gen) * 4
    got = check_combine(y, topk, w, offs, slot, r, s, g)
    assert got.dtype == TYPES[dtype]
    check_combine(y, topk, w, offs, slot, r)
    check_combine(y, topk, w, offs, slot, None, s)
    check_combine(y, topk, w, offs, slot, dtype=TYPES[dtype])


def test_the_same_expert_twice_and_experts_without_tokens():
    gen = torch.Generator("cuda").manual_seed(9)
    topk = torch.randint(0, 3, (40, 5), generator=gen, **I32) * 4  # 0, 4 and 8 of twelve, each token some of them twice
    offs, slot = lists(topk, 12)
    y, w = torch.randn((200, 130), device="cuda", generator=gen), torch.randn((40, 5), device="cuda", generator=gen)
    check_combine(y, topk, w, offs, slot)
    one = torch.zeros((8192, 8), **I32)  # all slots there are, of one expert
    offs, slot = lists(one, 1)
    y, w = torch.randn((65536, 12), device="cuda", generator=gen), torch.randn((8192, 8), device="cuda", generator=gen)
    check_combine(y, one, w, offs, slot)


def test_slots_without_an_expert_and_lists_that_do_not_fit():
    gen = torch.Generator("cuda").manual_seed(10)
    n, k, E, H = 21, 4, 9, 70
    topk = torch.rand((n, E), device="cuda", generator=gen).argsort(1)[:, :k].to(torch.int32).contiguous()
    topk[3, 1] = topk[4, :] = topk[20, 3] = -1
    offs, slot = lists(topk, E)
    y, w = torch.randn((n * k, H), device="cuda", generator=gen), torch.randn((n, k), device="cuda", generator=gen)
    y[int(offs[E]):] = float("nan")  # rows that no slot stands for
    r = torch.randn((n, H), device="cuda", generator=gen)
    got = check_combine(y, topk, w, offs, slot, r)
    assert torch.equal(got[4], r[4])
    wrong = topk.clone()
    wrong[5, 2], wrong[6, 0] = E, -7            # no such experts
    ok = lists(wrong, E)
    check_combine(y, wrong, w, *ok, r, status=mmvq.ERR_ROUTING)
    # lists of another batch, and lists that are none: the slots that they do not hold add nothing
    other = lists(torch.zeros_like(topk), E)
    st = torch.zeros(1, **I32)
    a = mmvq.combine_experts(y.nan_to_num(), topk, w, *other, residual=r, status=st)
    assert int(st[0]) == mmvq.ERR_ROUTING and bool(torch.isfinite(a).all())
    junk = torch.tensor([-5, 10 ** 9, 3, 7, -2 ** 31, 2 ** 31 - 1, 50, 1, 2, 84], **I32), torch.full_like(slot, 2 ** 31 - 1)
    assert torch.equal(mmvq.combine_experts(y.nan_to_num(), topk, w, *junk, residual=r, status=st), r)
    # fewer rows than the lists say
    st.zero_()
    few = mmvq.combine_experts(y[:10].contiguous(), topk, w, offs, slot, residual=r, status=st)
    assert int(st[0]) == mmvq.ERR_ROUTING
    part = torch.zeros((n * k, H), device="cuda")
    part[:10] = y[:10]
    check = mmvq.combine_experts(part, topk, w, offs, slot, residual=r)
    assert torch.equal(few, check)


def test_combine_strides_and_places():
    gen = torch.Generator("cuda").manual_seed(11)
    n, k, E, H = 13, 4, 20, 260
    topk = torch.rand((n, E), device="cuda", generator=gen).argsort(1)[:, :k].to(torch.int32).contiguous()
    offs, slot = lists(topk, E)
    y, w = torch.randn((n * k, H), device="cuda", generator=gen), torch.randn((n, k), device="cuda", generator=gen)
    for dtype in TYPES.values():
        wide = torch.randn((2, n, 300), device="cuda", generator=gen).to(dtype)
        for first in (0, 3, 8):
            r, s = wide[0][:, first:first + H], wide[1][:, first + 5:first + 5 + H]
            want = check_combine(y, topk, w, offs, slot, r, s)
            for place in (0, 1):
                there = wide.clone()
                x = (there[0][:, first:first + H], there[1][:, first + 5:first + 5 + H])
                got = mmvq.combine_experts(y, topk, w, offs, slot, residual=x[0], shared=x[1], out=x[place])
                assert torch.equal(got, want)
                x[place].copy_((r, s)[place])
                assert torch.equal(there, wide)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = mmvq.combine_experts(y, topk, w, offs, slot, residual=r, shared=s, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    none = torch.zeros((0, k), **I32)
    assert mmvq.combine_experts(y, none, w[:0], offs, slot).shape == (0, H)


def test_a_prompts_tokens_through_routing_products_and_combining():
    """route_topk, the expert layer with its lists, combining."""
    from block_quantized_matvec_gb300 import synth
    gen = torch.Generator("cuda").manual_seed(12)
    n, E, k, H, F = 8, 16, 4, 256, 256
    W_gu, W_dn = synth.expert_weights("q4_k", E, 2 * F, H, salt=5), synth.expert_weights("q4_k", E, H, F, salt=6)
    planar = lambda W: torch.cat([mmvq.repack_planar(dev(W[e]), W.shape[1], W.shape[2] * 256, type_=mmvq.TYPE_Q4_K) for e in range(E)])  # noqa: E731
    gu, dn = planar(W_gu), planar(W_dn)
    x = dev(synth.moe_hidden(H, n, salt=5))
    logits = torch.randn((n, E), device="cuda", generator=gen)
    logits[2, 5:] = float("-inf")
    ids, w = mmvq.route_topk(logits, k, scoring="sigmoid", bias=torch.randn(E, device="cuda", generator=gen), n_groups=4, top_groups=2)
    out = mmvq.expert_ffn(mmvq.TYPE_Q4_K_PLANAR, gu, dn, E, H, F, x, ids)
    assert bool(torch.isfinite(out["y"]).all())
    check_combine(out["y"], ids, w, out["offsets"], out["slot_of"], x)


def test_graph_replay_with_new_logits():
    n, E, k, H = 4, 32, 4, 96
    x, y, r = torch.randn((n, E), device="cuda"), torch.randn((n * k, H), device="cuda"), torch.randn((n, H), device="cuda")
    out = (torch.empty((n, k), **I32), torch.empty((n, k), device="cuda"))

    def step():
        ids, w = mmvq.route_topk(x, k, out=out)
        _, offs, _, slot, _ = mmvq.route_groups(ids, E)
        return mmvq.combine_experts(y, ids, w, offs, slot, residual=r)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(3):
        x.normal_(), y.normal_()
        g.replay()
        have = got.clone()
        assert torch.equal(have, step())
