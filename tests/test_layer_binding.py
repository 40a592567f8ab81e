"""The layer's steps between the products on the CPU: what the library and the binding refuse before any CUDA call,
on which stream a call's own tensors are made, and the rotation's table."""
import math
from fractions import Fraction

import pytest
import torch

from block_quantized_matvec_gb300 import build, mmvq
from tests import _layer
from tests.test_kv4_binding import Elsewhere, Tensor, tensor

A = 0x10000  # an aligned fake device address: these calls fail before any CUDA call

ROPE = dict(dtype=0, q=A, ldq=512, hq=128, n_heads=4, k=A, ldk=256, hk=128, n_kv_heads=2, head_dim=128, n_tokens=3, positions=A, ld_positions=0,
            n_axes=1, table=A, rot_dim=64, q_weight=None, k_weight=None, eps=1e-6, flags=0, yq=A, ldyq=512, hyq=128, yk=A, ldyk=256, hyk=128,
            status=None, stream=None)
ROUTE = dict(dtype=0, logits=A, ld=64, n_tokens=3, n_experts=64, k=8, scoring=0, bias=None, n_groups=8, top_groups=4, renormalize=1, scale=1.0,
             topk=A, weights=A, status=None, stream=None)
COMBINE = dict(dtype=0, y=A, n_positions=24, H=64, topk=A, weights=A, n_tokens=3, k=8, token_offsets=A, n_experts=64, slot_of=A, residual=A, ldr=64,
               shared=A, lds=64, shared_gate=A, out=A, ldo=64, status=None, stream=None)
LOGPROBS = dict(dtype=0, logits=A, ld=1000, n_rows=3, vocab=1000, scale=1.0, tokens=A, n_tokens=2, top=5, lse=A, entropy=A, logprobs=A, top_ids=A,
                top_logprobs=A, status=None, stream=None)
SHAPE, NULL, ALIGN, TYPE = mmvq.ERR_SHAPE, mmvq.ERR_NULL, mmvq.ERR_ALIGN, mmvq.ERR_TYPE
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mmvq.lib()


@pytest.mark.parametrize("name,base,bad", [
    ("mmvq_norm_rope", ROPE, [
        (dict(dtype=2), TYPE), (dict(q=None), NULL), (dict(yq=None), NULL), (dict(k=None), NULL), (dict(yk=None), NULL), (dict(positions=None), NULL),
        (dict(table=None), NULL), (dict(head_dim=96), SHAPE), (dict(head_dim=0), SHAPE), (dict(n_tokens=-1), SHAPE), (dict(n_heads=0), SHAPE),
        (dict(n_heads=1025), SHAPE), (dict(n_kv_heads=-1), SHAPE), (dict(rot_dim=0), SHAPE), (dict(rot_dim=63), SHAPE), (dict(rot_dim=130), SHAPE),
        (dict(n_axes=0), SHAPE), (dict(n_axes=5), SHAPE), (dict(ld_positions=-1), SHAPE), (dict(ldq=-1), SHAPE), (dict(hk=-1), SHAPE),
        (dict(hyk=-8), SHAPE), (dict(hyq=0), SHAPE), (dict(ldyk=100), SHAPE), (dict(hyk=127), SHAPE), (dict(flags=4), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=NAN), SHAPE), (dict(eps=INF), SHAPE),
        (dict(n_tokens=2 ** 31 - 1), SHAPE), (dict(q=A + 2), ALIGN), (dict(dtype=1, yk=A + 1), ALIGN), (dict(table=A + 4), ALIGN),
        (dict(positions=A + 2), ALIGN), (dict(k_weight=A + 1), ALIGN), (dict(status=A + 1), ALIGN)]),
    ("mmvq_route_topk", ROUTE, [
        (dict(dtype=3), TYPE), (dict(scoring=2), TYPE), (dict(logits=None), NULL), (dict(topk=None), NULL), (dict(weights=None), NULL),
        (dict(n_tokens=-1), SHAPE), (dict(n_experts=0), SHAPE), (dict(n_experts=1025, ld=1025, n_groups=1, top_groups=1), SHAPE), (dict(ld=63), SHAPE),
        (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(n_groups=7), SHAPE), (dict(n_groups=0), SHAPE), (dict(n_groups=64), SHAPE),
        (dict(top_groups=0), SHAPE), (dict(top_groups=9), SHAPE), (dict(k=9, top_groups=1), SHAPE), (dict(scale=INF), SHAPE), (dict(scale=NAN), SHAPE),
        (dict(dtype=30, logits=A + 1), ALIGN), (dict(bias=A + 2), ALIGN), (dict(topk=A + 2), ALIGN), (dict(weights=A + 1), ALIGN),
        (dict(status=A + 2), ALIGN)]),
    ("mmvq_combine_experts", COMBINE, [
        (dict(dtype=-1), TYPE), (dict(y=None), NULL), (dict(topk=None), NULL), (dict(weights=None), NULL), (dict(token_offsets=None), NULL),
        (dict(slot_of=None), NULL), (dict(out=None), NULL), (dict(shared=None), NULL), (dict(n_tokens=-1), SHAPE), (dict(k=0), SHAPE),
        (dict(k=257), SHAPE), (dict(n_tokens=8193), SHAPE), (dict(n_experts=0), SHAPE), (dict(n_experts=4097), SHAPE), (dict(H=0), SHAPE),
        (dict(H=2 ** 24 + 1), SHAPE), (dict(n_positions=-1), SHAPE), (dict(ldr=63), SHAPE), (dict(lds=0), SHAPE), (dict(ldo=63), SHAPE),
        (dict(y=A + 2), ALIGN), (dict(dtype=1, residual=A + 1), ALIGN), (dict(slot_of=A + 2), ALIGN), (dict(out=A + 2), ALIGN)]),
    ("mmvq_token_logprobs", LOGPROBS, [
        (dict(dtype=12), TYPE), (dict(logits=None), NULL), (dict(tokens=None), NULL), (dict(logprobs=None), NULL), (dict(top_ids=None), NULL),
        (dict(top_logprobs=None), NULL), (dict(n_rows=-1), SHAPE), (dict(vocab=0), SHAPE), (dict(vocab=2 ** 24 + 1, ld=2 ** 25), SHAPE),
        (dict(ld=999), SHAPE), (dict(n_tokens=-1), SHAPE), (dict(n_tokens=65537), SHAPE), (dict(top=-1), SHAPE), (dict(top=33), SHAPE),
        (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=NAN), SHAPE), (dict(scale=INF), SHAPE), (dict(logits=A + 2), ALIGN),
        (dict(lse=A + 1), ALIGN), (dict(top_ids=A + 2), ALIGN), (dict(status=A + 3), ALIGN)]),
])
def test_bad_arguments_are_rejected_on_the_host(lib, name, base, bad):
    f = getattr(lib, name)
    assert len(base) == len(mmvq.SIGNATURES[name][1])
    for change, code in bad:
        assert set(change) <= set(base)
        assert f(*{**base, **change}.values()) == code, change
    assert f(*{**base, ("n_rows" if "n_rows" in base else "n_tokens"): 0}.values()) == mmvq.OK  # nothing to do: nothing is launched


# ------------------------------------------------------------------ binding --

class Here(Tensor):
    @property
    def device(self):
        return torch.device("cpu")


def calls_of():
    """Each operator's call on tensors that it takes, as a function of what replaces one of them."""
    f32, i32 = torch.float32, torch.int32
    q, k, pos, w = tensor((3, 4, 64), f32), tensor((3, 2, 64), f32), tensor((3,), i32), tensor((64,), f32)
    table = tensor((2, 16), torch.int64)
    logits, bias = tensor((3, 16), f32), tensor((16,), f32)
    topk, weights = tensor((3, 4), i32), tensor((3, 4), f32)
    y, offs, slot, res, gate = tensor((12, 8), f32), tensor((17,), i32), tensor((12,), i32), tensor((3, 8), f32), tensor((3,), f32)
    toks = tensor((3, 2), i32)
    out = dict(lse=tensor((3,), f32), entropy=tensor((3,), f32), logprobs=tensor((3, 2), f32), top_ids=tensor((3, 5), i32),
               top_logprobs=tensor((3, 5), f32))
    st = tensor((1,), i32)
    return [
        (lambda q, k, pos, table, qw, kw, yq, yk, st, **s: mmvq.norm_rope(q, k, pos, table, q_weight=qw, k_weight=kw, out=(yq, yk), status=st, **s),
         [q, k, pos, table, w, w.clone().as_subclass(Tensor), q.clone().as_subclass(Tensor), k.clone().as_subclass(Tensor), st]),
        (lambda x, b, ids, w, st, **s: mmvq.route_topk(x, 4, bias=b, n_groups=4, top_groups=2, out=(ids, w), status=st, **s),
         [logits, bias, topk, weights, st]),
        (lambda y, ids, w, offs, slot, r, sh, g, out, st, **s: mmvq.combine_experts(y, ids, w, offs, slot, residual=r, shared=sh, shared_gate=g,
                                                                                 out=out, status=st, **s),
         [y, topk, weights, offs, slot, res, res.clone().as_subclass(Tensor), gate, res.clone().as_subclass(Tensor), st]),
        (lambda x, t, a, b, c, d, e, st, **s: mmvq.token_logprobs(x, t, top=5, out=dict(zip(out, (a, b, c, d, e))), status=st, **s),
         [tensor((3, 50), f32), toks, *out.values(), st]),
    ]


@pytest.fixture
def launched(monkeypatch):
    import contextlib
    import types
    seen, current = [], [None]

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()
    for name in ("empty", "empty_like"):
        make = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, make=make, **kw: seen.append(current[-1]) or make(*a, **{**kw, **({"device": "cpu"} if "device" in kw else {})}).as_subclass(Tensor))

    def launch(*args):
        seen.append(("launch", args[-1]))
        return mmvq.OK
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(mmvq, "_current_device", lambda: 0)
    monkeypatch.setattr(mmvq, "lib", lambda: types.SimpleNamespace(**{n: launch for n in mmvq.SIGNATURES}))
    monkeypatch.setattr(mmvq, "_stream", lambda s: s and s.cuda_stream)
    monkeypatch.setattr(mmvq, "_raw_stream", None)
    return seen


def test_tensors_of_other_types_shapes_and_places_are_refused(launched):
    for call, args in calls_of():
        launched.clear()
        call(*args)
        assert launched == [("launch", None)]
        launched.clear()
        for i, t in enumerate(args):
            others = [t.as_subclass(torch.Tensor), t.as_subclass(Elsewhere), t.to(torch.int16).as_subclass(Tensor), t.double().as_subclass(Tensor)]
            if t.numel() > 1:
                others += [tensor((*t.shape[:-1], t.shape[-1] + 1), t.dtype), tensor((*t.shape[:-1], 2 * t.shape[-1]), t.dtype)[..., ::2]]
            else:
                others += [tensor((0,), t.dtype)]
            for other in others:
                # a longer table, more logits or lists of more slots can be right by themselves, where nothing contradicts them
                if other.dtype == t.dtype and other.shape != t.shape and other.is_contiguous() and other.is_cuda and other.get_device() == 0 and \
                        i in {9: [3], 5: [], 10: [3, 4], 8: [0]}[len(args)]:
                    continue
                with pytest.raises(ValueError):
                    call(*args[:i], other, *args[i + 1:])
        assert launched == []


def test_calls_run_and_allocate_on_the_stream_given(launched):
    import types
    side = types.SimpleNamespace(cuda_stream=77, device_index=0)
    (rope, a), (route, b), (combine, c), (logp, d) = calls_of()
    for call in (lambda: mmvq.norm_rope(*a[:4], stream=side), lambda: mmvq.route_topk(b[0], 4, stream=side),
                 lambda: mmvq.combine_experts(*c[:5], stream=side), lambda: mmvq.token_logprobs(*d[:2], top=5, stream=side)):
        launched.clear()
        call()
        assert launched[-1] == ("launch", 77) and len(launched) > 1 and all(s is side for s in launched[:-1])
    for call, args in calls_of():  # a stream of another device than the tensors'
        launched.clear()
        with pytest.raises(ValueError):
            call(*args, stream=types.SimpleNamespace(cuda_stream=77, device_index=1))
        assert launched == []


def test_other_refusals(launched):
    (_, a), (_, b), (_, c), (_, d) = calls_of()
    with pytest.raises(ValueError):
        mmvq.norm_rope(*a[:4], out=(a[6], None))
    with pytest.raises(ValueError):
        mmvq.route_topk(b[0], 4, scoring="tanh")
    with pytest.raises(ValueError):
        mmvq.combine_experts(*c[:5], dtype=torch.float64)
    with pytest.raises(ValueError):
        mmvq.combine_experts(*c[:4], c[4][:11])
    with pytest.raises(ValueError):
        mmvq.combine_experts(*c[:5], residual=c[5].expand(3, 8)[:1].expand(3, 8))  # rows that overlap
    for bad in ([], [INF], [NAN], [2.0 ** 64]):
        with pytest.raises(ValueError):
            mmvq.rope_table(bad, device="cpu")
    with pytest.raises(ValueError):
        mmvq.rope_table([1.0, 2.0], axis_of=[0], device="cpu")
    with pytest.raises(ValueError):
        mmvq.rope_table([1.0], axis_of=[4], device="cpu")
    with pytest.raises(ValueError):
        mmvq.rope_table([1.0, 0.5], sections=(1, 1), axis_of=[0, 0], device="cpu")
    with pytest.raises(ValueError):
        mmvq.rope_table([1.0, 0.5], sections=(1,), device="cpu")


def test_the_tables_steps_are_the_frequencies_in_turns():
    freqs = [1.0, 0.1, 1e4 ** -0.5, 1e-7, 7.25, 100.0, -0.3, 0.0, 2.0 ** 63, 5e-324, 1e-18]
    table = mmvq.rope_table(freqs, axis_of=range(0, 11, 1) and [i % 4 for i in range(11)], device="cpu")
    assert table.dtype == torch.int64 and table[1].tolist() == [i % 4 for i in range(11)]
    for f, step in zip(freqs, table[0].tolist()):
        turns = Fraction(f) / _layer.TWO_PI                      # pi to 60 digits: to 2^-130 of 2^63
        off = (Fraction(step, 2 ** 64) - turns) % 1
        assert min(off, 1 - off) <= Fraction(1, 2 ** 65) * Fraction(1001, 1000)
    for f, pos in ((0.3, 2 ** 31 - 1), (1.0, -2 ** 31), (1e-4, 131071)):  # as the kernel multiplies and wraps
        step = mmvq.rope_table([f], device="cpu")[0, 0].item()
        phase = step * pos % 2 ** 64 / 2 ** 64 * 2 * math.pi
        c, s = _layer.turns(pos, f)
        assert abs(math.cos(phase) - c) < 2e-9 and abs(math.sin(phase) - s) < 2e-9
