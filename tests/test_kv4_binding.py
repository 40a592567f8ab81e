"""The binding on the CPU: on which stream a call's own tensors are made, and the tensors that the 4-bit
cache's calls refuse."""
import contextlib
import types

import pytest
import torch

from block_quantized_matvec_gb300 import mmvq


class Tensor(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""
    is_cuda = True
    number = 0

    def get_device(self):
        return self.number


class Elsewhere(Tensor):
    """One that says it is on another."""
    number = 1


def tensor(shape, dtype):
    return torch.zeros(shape, dtype=dtype).as_subclass(Tensor)


def batch():
    """A cache of one page of 16 tokens, and one sequence in it."""
    return (tensor((1, 1, 1, 20 * 64), torch.uint8), tensor((1, 1), torch.int32), tensor((2,), torch.int32),
            tensor((1,), torch.int32))


@pytest.fixture
def calls(monkeypatch):
    """The stream that is current at each allocation and at each launch, the launch's last argument too."""
    seen, current = [], [None]

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def watched(name):
        make = getattr(torch, name)

        def f(*args, **kw):
            seen.append((name, current[-1]))
            return make(*args, **kw)
        return f
    for name in ("empty", "empty_like", "zeros"):
        monkeypatch.setattr(torch, name, watched(name))
    new_empty = torch.Tensor.new_empty
    monkeypatch.setattr(torch.Tensor, "new_empty", lambda t, *a, **kw: seen.append(("new_empty", current[-1])) or new_empty(t, *a, **kw))
    monkeypatch.setattr(torch.cuda, "stream", stream)

    def launch(*args):
        seen.append(("launch", args[-1]))
        return mmvq.OK
    fake = types.SimpleNamespace(mmvq_quantize_q8_1=launch, mmvq_gemv=launch, mmvq_route_groups=launch,
                                 mmvq_expert_ffn=launch, mmvq_kv4_append=launch, mmvq_kv4_read=launch,
                                 mmvq_kv4_attention=launch,
                                 mmvq_kv4_attention_workspace_bytes=lambda dim: 1024)
    monkeypatch.setattr(mmvq, "lib", lambda: fake)
    monkeypatch.setattr(mmvq, "_workspace_bytes", {})
    monkeypatch.setattr(mmvq, "_stream", lambda s: s and s.cuda_stream)
    return seen


def test_a_calls_own_tensors_are_made_on_its_stream(calls):
    """Made on another stream, they would be zeroed after the kernel began, or belong to that stream's pool while
    the kernel uses them."""
    side = types.SimpleNamespace(cuda_stream=77)
    q, where = tensor((1, 2, 64), torch.float32), batch()
    calls.clear()
    mmvq.kv4_attention(q, *where, with_lse=True, stream=side)
    assert {name for name, _ in calls} == {"empty_like", "new_empty", "zeros", "launch"}
    assert calls[-1] == ("launch", 77) and all(s is side for _, s in calls[:-1])
    calls.clear()
    mmvq.kv4_read(*where, 1, stream=side)
    assert calls[-1] == ("launch", 77) and len(calls) == 3 and all(s is side for _, s in calls[:2])


def test_so_are_the_products_and_the_expert_layers(calls):
    """The expert layer's barrier word and the routing's status are zeroed by the call."""
    side = types.SimpleNamespace(cuda_stream=77)
    x, topk, W = tensor((2, 256), torch.float32), tensor((2, 4), torch.int32), tensor((64,), torch.uint8)
    for call in (lambda: mmvq.quantize_q8_1(x, stream=side),
                 lambda: mmvq.gemv(mmvq.TYPE_Q4_K_PLANAR, W, 16, 256, W, 2, stream=side),
                 lambda: mmvq.route_groups(topk, 8, stream=side),
                 lambda: mmvq.expert_ffn(mmvq.TYPE_Q4_K_PLANAR, W, W, 8, 256, 256, x, topk, stream=side)):
        calls.clear()
        call()
        assert len(calls) > 1 and calls[-1] == ("launch", 77) and all(s is side for _, s in calls[:-1])


def test_status_and_tensors_of_other_places_are_refused(calls):
    """Their addresses go to the kernels as they are."""
    where, q, k = batch(), tensor((1, 2, 64), torch.float32), tensor((1, 1, 64), torch.float32)
    workspace = tensor((1024,), torch.uint8)
    each = (lambda w, q, k, workspace, **kw: mmvq.kv4_append(k, k, *w, **kw),
            lambda w, q, k, workspace, **kw: mmvq.kv4_read(*w, 1, **kw),
            lambda w, q, k, workspace, **kw: mmvq.kv4_attention(q, *w, workspace=workspace, **kw))
    plain = lambda t: t.as_subclass(torch.Tensor)  # noqa: E731
    for call in each:
        call(where, q, k, workspace, status=tensor((1,), torch.int32))
    calls.clear()
    for call in each:
        for status in (torch.zeros(1, dtype=torch.int32), tensor((1,), torch.int64), tensor((0,), torch.int32),
                       tensor((1,), torch.int32).as_subclass(Elsewhere)):
            with pytest.raises(ValueError):
                call(where, q, k, workspace, status=status)
        for to in (plain, lambda t: t.as_subclass(Elsewhere)):
            for i in range(4):
                with pytest.raises(ValueError):
                    call((*where[:i], to(where[i]), *where[i + 1:]), q, k, workspace)
    for to in (plain, lambda t: t.as_subclass(Elsewhere)):
        for args in ((q, to(k), workspace), (to(q), k, workspace), (q, k, to(workspace))):
            for call in (each[0], each[2]):
                if (call is each[0]) == (args[1] is not k):
                    with pytest.raises(ValueError):
                        call(where, *args)
        with pytest.raises(ValueError):
            mmvq.kv4_read(*where, 1, out=(k, to(k)))
        with pytest.raises(ValueError):
            mmvq.kv4_attention(q, *where, workspace=workspace, out=to(q.clone()))
        with pytest.raises(ValueError):
            mmvq.kv4_attention(q, *where, workspace=workspace, lse=to(tensor((1, 2), torch.float32)))
    assert not [name for name, _ in calls if name == "launch"]
