"""Whose buffers a layer call allocates when it is given a stream, and the tensors that the checkpointed
step refuses (no GPU: streams, kernels and the allocator's records are stood in for)."""
import contextlib

import pytest
import torch

from token_choice_routing_b200 import binding as B
from token_choice_routing_b200.layer import MoENullLayer

T, K, d, N, F = 4, 2, 128, 4, 64


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def layer(monkeypatch):
    """A layer on the CPU whose library calls do nothing, and the record of what it allocated:
    allocated[data_ptr] = the stream that was current, recorded = the (data_ptr, stream) pairs."""
    current = [Stream(1)]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream or current[-1])
        yield
        current.pop()

    real, allocated, recorded = torch.empty, {}, set()

    def empty(*a, **k):
        t = real(*a, **k)
        allocated[t.data_ptr()] = current[-1].cuda_stream
        return t

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(B, "_device", lambda: -1)      # what get_device() gives for a CPU tensor
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.add((t.data_ptr(), s.cuda_stream)))
    for n in ("sort_slots", "permute", "permute_backward", "unpermute", "unpermute_backward", "expert_gate_up",
              "expert_down", "expert_ffn_backward", "clear_device_status", "forward", "backward",
              "forward_checkpoint8", "backward_checkpoint8"):
        monkeypatch.setattr(B, n, lambda *a, **k: None)
    m = object.__new__(MoENullLayer)
    m.d, m.N, m.M, m.K, m.F, m.F_shared, m.C, m.V = d, N, 2, K, F, F, 0, 0
    m.device, m.ffn, m.flags = torch.device("cpu"), "single", 0
    m.gate_up = m.shared_gate_up = m.w_down = m.shared_down = torch.zeros(1)
    m._weights = B.Weights()
    m.allocated, m.recorded = allocated, recorded
    return m


def calls(m, stream):
    """Each call's buffers, that the call itself allocated."""
    x = torch.zeros((T, d), dtype=torch.bfloat16)
    idx, gate = torch.zeros((T, K), dtype=torch.int32), torch.zeros((T, K))
    out, routed, ck = m.alloc(T), m.alloc_routed(T, K), m.alloc_checkpoint8(T)
    m.allocated.clear()
    yield "forward", m.forward(x, stream=stream)
    yield "backward", m.backward(x, out, x, stream=stream)
    yield "backward_checkpoint8", m.backward_checkpoint8(x, ck, x, stream=stream)
    yield "forward_routed", m.forward_routed(x, idx, gate, stream=stream)
    yield "backward_routed", m.backward_routed(x, gate, routed, x, stream=stream)


def test_buffers_belong_to_the_stream_passed(layer):
    for name, bufs in calls(layer, Stream(2)):
        for n, t in bufs.items():
            if t is not None and t.numel():
                assert layer.allocated[t.data_ptr()] == 2, (name, n)
                assert (t.data_ptr(), 1) in layer.recorded, (name, n)


@pytest.mark.parametrize("stream", [None, Stream(1)])
def test_buffers_of_a_call_on_the_current_stream(layer, stream):
    for name, bufs in calls(layer, stream):
        for n, t in bufs.items():
            if t is not None and t.numel():
                assert layer.allocated[t.data_ptr()] == 1, (name, n)
    assert not layer.recorded


def test_tokens_that_the_checkpointed_step_refuses(layer, monkeypatch):
    """The library takes addresses: another type, width, layout or device would be read as bf16 rows."""
    x = torch.zeros((T, d), dtype=torch.bfloat16)
    out, ck = layer.alloc(T), layer.alloc_checkpoint8(T)
    layer.forward_checkpoint8(x, None, out, ck)
    layer.backward_checkpoint8(x, ck, x)
    for bad in (x.float(), x[:, :64], x[:, :64].contiguous(), torch.zeros((d, T), dtype=torch.bfloat16).t(),
                torch.zeros((T, 2 * d), dtype=torch.bfloat16)[:, ::2], x.view(torch.float16)):
        with pytest.raises(ValueError):
            layer.forward_checkpoint8(bad, None, out, ck)
        with pytest.raises(ValueError):
            layer.backward_checkpoint8(bad, ck, x)
        with pytest.raises(ValueError):
            layer.backward_checkpoint8(x, ck, bad)
    with pytest.raises(ValueError):
        layer.backward_checkpoint8(x, ck, x[:-1])
    monkeypatch.setattr(B, "_device", lambda: 0)
    with pytest.raises(ValueError):
        layer.forward_checkpoint8(x, None, out, ck)
    with pytest.raises(ValueError):
        layer.backward_checkpoint8(x, ck, x)
