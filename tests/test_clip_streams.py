"""Which stream the buffers of a clipping belong to (no GPU): tensors, streams and the call are stand-ins."""
import contextlib

import pytest
import torch

from differentiable_gaussian_splat_amd import optim as O


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle
        self.waited = []

    def wait_stream(self, other):
        self.waited.append(other.cuda_stream)


class Buffer:
    """A tensor's stand-in: where it was allocated, and the streams that it is said to be in use on."""
    def __init__(self, of):
        self.of, self.recorded, self.device = of, set(), 0

    def record_stream(self, stream):
        self.recorded.add(stream.cuda_stream)


@pytest.fixture
def gpu(monkeypatch):
    """A world of one current stream at a time; calls are kept as (norm, workspace, stream)."""
    state = dict(now=Stream(0), capturing=False, calls=[], made=[])
    streams = {0: state["now"]}

    @contextlib.contextmanager
    def stream(s):
        before, state["now"] = state["now"], s
        streams[s.cuda_stream] = s
        yield
        state["now"] = before

    class Tensors:
        def __init__(self, grads, outs):
            self.grads, self.outs, self.device = list(grads), list(outs), 0

        def call(self, max_norm, norm, workspace, on):
            state["calls"].append((norm, workspace, (on or state["now"]).cuda_stream))

    def empty(*_, **__):
        state["made"].append(Buffer(state["now"].cuda_stream))
        return state["made"][-1]

    monkeypatch.setattr(O, "_Tensors", Tensors)
    monkeypatch.setattr(O, "gs_clip_grads_workspace_size", lambda n: 16)
    monkeypatch.setattr(O, "_stream", lambda s, _: (s or state["now"]).cuda_stream)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: state["now"])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *_: streams[0])
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, *_: streams[h])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    return state


class Parameter:
    def __init__(self):
        self.grad = Buffer(0)


def test_a_call_on_a_stream_has_the_streams_own_buffers(gpu):
    """The handle of clip_grads is dropped when it returns: what its buffers hold must go on living on that stream."""
    params, side = [Parameter() for _ in range(3)], Stream(7)
    norm = O.clip_grads(params, 1.0, stream=side)
    (used, workspace, on), = gpu["calls"]
    assert on == 7 and used is norm and gpu["now"].cuda_stream == 0
    assert norm.of == workspace.of == 7
    assert 0 in norm.recorded  # the caller reads it on the current stream
    assert all(7 in p.grad.recorded for p in params)


def test_a_call_on_the_current_stream_records_nothing(gpu):
    params = [Parameter() for _ in range(3)]
    norm = O.clip_grads(params, 1.0)
    (_, workspace, on), = gpu["calls"]
    assert on == norm.of == workspace.of == 0 and not norm.recorded and not workspace.recorded


@pytest.mark.parametrize("named", [True, False], ids=["named", "current"])
def test_a_handle_used_on_another_stream_is_tied_to_it(gpu, named):
    """Made on one stream and called on another, named in the call or the current one then: that waits once for the
    first, and the memory is not given on before it is through."""
    grads, side = [Buffer(0), Buffer(0)], Stream(9)
    clip = O.GradClip(grads)
    for _ in range(2):
        if named:
            clip(1.0, side)
        else:
            with torch.cuda.stream(side):
                clip(1.0)
    assert [c[2] for c in gpu["calls"]] == [9, 9] and side.waited == [0]
    assert all(9 in b.recorded for b in gpu["made"] + grads)
    clip(1.0)
    assert gpu["now"].waited == []


def test_a_captured_call_waits_for_nothing(gpu):
    """A graph cannot wait for a stream that is not recorded with it."""
    grads, side = [Buffer(0)], Stream(9)
    clip = O.GradClip(grads)
    gpu["capturing"] = True
    clip(1.0, side)
    assert side.waited == [] and not grads[0].recorded
    gpu["capturing"] = False
    clip(1.0, side)
    assert side.waited == [0]


def test_a_named_stream_is_the_one_that_is_called(gpu, monkeypatch):
    """A stream of another device is not the current one of the gradients' device, whatever context it is in: it goes to
    the call, which refuses it, and nothing runs on that device's own stream instead."""
    monkeypatch.setattr(O, "_stream", lambda s, _: 0 if s is None else s.cuda_stream)
    O.clip_grads([Parameter()], 1.0, stream=Stream(7))
    assert [c[2] for c in gpu["calls"]] == [7]
