"""Where the layer and gradient-set calls take their memory from: with a stream
of the caller's, from that stream's pool.  A block of the current stream's pool
may still be used by work that is under way there, and nothing makes the
caller's stream wait for it.  Without a GPU: torch's allocation and streams are
replaced by a record of them."""

import contextlib

import pytest
import torch

from sparsified_gradient_compression_amd import dgc


class Tensor:
    """A tensor on a GPU as far as these calls look at it."""
    is_cuda, device = True, "cuda"

    def __init__(self, made_on="current"):
        self.made_on, self.recorded = made_on, []

    def get_device(self):
        return 0

    def numel(self):
        return 1 << 40

    def data_ptr(self):
        return 1 << 20

    def record_stream(self, stream):
        self.recorded.append(stream)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def torch_record(monkeypatch):
    current = [Stream(11)]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    monkeypatch.setattr(torch, "empty", lambda *a, **k: Tensor(current[-1].cuda_stream))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: current[-1].cuda_stream, raising=False)


@pytest.mark.parametrize("stream,pool", [(None, 11), (Stream(22), 22), (22, 22)])
def test_workspaces_and_outputs_come_from_the_calls_stream(torch_record, stream, pool):
    assert dgc._fresh(64, Tensor(), stream).made_on == pool
    out = dgc._new(Tensor(), (2, 3), torch.bfloat16, stream)
    assert out.made_on == pool
    # the caller's own stream uses the output as well
    assert [s.cuda_stream for s in out.recorded] == ([] if stream is None else [11])


@pytest.mark.parametrize("stream,pool", [(None, 11), (Stream(22), 22), (22, 22)])
def test_a_sets_tensors_come_from_its_stream_and_are_held_for_others(torch_record, monkeypatch, stream, pool):
    calls = []

    class Lib:
        def dgc_gradset_bytes(self, *a):
            return dgc.DGC_OK

        def dgc_gradset_init(self, out, *a):
            calls.append(a[-1])
            return dgc.DGC_OK

        def dgc_gradset_destroy(self, s):
            pass

    monkeypatch.setattr(dgc, "lib", Lib)
    s = dgc.GradSet([(4,)], [torch.float32], stream=stream)
    own = (s.workspace, s.total, s.scale)
    assert calls == [pool] and [t.made_on for t in own] == [pool] * 3
    for other in (None, Stream(22), Stream(33), 33):
        for t in own:
            t.recorded.clear()
        handle = s._on(other)
        assert handle == (11 if other is None else other if isinstance(other, int) else other.cuda_stream)
        for t in own:
            assert [r.cuda_stream for r in t.recorded] == ([] if handle == pool else [handle])
