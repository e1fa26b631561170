"""Which stream a call of ``ops`` allocates on, without a GPU: the wrappers run over host
tensors with torch's stream state and the entry points replaced by recorders."""

import types

import pytest
import torch

from chunk_schedule_execution_amd import ops


class Stream:
    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


class Recorder:
    """Stands in for torch inside ``ops``: notes the stream that is current whenever memory
    is allocated or an entry point launches."""

    def __init__(self, monkeypatch):
        self.current, self.made, self.launched, self.recorded = Stream(7), [], [], []
        recorder = self

        class switch:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                self.outer, recorder.current = recorder.current, self.stream

            def __exit__(self, *a):
                recorder.current = self.outer

        cuda = types.SimpleNamespace(
            Stream=Stream, ExternalStream=Stream, stream=switch, current_device=lambda: -1,
            set_device=lambda d: None, current_stream=lambda *a: self.current, default_stream=lambda *a: Stream(0))

        def noting(f):
            def make(*a, **kw):
                t = f(*a, **kw)
                self.made.append((t, self.current.cuda_stream))
                return t
            return make

        fake = types.SimpleNamespace(**{n: getattr(torch, n) for n in ("Tensor", "float32", "bfloat16", "int32", "uint8")},
                                     cuda=cuda, empty=noting(torch.empty), empty_like=noting(torch.empty_like))
        monkeypatch.setattr(ops, "torch", fake)
        monkeypatch.setattr(ops, "_raw_stream", lambda device: self.current.cuda_stream)
        monkeypatch.setattr(ops, "_first", lambda t, name: -1)
        monkeypatch.setattr(ops, "_like", lambda *a: None)
        monkeypatch.setattr(torch.Tensor, "record_stream",
                            lambda t, s: self.recorded.append((t.data_ptr(), s.cuda_stream)), raising=False)
        for n in ("ccl_linear", "ccl_linear_backward", "ccl_grouped_linear", "ccl_grouped_linear_backward",
                  "ccl_expert_route", "ccl_expert_dispatch", "ccl_expert_combine", "ccl_expert_combine_backward"):
            monkeypatch.setattr(ops.capi, n, lambda *a: self.launched.append(a[-1]))


def calls():
    """Every function of ``ops``, sized so that each needs a workspace where it can."""
    x, w = torch.zeros(40, 33), torch.zeros(24, 33)
    z, o = torch.zeros(40, 24), torch.tensor([0, 40], dtype=torch.int32)
    ids = torch.zeros(5000, 2, dtype=torch.int32)
    flat = torch.zeros(10000, dtype=torch.int32)
    tokens, rows = torch.zeros(5000, 8), torch.zeros(10000, 8)
    return {
        "linear": lambda s: ops.linear(x, w, save_preact=True, stream=s),
        "linear_backward": lambda s: ops.linear_backward(z, x, w, preact=z, activation="silu", bias=True, stream=s),
        "grouped_linear": lambda s: ops.grouped_linear(x, w[None], o, save_preact=True, stream=s),
        "grouped_linear_backward": lambda s: ops.grouped_linear_backward(z, x, w[None], o, preact=z, activation="silu",
                                                                         bias=True, stream=s),
        "expert_route": lambda s: ops.expert_route(ids, 4, stream=s),
        "expert_dispatch": lambda s: ops.expert_dispatch(tokens, flat, 2, stream=s),
        "expert_combine": lambda s: ops.expert_combine(rows, ids, stream=s),
        "expert_combine_backward": lambda s: ops.expert_combine_backward(tokens, rows, ids, flat, stream=s),
    }


@pytest.mark.parametrize("stream,handle", [(Stream(99), 99), (99, 99), (0, 0)])
@pytest.mark.parametrize("name", list(calls()))
def test_memory_comes_from_the_calls_stream(monkeypatch, name, stream, handle):
    r = Recorder(monkeypatch)
    out = calls()[name](stream)
    out = list(out) if isinstance(out, (tuple, list)) else [out]
    assert r.launched == [handle]
    assert len(r.made) >= len(out) and all(s == handle for _, s in r.made)
    # the outputs go to the stream that was current, which is current again
    assert sorted(r.recorded) == sorted((t.data_ptr(), 7) for t in out)
    assert r.current.cuda_stream == 7


@pytest.mark.parametrize("stream", [None, Stream(7), 7])
@pytest.mark.parametrize("name", list(calls()))
def test_the_current_stream_needs_nothing(monkeypatch, name, stream):
    r = Recorder(monkeypatch)
    calls()[name](stream)
    assert r.launched == [7] and all(s == 7 for _, s in r.made) and not r.recorded


@pytest.mark.parametrize("name", list(calls()))
def test_a_stream_of_another_device_is_refused(monkeypatch, name):
    r = Recorder(monkeypatch)
    other = Stream(99)
    other.device = types.SimpleNamespace(index=3)
    with pytest.raises(ValueError, match="stream"):
        calls()[name](other)
    assert not r.launched and not r.made


def test_the_stream_is_restored_after_an_error(monkeypatch):
    r = Recorder(monkeypatch)

    def refuse(*a):
        raise RuntimeError("refused")

    monkeypatch.setattr(ops.capi, "ccl_linear", refuse)
    with pytest.raises(RuntimeError):
        calls()["linear"](Stream(99))
    assert r.current.cuda_stream == 7
