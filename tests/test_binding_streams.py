"""Workspaces that the binding allocates itself, on the CPU with a stand-in for the library.

torch's allocator orders the reuse of a block only within the stream that was current when it was
allocated.  A call on an explicit stream must therefore allocate its workspace with that stream
current: otherwise the block may be one that a call still running on the current stream has given back.
"""
import contextlib
import types

import pytest
import torch

import parallelizable_recurrence_b200 as sru


class _Library:
    """Answers 4096 to every question for a size and SRU_OK to every call."""

    def __getattr__(self, name):
        def call(*args):
            return 4096 if name.endswith("_bytes") else 0
        call.__name__ = name
        return call


@pytest.fixture
def allocations(monkeypatch):
    """The stream that was current at each allocation that the binding made."""
    seen, current = [], []
    empty = torch.empty

    def fake_empty(*shape, **kw):
        if kw.pop("device", None) is None:
            return empty(*shape, **kw)
        seen.append(current[-1] if current else "current")
        return empty(*shape, **kw)

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    monkeypatch.setattr(torch, "empty", fake_empty)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=1))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: None)
    monkeypatch.setattr(sru, "_lib", _Library())
    monkeypatch.setattr(sru, "_raw_stream", lambda device: 1)
    monkeypatch.setattr(sru, "_device_of", lambda *tensors: 0)
    monkeypatch.setattr(sru, "_ptr", lambda t, dtype=None: None if t is None else t.data_ptr())
    return seen


def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def _i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


CALLS = {
    "sru_softmax_loss": lambda **kw: sru.sru_softmax_loss(
        _bf(4, 8), _bf(5, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4), torch.zeros(4), **kw),
    "sru_softmax_loss_backward": lambda **kw: sru.sru_softmax_loss_backward(
        _bf(4, 8), _bf(5, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4), torch.zeros(4), _bf(4, 8), _bf(5, 8),
        **kw),
    "sru_attention_decode": lambda **kw: sru.sru_attention_decode(
        _bf(3, 4, 64), _bf(4, 2, 16, 64), _bf(4, 2, 16, 64), _i32(3, 2), _i32(3), _bf(3, 4, 64), **kw),
    "sru_project_factored_backward": lambda **kw: sru.sru_project_factored_backward(
        _bf(6, 24), _bf(6, 8), _bf(4, 8), _bf(24, 4), _bf(6, 4), _bf(6, 4), **kw),
    "sru_attention_project": lambda **kw: sru.sru_attention_project(
        _bf(6, 8), _bf(4, 8), _bf(8, 4), _bf(24, 4), _bf(6, 24), 3, 2, 1.0, **kw),
    "sru_attention_project_backward": lambda **kw: sru.sru_attention_project_backward(
        _bf(6, 24), _bf(6, 8), _bf(4, 8), _bf(8, 4), _bf(24, 4), 3, 2, 1.0, _bf(8), torch.zeros(6, 8),
        torch.zeros(4, 8), torch.zeros(8, 4), torch.zeros(24, 4), **kw),
    "sru_decode_step": lambda **kw: sru.sru_decode_step(
        _bf(8, 8), _bf(24, 8), torch.zeros(8, 8), torch.zeros(2, 8), torch.zeros(2, 8), torch.zeros(8, 8),
        torch.zeros(8, 8), **kw),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_workspace_comes_from_the_stream_of_its_call(allocations, name):
    side = types.SimpleNamespace(cuda_stream=2)
    CALLS[name](stream=side)
    assert allocations == [side]
    CALLS[name]()
    assert allocations == [side, "current"]


@pytest.mark.parametrize("name", CALLS)
def test_a_given_workspace_is_used(allocations, name):
    CALLS[name](workspace=torch.zeros(4096, dtype=torch.uint8))
    assert allocations == []
