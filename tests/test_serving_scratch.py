"""Scratch memory of the serving calls (CPU): which stream the binding takes it
on and clears it on, eagerly and under capture."""
import contextlib

import pytest
import torch

from group_wise_affine_amd import qmm as Q


class Log:
    """Stands for torch in the binding: notes the stream of every allocation and
    of every clearing."""

    def __init__(self, pool):
        self.events, self.now, self.pool = [], "current", pool
        self.cuda, self.uint8 = self, torch.uint8

    def ExternalStream(self, handle, device=None):
        return handle

    @contextlib.contextmanager
    def stream(self, s):
        before, self.now = self.now, s
        yield
        self.now = before

    def empty(self, n, dtype=None, device=None):
        self.events.append(("empty", self.now))
        return Buffer(self, n)

    def memory_snapshot(self):
        return [dict(address=0, total_size=100, segment_pool_id=(0, 0)),
                dict(address=100, total_size=1 << 30, segment_pool_id=self.pool)]


class Buffer:
    def __init__(self, log, n):
        self.log, self.n = log, n

    def data_ptr(self):
        return 4096

    def __getitem__(self, s):
        return self

    def zero_(self):
        self.log.events.append(("zero", self.log.now))


@pytest.mark.parametrize("capture", [0, 1001])
def test_scratch_belongs_to_the_stream_of_the_call(monkeypatch, capture):
    log = Log((0, 7))
    monkeypatch.setattr(Q, "torch", log)
    t = Q._grow(1 << 21, 0, 77, capture)
    assert t.n == 1 << 21
    assert log.events == [("empty", 77), ("zero", 77)] and log.now == "current"


def test_capture_without_a_pool_is_refused(monkeypatch):
    """Memory of the ordinary pool would be handed out again under the graph."""
    log = Log((0, 0))
    monkeypatch.setattr(Q, "torch", log)
    with pytest.raises(ValueError, match="torch.cuda.graph"):
        Q._grow(1 << 21, 0, 77, 1002)
    assert ("zero", 77) not in log.events
    assert Q._grow(1 << 21, 0, 77, 0) is not None
