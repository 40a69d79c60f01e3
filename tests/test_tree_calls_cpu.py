"""What the Python side of the tree operators does around a call, on a machine
without a GPU."""
import contextlib

import pytest
import torch

from speculative_decoding_verification_92_b200 import cache


class Stream:
    """Stands for a CUDA stream; two of one number are the same stream."""

    def __init__(self, number):
        self.number = number

    def __eq__(self, other):
        return self.number == other.number


class Tensor:
    """Notes which stream was current when memory was taken, and whom it was
    recorded for."""

    def __init__(self, world, stream=None):
        self.world, self.device, self.taken_on, self.recorded = world, torch.device("cuda", 0), stream, []

    def new_empty(self, shape):
        return Tensor(self.world, self.world[-1])

    def record_stream(self, stream):
        self.recorded.append(stream.number)


@pytest.fixture
def world(monkeypatch):
    current = [Stream(0)]

    @contextlib.contextmanager
    def made_current(stream):
        current.append(stream)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "stream", made_current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    return current


def test_a_call_s_own_tensors_come_from_the_memory_of_its_stream(world):
    """A block of the current stream's memory may still be written by work that
    is pending there; the call's stream must not be given it."""
    like = Tensor(world)
    assert cache._fresh(like, (4,), None).taken_on.number == 0
    t = cache._fresh(like, (4,), Stream(7))
    assert t.taken_on.number == 7 and len(world) == 1
    assert 7 not in t.recorded       # its own stream: nothing to record


def test_an_output_is_kept_from_reuse_while_the_caller_s_stream_reads_it(world):
    assert cache._fresh(Tensor(world), (4,), Stream(7)).recorded == [0]
    assert cache._fresh(Tensor(world), (4,), Stream(0)).recorded == []   # one stream: nothing to record
    assert cache._fresh(Tensor(world), (4,), Stream(7), own=True).recorded == []
