"""What the Python side of the tree operators does around a call, on a machine
without a GPU."""
import contextlib

import pytest
import torch

from speculative_decoding_verification_92_b200 import cache, tree


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


def step_on_the_cpu(monkeypatch, slots=3, nodes=4):
    """A TreeStep as its constructor leaves it, in CPU memory, whose page calls
    do nothing: what begin() does to its own tensors."""
    ints = lambda *shape: torch.zeros(shape, dtype=torch.int32)
    step = tree.TreeStep.__new__(tree.TreeStep)
    step.nodes, step.lens, step.page_table, step.refcount = nodes, ints(slots), ints(slots, 2), ints(6)
    step.k_cache = torch.zeros(1, 6, 16, 1, 64, dtype=torch.bfloat16)
    step.status, step.counts, step.parents, step._full = ints(slots), None, None, torch.full((slots,), nodes).int()
    step._want, step._counts = ints(slots), ints(slots)
    monkeypatch.setattr(tree, "cache_resize", lambda *a, **kw: None)
    return step


@pytest.mark.parametrize("shape", [(1,), (2,), (4,), (64,), (3, 1), ()])
def test_counts_of_another_shape_do_not_touch_the_step_s_tensors(monkeypatch, shape):
    """A captured graph holds the addresses of the step's tensors: a refused
    call leaves them where and as they are."""
    step = step_on_the_cpu(monkeypatch)
    own = {n: (getattr(step, n).data_ptr(), getattr(step, n).clone()) for n in ("_want", "_counts", "status", "lens")}
    with pytest.raises(ValueError):
        step.begin(counts=torch.ones(shape, dtype=torch.int32))
    for n, (at, was) in own.items():
        t = getattr(step, n)
        assert t.data_ptr() == at and t.shape == was.shape and torch.equal(t, was), n
    with pytest.raises(RuntimeError):    # and no step has begun
        step._begun()


def test_parents_are_checked_before_pages_are_taken(monkeypatch):
    step = step_on_the_cpu(monkeypatch)
    monkeypatch.setattr(tree, "cache_resize", lambda *a, **kw: pytest.fail("pages taken"))
    for want, parents in ((ValueError, torch.zeros(3, 5, dtype=torch.int32)),
                          (ValueError, torch.zeros(2, 4, dtype=torch.int32)),
                          (ValueError, torch.zeros(3, 8, dtype=torch.int32)[:, ::2]),
                          (TypeError, torch.zeros(3, 4, dtype=torch.int64))):
        with pytest.raises(want):
            step.begin(parents)


def test_counts_may_be_a_view(monkeypatch):
    step = step_on_the_cpu(monkeypatch)
    step.begin(counts=torch.tensor([2, 9, 3, 9, 4, 9], dtype=torch.int32)[::2])
    assert step._want.tolist() == [2, 3, 4] and step._begun().tolist() == [2, 3, 4]
