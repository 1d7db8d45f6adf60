"""On which stream the paged cache's binding allocates and what it records (no GPU needed:
the library, the allocator and the streams are fakes)."""
import contextlib
import types

import pytest
import torch

import attention_scored_kv_gb300 as kvs
from attention_scored_kv_gb300 import paged


class Tensor(torch.Tensor):
    def record_stream(self, s):
        self.log.append(s)


def stream(raw, index=0):
    return types.SimpleNamespace(cuda_stream=raw, device=torch.device("cuda", index))


@pytest.fixture
def world(monkeypatch):
    """A cache whose allocations and launches are noted with the stream that they are on."""
    w = types.SimpleNamespace(current=stream(1), allocated=[], launched=[])

    @contextlib.contextmanager
    def on(s):
        before, w.current = w.current, s or w.current
        yield
        w.current = before

    def empty(shape, dtype, device):
        t = torch.empty(shape, dtype=dtype).as_subclass(Tensor)
        t.log = []
        w.allocated.append((t, w.current))
        return t

    class Lib:
        def __getattr__(self, name):
            if name.endswith("scratch_bytes"):
                return lambda *a: 256
            return lambda *a: w.launched.append((name, a[-1])) or 0

    monkeypatch.setattr(paged, "_empty", empty)
    monkeypatch.setattr(paged, "_raw_stream", lambda index: w.current.cuda_stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w.current)
    c = object.__new__(kvs.PagedCache)
    c.device, c._index, c._lib, c._ctx, c._streams = torch.device("cuda", 0), 0, Lib(), None, set()
    c.in_dtype, c._row, c._qrow = torch.bfloat16, (2, 64), (8, 64)
    c.workspace = torch.empty(1).as_subclass(Tensor)
    c.workspace.log = []
    c._need = lambda t, name, dtype, shape: t.data_ptr()
    c._need_dims = lambda t, name, dtype, dims: t.shape
    w.cache = c
    ints = torch.zeros(3, dtype=torch.int32)
    table, q, one = torch.zeros((3, 4), dtype=torch.int32), torch.zeros((3, 8, 64)), ints[:1]
    kv = torch.zeros((3, 2, 64))
    w.calls = {
        "plan": lambda s: c.plan(ints, ints, table, ints, one, 5, stream=s),
        "slot_map": lambda s: c.slot_map(ints, table, 5, stream=s),
        "gather": lambda s: c.gather(0, ints, stream=s),
        "attend": lambda s: c.attend(0, q, table, ints, stream=s),
        "append": lambda s: c.append(0, kv, kv, ints, stream=s),
        "release": lambda s: c.release(ints, table, ints, one, stream=s),
    }
    return w


@pytest.mark.parametrize("name", ["plan", "slot_map", "gather", "attend"])
def test_memory_is_allocated_on_the_stream_of_the_call(world, name):
    """Memory of the current stream may still be in use there when another stream writes it."""
    side = stream(9)
    world.calls[name](side)
    assert world.allocated and all(s is side for _, s in world.allocated)
    assert all(t.log == [world.current] for t, _ in world.allocated)      # used on the current stream afterwards
    assert [raw for _, raw in world.launched] == [9]


@pytest.mark.parametrize("name", ["plan", "slot_map", "gather", "attend"])
def test_without_a_stream_everything_is_on_the_current_one(world, name):
    world.calls[name](None)
    assert world.allocated and all(s is world.current for _, s in world.allocated)
    assert [raw for _, raw in world.launched] == [1]


@pytest.mark.parametrize("name", ["plan", "slot_map", "gather", "attend", "append", "release"])
def test_the_workspace_is_recorded_on_every_stream(world, name):
    side, other = stream(9), stream(11)
    for s in (side, None, other, side, None):
        world.calls[name](s)
    assert world.cache.workspace.log == [side, world.current, other]


@pytest.mark.parametrize("name", ["plan", "slot_map", "gather", "attend", "append", "release"])
def test_streams_of_other_devices_are_refused(world, name):
    with pytest.raises(ValueError):
        world.calls[name](stream(9, index=1))
    assert not world.launched
